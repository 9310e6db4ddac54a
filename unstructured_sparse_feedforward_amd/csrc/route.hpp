// The choice of a token's experts (route.hip), as api_route.hip launches it.
#pragma once

#include "sffn_internal.hpp"

namespace sffn {

constexpr int kRouteMaxE = 1024;   // experts
constexpr int kRouteMaxK = 32;     // experts a token
constexpr int kRouteMaxG = 64;     // groups

struct RouteArgs {
  const void* logits;        // [T, E] float32 or bf16
  const float* bias;         // [E], nullable
  const int32_t* t_dev;      // nullable: the number of valid tokens
  int64_t ldl;
  int64_t T;
  int E, k, groups, per, top_groups, best;   // per: experts a group
  int sigmoid, normalize, bf;
  float scale;
  float inv_per;             // 1 / per
  int lp[3];                 // log2 of a group's lanes, of 64, 32 and 16 a token
  int32_t* ids;              // [T, k]
  float* probs;              // [T, k]
  // backward
  const float* dprobs;       // [T, k]
  void* dl;                  // [T, E]
  int64_t lddl;
  int dl_bf;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_route_grad(const RouteArgs& a, hipStream_t s);

}  // namespace sffn
