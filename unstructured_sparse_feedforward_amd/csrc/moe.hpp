// A mixture-of-experts layer for few tokens (moe.hip), as api_moe.hip
// launches it.
#pragma once

#include "mx.hpp"

namespace sffn {

constexpr int kMoeMaxT = 256;      // tokens a call
constexpr int kMoeMaxE = 1024;     // experts
constexpr int kMoeMaxK = 32;       // experts a token
constexpr int kMoeSlice = 128;     // most neurons of an expert a workgroup

struct MoeArgs {
  const uint16_t* x;         // [T, d] bf16
  const uint16_t* router;    // [E, d] bf16
  const void* wg;            // [E, F, d] bf16, or the codes of [E F, d]
  const void* wu;            // nullptr: non-gated
  const void* wd;
  const uint8_t* sg;         // MXFP4 scales
  const uint8_t* su;
  const uint8_t* sd;
  int T, d, F, E, k;
  int normalize;
  const int32_t* t_dev;      // nullable: the number of valid tokens
  int nb;                    // neurons a workgroup (a multiple of 32)
  int S;                     // workgroups an expert: ceil(F / nb)
  long long* keys;           // [T, E] the logits as ordered integers
  long long* chosen;         // [T, k] the selected experts' keys, by rank
  float* part;               // [S, T k, d] partial outputs of each (token, rank)
  float* y;                  // [T, d]
  int32_t* ids;              // [T, k] (nullable)
  float* probs;              // [T, k] (nullable)
};

// neurons a workgroup and workgroups an expert for T tokens
void moe_slices(int T, int F, int E, int k, int* nb, int* S);
hipError_t launch_moe(bool mx, const MoeArgs& a, hipStream_t s);

}  // namespace sffn
