// C ABI of the expert router (sffn_route*): argument validation and
// launches. See include/sffn.h for the contract.
#include <cmath>

#include "place.hpp"
#include "route.hpp"
#include "sffn.h"

namespace {

using namespace sffn;

constexpr int64_t kMaxTokens = (int64_t)1 << 25;    // 64 threads each, below 2^32 a launch

bool aligned(const void* p, size_t a) { return p != nullptr && (uintptr_t)p % a == 0; }
int elem(int32_t dt) { return dt == SFFN_BF16 ? 2 : 4; }
bool floats(const void* p, int32_t dt) {
  return (dt == SFFN_F32 || dt == SFFN_BF16) && aligned(p, elem(dt));
}

sffn_status validate(const sffn_route_desc* D, RouteArgs* a) {
  if (!D) return SFFN_E_ARG;
  if (D->n_experts < 1 || D->top_k < 1 || D->groups < 1 || D->top_groups < 1) return SFFN_E_ARG;
  if (D->sigmoid != 0 && D->sigmoid != 1) return SFFN_E_ARG;
  if (D->normalize != 0 && D->normalize != 1) return SFFN_E_ARG;
  if (D->group_best != 1 && D->group_best != 2) return SFFN_E_ARG;
  if (!std::isfinite(D->scale)) return SFFN_E_ARG;
  if (D->n_experts % D->groups != 0 || D->top_groups > D->groups) return SFFN_E_ARG;
  const int per = D->n_experts / D->groups;
  if (D->group_best > per || (int64_t)D->top_k > (int64_t)D->top_groups * per) return SFFN_E_ARG;
  if (D->n_experts > kRouteMaxE || D->top_k > kRouteMaxK || D->groups > kRouteMaxG)
    return SFFN_E_UNSUPPORTED;
  a->E = D->n_experts;
  a->k = D->top_k;
  a->groups = D->groups;
  a->per = per;
  a->top_groups = D->top_groups;
  a->best = D->group_best;
  a->sigmoid = D->sigmoid;
  a->normalize = D->normalize;
  a->scale = D->scale;
  a->inv_per = 1.0f / (float)per;
  return SFFN_OK;
}

sffn_status tokens(int64_t T, const int32_t* n_tokens) {
  if (T < 0 || (n_tokens && !aligned(n_tokens, 4))) return SFFN_E_ARG;
  return T > kMaxTokens ? SFFN_E_UNSUPPORTED : SFFN_OK;
}

}  // namespace

extern "C" {

sffn_status sffn_route(const sffn_route_desc* desc, const void* logits, int32_t dtype, int64_t T,
                       int64_t ldl, const float* bias, const int32_t* n_tokens, int32_t* ids,
                       float* probs, hipStream_t stream) {
  RouteArgs a = {};
  sffn_status st = validate(desc, &a);
  if (st == SFFN_OK) st = tokens(T, n_tokens);
  if (st != SFFN_OK) return st;
  if (T == 0) return SFFN_OK;
  if (!floats(logits, dtype) || ldl < a.E || (bias && !aligned(bias, 4)) || !aligned(ids, 4) ||
      !aligned(probs, 4))
    return SFFN_E_ARG;
  a.logits = logits;
  a.bf = dtype == SFFN_BF16;
  a.ldl = ldl;
  a.T = T;
  a.bias = bias;
  a.t_dev = n_tokens;
  a.ids = ids;
  a.probs = probs;
  return launch_route(a, stream) == hipSuccess ? SFFN_OK : SFFN_E_HIP;
}

sffn_status sffn_route_backward(const sffn_route_desc* desc, const float* dprobs,
                                const void* logits, int32_t dtype, int64_t T, int64_t ldl,
                                const int32_t* ids, const int32_t* n_tokens, void* dlogits,
                                int32_t dl_dtype, int64_t lddl, hipStream_t stream) {
  RouteArgs a = {};
  sffn_status st = validate(desc, &a);
  if (st == SFFN_OK) st = tokens(T, n_tokens);
  if (st != SFFN_OK) return st;
  if (T == 0) return SFFN_OK;
  if (!floats(logits, dtype) || ldl < a.E || !aligned(dprobs, 4) || !aligned(ids, 4) ||
      !floats(dlogits, dl_dtype) || lddl < a.E)
    return SFFN_E_ARG;
  const int e = elem(dtype), de = elem(dl_dtype);
  if (meeting({logits, T, ldl * e, (int64_t)a.E * e, e},
              {dlogits, T, lddl * de, (int64_t)a.E * de, de}) == kMixed)
    return SFFN_E_ARG;
  a.logits = logits;
  a.bf = dtype == SFFN_BF16;
  a.ldl = ldl;
  a.T = T;
  a.t_dev = n_tokens;
  a.ids = const_cast<int32_t*>(ids);
  a.dprobs = dprobs;
  a.dl = dlogits;
  a.dl_bf = dl_dtype == SFFN_BF16;
  a.lddl = lddl;
  return launch_route_grad(a, stream) == hipSuccess ? SFFN_OK : SFFN_E_HIP;
}

}  // extern "C"
