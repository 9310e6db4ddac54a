// C ABI of the expert layer (sffn_moe_*): argument validation, workspace
// layout and launches. See include/sffn.h for the contract.
#include "moe.hpp"
#include "sffn.h"

namespace {

using namespace sffn;

constexpr size_t kAlign = 256;

bool aligned(const void* p, size_t a) { return p != nullptr && (uintptr_t)p % a == 0; }

sffn_status validate(const sffn_moe_desc* D) {
  if (!D) return SFFN_E_ARG;
  if (D->d < 1 || D->d_ff < 1 || D->n_experts < 1 || D->top_k < 1) return SFFN_E_ARG;
  if ((D->gated != 0 && D->gated != 1) || (D->normalize != 0 && D->normalize != 1))
    return SFFN_E_ARG;
  if (D->weights != SFFN_BF16 && D->weights != SFFN_MXFP4) return SFFN_E_ARG;
  if (D->top_k > D->n_experts) return SFFN_E_ARG;
  if (D->d % 128 != 0 || D->d > 8192 || D->d_ff % 32 != 0 || D->d_ff > 65536)
    return SFFN_E_UNSUPPORTED;
  if (D->n_experts > kMoeMaxE || D->top_k > kMoeMaxK ||
      (int64_t)D->n_experts * D->d_ff > (int64_t)1 << 27)
    return SFFN_E_UNSUPPORTED;
  return SFFN_OK;
}

struct Layout {
  size_t keys, expert, weight, on, h, part, total;
};

// the sizes of a call, with what moe_plan derives from them (given: the caller
// chooses the experts)
MoeArgs sizes(const sffn_moe_desc& D, int64_t T, const int32_t* given) {
  MoeArgs a = {};
  a.in_ids = given;
  a.T = (int)T;
  a.d = D.d;
  a.F = D.d_ff;
  a.E = D.n_experts;
  a.k = D.top_k;
  a.normalize = D.normalize;
  moe_plan(D.weights == SFFN_MXFP4, &a);
  return a;
}

Layout layout(const MoeArgs& a) {
  Layout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + kAlign - 1) / kAlign * kAlign;
    return at;
  };
  const size_t T = a.T, pairs = T * a.k;
  L.keys = take(T * a.E * 8);
  L.expert = take(pairs * 4);
  L.weight = take(pairs * 4);
  L.on = take((size_t)a.zh * a.Y * a.F);
  L.h = take(pairs * a.F * 4);
  L.part = take((size_t)a.split * pairs * a.d * 4);
  L.total = o;
  return L;
}

// a call whose experts come from its router, or are ids and probs
sffn_status forward(const sffn_moe_desc& D, const void* x, const sffn_moe_weights* w, int64_t T,
                    const int32_t* n_tokens, float* y, const int32_t* in_ids,
                    const float* in_probs, int32_t* ids, float* probs, void* ws, size_t ws_bytes,
                    hipStream_t stream) {
  const bool mx = D.weights == SFFN_MXFP4;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(w->gate, 16) || !aligned(w->down, 16))
    return SFFN_E_ARG;
  if (in_ids ? w->router != nullptr : !aligned(w->router, 16)) return SFFN_E_ARG;
  if (D.gated ? !aligned(w->up, 16) : w->up != nullptr) return SFFN_E_ARG;
  if (mx) {
    if (!aligned(w->gate_scales, 4) || !aligned(w->down_scales, 4)) return SFFN_E_ARG;
    if (D.gated ? !aligned(w->up_scales, 4) : w->up_scales != nullptr) return SFFN_E_ARG;
  } else if (w->gate_scales || w->up_scales || w->down_scales) {
    return SFFN_E_ARG;
  }
  if ((n_tokens && !aligned(n_tokens, 4)) || (ids && !aligned(ids, 4)) ||
      (probs && !aligned(probs, 4)))
    return SFFN_E_ARG;
  MoeArgs a = sizes(D, T, in_ids);
  const Layout L = layout(a);
  if (!aligned(ws, kAlign) || ws_bytes < L.total) return SFFN_E_ARG;
  char* base = (char*)ws;
  a.x = (const uint16_t*)x;
  a.router = (const uint16_t*)w->router;
  a.in_probs = in_probs;
  a.wg = w->gate;
  a.wu = w->up;
  a.wd = w->down;
  a.sg = w->gate_scales;
  a.su = w->up_scales;
  a.sd = w->down_scales;
  a.t_dev = n_tokens;
  a.keys = (long long*)(base + L.keys);
  a.expert = (int32_t*)(base + L.expert);
  a.weight = (float*)(base + L.weight);
  a.on = (uint8_t*)(base + L.on);
  a.h = (float*)(base + L.h);
  a.part = (float*)(base + L.part);
  a.y = y;
  a.ids = ids;
  a.probs = probs;
  return launch_moe(mx, a, stream) == hipSuccess ? SFFN_OK : SFFN_E_HIP;
}

}  // namespace

extern "C" {

sffn_status sffn_moe_workspace_bytes(const sffn_moe_desc* desc, int64_t T, size_t* bytes) {
  const sffn_status st = validate(desc);
  if (st != SFFN_OK) return st;
  if (!bytes || T < 0) return SFFN_E_ARG;
  if (T > SFFN_MOE_MAX_TOKENS) return SFFN_E_UNSUPPORTED;
  // (of either call: any pointer says that the experts are given)
  static const int32_t given = 0;
  const size_t own = T == 0 ? 0 : layout(sizes(*desc, T, nullptr)).total;
  const size_t other = T == 0 ? 0 : layout(sizes(*desc, T, &given)).total;
  *bytes = own > other ? own : other;
  return SFFN_OK;
}

sffn_status sffn_moe_forward(const sffn_moe_desc* desc, const void* x, const sffn_moe_weights* w,
                             int64_t T, const int32_t* n_tokens, float* y, int32_t* ids,
                             float* probs, void* ws, size_t ws_bytes, hipStream_t stream) {
  const sffn_status st = validate(desc);
  if (st != SFFN_OK) return st;
  if (!w || T < 0) return SFFN_E_ARG;
  if (T > SFFN_MOE_MAX_TOKENS) return SFFN_E_UNSUPPORTED;
  if (T == 0) return SFFN_OK;
  return forward(*desc, x, w, T, n_tokens, y, nullptr, nullptr, ids, probs, ws, ws_bytes, stream);
}

sffn_status sffn_moe_forward_chosen(const sffn_moe_desc* desc, const void* x,
                                    const sffn_moe_weights* w, int64_t T, const int32_t* n_tokens,
                                    const int32_t* ids, const float* probs, float* y, void* ws,
                                    size_t ws_bytes, hipStream_t stream) {
  const sffn_status st = validate(desc);
  if (st != SFFN_OK) return st;
  if (!w || T < 0) return SFFN_E_ARG;
  if (T > SFFN_MOE_MAX_TOKENS) return SFFN_E_UNSUPPORTED;
  if (T == 0) return SFFN_OK;
  if (!aligned(ids, 4) || !aligned(probs, 4)) return SFFN_E_ARG;
  return forward(*desc, x, w, T, n_tokens, y, ids, probs, nullptr, nullptr, ws, ws_bytes, stream);
}

}  // extern "C"
