// The choice of a token's experts from the router's logits l: scores s =
// softmax l over all experts, or s = 1 / (1 + e^-l); c = s + b with a bias b
// for balance. With groups of consecutive experts, a group's score is the sum
// of its one or two largest c, and the experts of the top_groups groups with
// the largest score stand for election; the k with the largest c are the
// token's, in descending order (ties: the lower index first), and their
// weights are p = scale s, or scale s / (the sum of the k's s).
//
// c is compared in 64 bits, so that the choice is that of the formulas and
// not of a rounding. Without a bias experts are compared by their logits,
// which have the order of the scores.
//
// A wave has a token, a lane experts lane, 64 + lane, ..
#include "route.hpp"
#include "rowio.hpp"

namespace sffn {
namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// A value as an integer of the same order (NaN above everything, the two
// zeros equal), so that ranks are unique whatever the values.
__device__ __forceinline__ long long order_key(double l) {
  if (l != l) return 0x7FF8000000000000ll;
  const long long b = __double_as_longlong(l + 0.0);
  return b < 0 ? b ^ 0x7FFFFFFFFFFFFFFFll : b;
}
constexpr long long kNone = (long long)0x8000000000000000ull;   // below every value's key

__device__ __forceinline__ float logit(const RouteArgs& a, int64_t t, int e) {
  return a.bf ? bf16lo(((const uint16_t*)a.logits)[t * a.ldl + e])
              : ((const float*)a.logits)[t * a.ldl + e];
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// The scores of the lane's experts in 64 bits. (Of a row without a logit above
// -infinity they are 0.)
template <int N>
__device__ __forceinline__ void scores(const RouteArgs& a, const float (&l)[N], double (&s)[N]) {
  const int lane = threadIdx.x & 63;
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    return;
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, l[i]);   // (a NaN is ignored here)
  m = wave_max(m);
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i] = i * 64 + lane < a.E && m != -INFINITY ? exp((double)l[i] - (double)m) : 0.0;
    if (l[i] != l[i]) s[i] = l[i];
    sum += s[i];
  }
  sum = wave_sum(sum);
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = sum == 0.0 ? 0.0 : s[i] / sum;
}

template <int N>
__global__ __launch_bounds__(kWaves * 64) void route_kernel(RouteArgs a) {
  __shared__ double cs[kWaves][N * 64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= a.T || (a.t_dev && t >= *a.t_dev)) return;
  float l[N];
#pragma unroll
  for (int i = 0; i < N; ++i) l[i] = i * 64 + lane < a.E ? logit(a, t, i * 64 + lane) : -INFINITY;
  double s[N];
  scores<N>(a, l, s);
  long long key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = i * 64 + lane;
    key[i] = e < a.E ? order_key(a.bias ? s[i] + (double)a.bias[e] : (double)l[i]) : kNone;
  }
  if (a.top_groups < a.groups) {
    // (a wave's own part of LDS: no barrier)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = i * 64 + lane;
      cs[wave][e] = a.bias && e < a.E ? s[i] + (double)a.bias[e] : s[i];
    }
    __builtin_amdgcn_wave_barrier();
    long long gk = kNone;
    if (lane < a.groups) {
      double b1 = -INFINITY, b2 = -INFINITY;
      bool nan = false;
      for (int j = 0; j < a.per; ++j) {
        const double c = cs[wave][lane * a.per + j];
        nan |= c != c;
        if (c > b1) {
          b2 = b1;
          b1 = c;
        } else if (c > b2) {
          b2 = c;
        }
      }
      gk = order_key(nan ? NAN : a.best == 2 ? b1 + b2 : b1);
    }
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const long long o = __shfl(gk, g);
      before += o > gk || (o == gk && g < lane);
    }
    const uint64_t keep = __ballot(lane < a.groups && before < a.top_groups);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = i * 64 + lane;
      if (e < a.E && !((keep >> (e / a.per)) & 1)) key[i] = kNone;
    }
  }
  // the k largest, one after the other; lane r takes that of rank r
  int id = 0;
  float lr = -INFINITY;
  double sr = 0.0;
  for (int r = 0; r < a.k; ++r) {
    long long bk = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < N; ++i)
      if (key[i] > bk) {
        bk = key[i];
        bi = i;
      }
    int be = bi * 64 + lane;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const long long ok = __shfl_xor(bk, o);
      const int oe = __shfl_xor(be, o);
      if (ok > bk || (ok == bk && oe < be)) {
        bk = ok;
        be = oe;
      }
    }
    double sv = 0.0;
    float lv = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i == be >> 6) {
        sv = s[i];
        lv = l[i];
        if (lane == (be & 63)) key[i] = kNone;
      }
    sv = __shfl(sv, be & 63);
    lv = __shfl(lv, be & 63);
    if (lane == r) {
      id = be;
      sr = sv;
      lr = lv;
    }
  }
  if (a.normalize) {
    if (!a.sigmoid) {
      // relative to the chosen ones' largest logit: a bias may choose experts
      // whose scores are nothing beside the others'
      const float m = wave_max(lane < a.k ? lr : -INFINITY);
      const double ex = lane < a.k && m != -INFINITY ? exp((double)lr - (double)m) : 0.0;
      sr = lane < a.k && lr != lr ? (double)lr : ex;
    }
    const double sum = wave_sum(lane < a.k ? sr : 0.0);
    sr = sum == 0.0 ? 0.0 : sr / sum;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id;
    a.probs[t * a.k + lane] = (float)(sr * (double)a.scale);
  }
}

// The logits' gradient. With g_r = scale dp_r of the chosen experts,
//   scores' gradient: normalised ds_r = (g_r - sum_q g_q s_q / S) / S, S the
//   sum of the chosen s, else ds_r = g_r; 0 for the others
//   softmax: dl = s (ds - sum ds s), sigmoid: dl = ds s (1 - s).
// Normalised softmax weights are the softmax q over the chosen experts alone:
// dl_r = q_r (g_r - sum g q), nothing for the others.
template <int N>
__global__ __launch_bounds__(kWaves * 64) void route_grad_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= a.T || (a.t_dev && t >= *a.t_dev)) return;
  // lane r: the expert of rank r (none where the index is not one)
  int id = -1;
  float g = 0.0f, lr = -INFINITY;
  if (lane < a.k) {
    id = a.ids[t * a.k + lane];
    if (id < 0 || id >= a.E) id = -1;
    if (id >= 0) {
      g = a.scale * a.dprobs[t * a.k + lane];
      lr = logit(a, t, id);
    }
  }
  const bool all = !a.sigmoid && !a.normalize;
  float l[N], m = 0.0f, total = 0.0f, dr;
  if (all) {
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = i * 64 + lane < a.E ? logit(a, t, i * 64 + lane) : -INFINITY;
    m = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, l[i]);
    m = wave_max(m);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      l[i] = i * 64 + lane < a.E && m != -INFINITY ? expf(l[i] - m) : 0.0f;
      total += l[i];
    }
    total = wave_sum(total);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] *= inv;
    const float s = id >= 0 && m != -INFINITY ? expf(lr - m) * inv : 0.0f;
    total = wave_sum(g * s);     // sum ds s
    dr = g;
  } else if (a.sigmoid) {
    const float s = id >= 0 ? 1.0f / (1.0f + expf(-lr)) : 0.0f;
    const float c = id >= 0 ? 1.0f / (1.0f + expf(lr)) : 0.0f;    // 1 - s
    dr = g;
    if (a.normalize) {
      const float S = wave_sum(s);
      const float inv = S == 0.0f ? 0.0f : 1.0f / S;
      dr = (g - wave_sum(g * s) * inv) * inv;
    }
    dr *= s * c;
  } else {
    m = wave_max(lr);
    const float ex = id >= 0 && m != -INFINITY ? expf(lr - m) : 0.0f;
    const float S = wave_sum(ex);
    const float q = S == 0.0f ? 0.0f : ex / S;
    dr = q * (g - wave_sum(g * q));
  }
  float d[N] = {};
  for (int r = 0; r < a.k; ++r) {
    const int e = __shfl(id, r);
    const float v = __shfl(dr, r);
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] += e == i * 64 + lane ? v : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = i * 64 + lane;
    if (e >= a.E) break;
    const float v = all ? l[i] * (d[i] - total) : d[i];
    if (a.dl_bf) st((uint16_t*)a.dl + t * a.lddl + e, v);
    else st((float*)a.dl + t * a.lddl + e, v);
  }
}

template <typename F>
hipError_t by_experts(int E, F&& f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((a.T + kWaves - 1) / kWaves);
  return by_experts(a.E, [&](auto n) {
    route_kernel<decltype(n)::value><<<grid, kWaves * 64, 0, s>>>(a);
  });
}
hipError_t launch_route_grad(const RouteArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((a.T + kWaves - 1) / kWaves);
  return by_experts(a.E, [&](auto n) {
    route_grad_kernel<decltype(n)::value><<<grid, kWaves * 64, 0, s>>>(a);
  });
}

}  // namespace sffn
