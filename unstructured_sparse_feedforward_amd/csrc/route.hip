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
// A wave has a token, or, of many, LPT of its lanes have one, a lane N
// consecutive experts. Bytes are few (8192 tokens of 256 experts: 8.9 MB, 2 us);
// the time is that of the waves' instructions, most of them for the k maxima. So
// a token is first done in 32 bits, with a check that every comparison that
// matters was clear of the roundings, and in 64 only where one was not (a few
// tokens in a thousand).
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
__device__ __forceinline__ int order_key(float l) {
  if (l != l) return 0x7FC00000;
  const int b = __float_as_int(l + 0.0f);
  return b < 0 ? b ^ 0x7FFFFFFF : b;
}
__device__ __forceinline__ float key_value(int k) {
  return __int_as_float(k < 0 ? k ^ 0x7FFFFFFF : k);
}
// below every value's key
constexpr long long kNone64 = (long long)0x8000000000000000ull;
constexpr int kNone = (int)0x80000000u;

__device__ __forceinline__ float logit(const RouteArgs& a, int64_t t, int e) {
  return a.bf ? bf16lo(((const uint16_t*)a.logits)[t * a.ldl + e])
              : ((const float*)a.logits)[t * a.ldl + e];
}

// N consecutive elements of a row, those from `left` on as `fill`
template <int N, typename E>
__device__ __forceinline__ void load_run(const E* p, int left, float fill, float (&v)[N]) {
  if (left >= N) {
    if constexpr (N == 16) {
      load8(p, v);
      load8(p + 8, v + 8);
    } else if constexpr (N == 8) {
      load8(p, v);
    } else if constexpr (N == 4) {
      load4(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = ld(p + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < left ? ld(p + i) : fill;
  }
}
template <int N, typename E>
__device__ __forceinline__ void store_run(E* p, int left, const float (&v)[N]) {
  if (left >= N) {
    if constexpr (N == 16) {
      store8(p, v);
      store8(p + 8, v + 8);
    } else if constexpr (N == 8) {
      store8(p, v);
    } else if constexpr (N == 4) {
      store4(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) st(p + i, v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) st(p + i, v[i]);
  }
}
// A lane's place: seg the first lane of its token's, pos its own among them.
template <int LPT>
__device__ __forceinline__ int seg_of(int lane) { return LPT == 64 ? 0 : lane & -LPT; }
template <int LPT>
__device__ __forceinline__ int pos_of(int lane) { return LPT == 64 ? lane : lane & (LPT - 1); }

template <int N>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, int e0, int left,
                                            float (&l)[N]) {
  if (a.bf) load_run<N>((const uint16_t*)a.logits + t * a.ldl + e0, left, -INFINITY, l);
  else load_run<N>((const float*)a.logits + t * a.ldl + e0, left, -INFINITY, l);
}

// sums and maxima over a token's lanes, in all of them
template <int LPT, typename T>
__device__ __forceinline__ T seg_sum(T v) {
#pragma unroll
  for (int o = 1; o < LPT; o <<= 1) v += __shfl_xor(v, o);
  return v;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) { return seg_sum<64>(v); }
// the sum over the token's first k lanes (the others have 0), in those
__device__ __forceinline__ double lanes_sum(double v, int k) {
#pragma unroll 1
  for (int o = 1; o < k; o <<= 1) v += __shfl_xor(v, o);
  return v;
}
#define SFFN_DPP(ctrl) v = max(v, __builtin_amdgcn_update_dpp(v, v, ctrl, 0xF, 0xF, false))
// a scan by lanes of a row of 16, then rows into the next ones; the last lane
// has it
__device__ __forceinline__ int wave_max(int v) {
  SFFN_DPP(0x111);    // from the lane 1, 2, 4, 8 before, of the same 16
  SFFN_DPP(0x112);
  SFFN_DPP(0x114);
  SFFN_DPP(0x118);
  SFFN_DPP(0x142);    // the last of a row of 16 to the next row
  SFFN_DPP(0x143);    // lane 31 to the upper half
  return __builtin_amdgcn_readlane(v, 63);
}
template <int LPT>
__device__ __forceinline__ int seg_max(int v) {
  if constexpr (LPT == 64) return wave_max(v);
  SFFN_DPP(0xB1);     // neighbours, pairs, halves and wholes of a row of 16
  SFFN_DPP(0x4E);
  SFFN_DPP(0x141);
  SFFN_DPP(0x140);
  if constexpr (LPT == 32) {
    const auto o = __builtin_amdgcn_permlane16_swap(v, v, false, false);   // and of two rows
    v = max((int)o[0], (int)o[1]);
  }
  return v;
}
#undef SFFN_DPP
// (a NaN is ignored)
template <int LPT>
__device__ __forceinline__ float seg_max(float v) {
  return key_value(seg_max<LPT>(v != v ? kNone : order_key(v)));
}
__device__ __forceinline__ float wave_max(float v) { return seg_max<64>(v); }
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// the logit of the token's expert e, by lane
template <int N>
__device__ __forceinline__ float value_of(const float (&l)[N], int seg, int e) {
  float v = __shfl(l[0], seg + e / N);
#pragma unroll
  for (int i = 1; i < N; ++i) {
    const float o = __shfl(l[i], seg + e / N);
    v = e % N == i ? o : v;
  }
  return v;
}

// The largest of a row's logits; -infinity of an empty one.
template <int N, int LPT>
__device__ __forceinline__ float row_max(const float (&l)[N]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, l[i]);
  m = seg_max<LPT>(m);
  return m != m ? -INFINITY : m;     // (every one a NaN)
}

// A wave's own part of LDS holds 32-bit scores, then 64-bit ones, then their
// keys, for one token after the other: bytes, accessed as one type or another.
template <typename T>
__device__ __forceinline__ T lds_get(const char* p, int i) {
  T v;
  __builtin_memcpy(&v, __builtin_assume_aligned(p + i * sizeof(T), sizeof(T)), sizeof(T));
  return v;
}
template <typename T>
__device__ __forceinline__ void lds_put(char* p, int i, T v) {
  __builtin_memcpy(__builtin_assume_aligned(p + i * sizeof(T), sizeof(T)), &v, sizeof(T));
}
// Between a lane's accesses there and those of others: the hardware has a wave's
// in their order, and the compiler is to keep it.
__device__ __forceinline__ void lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The two largest of a group's c, in all of its lanes: P = 2^lp lanes have a
// group, and share out its members in LDS. (NaNs are ignored.)
template <typename T>
__device__ __forceinline__ void group_best(const RouteArgs& a, const char* cs, int pos, int lp,
                                           T& b1, T& b2) {
  const int g = pos >> lp, p = pos & ((1 << lp) - 1);
  b1 = b2 = -INFINITY;
  if (g < a.groups) {
    for (int j = p; j < a.per; j += 1 << lp) {
      const T c = lds_get<T>(cs, g * a.per + j);
      b2 = fmax(b2, fmin(b1, c));
      b1 = fmax(b1, c);
    }
  }
  for (int o = 1; o < 1 << lp; o <<= 1) {
    const T o1 = __shfl_xor(b1, o), o2 = __shfl_xor(b2, o);
    b2 = fmax(fmin(b1, o1), fmax(b2, o2));
    b1 = fmax(b1, o1);
  }
}

// e / per, by a product that is exact for e < 2^10
__device__ __forceinline__ int group_of(const RouteArgs& a, int e) {
  return (int)(((float)e + 0.5f) * a.inv_per);
}
// whether the group of expert e is among those kept (a bit for each lane, the
// token's from seg on)
__device__ __forceinline__ bool kept(const RouteArgs& a, uint64_t keep, int seg, int lp, int e) {
  return (keep >> (seg + (group_of(a, e) << lp))) & 1;
}

// What a token needs in 64 bits where 32 cannot tell: small code, rolled over
// the row in LDS, since a wave that needs it fetches it first, and alone.

// c of the token's experts, lane, 64 + lane, .. of each lane of the wave, into
// cs; of groups, 2^lp lanes each, the lanes of those that are kept.
template <bool BIAS, bool GROUPED>
__device__ __forceinline__ uint64_t scores64(const RouteArgs& a, int64_t t, float m, char* cs,
                                             int lp) {
  const int lane = threadIdx.x & 63;
  double sum = 1.0;
  if (!a.sigmoid) {
    sum = 0.0;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {
      const float l = logit(a, t, e);
      if (m != -INFINITY || l != l) sum += exp((double)l - (double)m);
    }
    sum = wave_sum(sum);
  }
  uint64_t nan = 0;      // the groups of the lane's NaNs
  lds_order();
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const double l = logit(a, t, e);
    const double x = exp(a.sigmoid ? -l : l - (double)m);
    // (of a row without a logit above -infinity the scores are 0)
    double c = a.sigmoid ? 1.0 / (1.0 + x) : sum == 0.0 ? 0.0 : x / sum;
    if (BIAS) c += (double)a.bias[e];
    if (c != c) nan |= 1ull << group_of(a, e);
    lds_put(cs, e, c);
  }
  if (!GROUPED) return ~0ull;
  lds_order();
  double b1, b2;
  group_best<double>(a, cs, lane, lp, b1, b2);
  const int mine = lane >> lp;
#pragma unroll 1
  for (int o = 1; o < 64; o <<= 1) nan |= __shfl_xor(nan, o);
  // a group with a NaN is above the others
  const long long gk = order_key((nan >> mine) & 1 ? (double)NAN : a.best == 2 ? b1 + b2 : b1);
  int before = 0;
#pragma unroll 1
  for (int g = 0; g < a.groups; ++g) {
    const long long o = __shfl(gk, g << lp);
    before += o > gk || (o == gk && g < mine);
  }
  return __ballot(mine < a.groups && before < a.top_groups);
}

// The token's experts: lane r returns that of rank r.
template <bool BIAS, bool GROUPED>
__device__ __forceinline__ int choose64(const RouteArgs& a, int64_t t, float m, char* cs, int lp) {
  const int lane = threadIdx.x & 63;
  const uint64_t keep = scores64<BIAS, GROUPED>(a, t, m, cs, lp);
  lds_order();
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const double c = BIAS ? lds_get<double>(cs, e) : (double)logit(a, t, e);
    lds_put(cs, e, !GROUPED || kept(a, keep, 0, lp, e) ? order_key(c) : kNone64);
  }
  int id = 0;
#pragma unroll 1
  for (int r = 0; r < a.k; ++r) {
    long long bk = kNone64;
    int be = lane;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {
      const long long key = lds_get<long long>(cs, e);
      if (key > bk) {
        bk = key;
        be = e;
      }
    }
    // the largest upper halves, of these the lower halves, of these the expert
    const int hi = (int)(bk >> 32), top = wave_max(hi);
    const int lo = hi == top ? (int)((uint32_t)bk ^ 0x80000000u) : kNone, low = wave_max(lo);
    be = -wave_max(hi == top && lo == low ? -be : kNone);
    if (lane == (be & 63)) lds_put(cs, be, kNone64);
    if (lane == r) id = be;
  }
  return id;
}

// The same from comparisons in 32 bits; *sure: the result is that of 64 bits.
//
// With u = 2^-24: the hardware's exponential of x log2 e is off by (2 |x| + 3) u
// of itself. A sigmoid score is off by s (1 - s) (2 |l| + 3) u, at most 2 u, and
// a sum and a reciprocal: 4 u. Softmax scores are off by at most 60 u of the
// largest: (2 |x| + 3) e^x <= 4 for the exponential, x = l - m, u |x| more for
// the difference; their sum, whose average of |x| is at most log 1024 = 7, by
// (24 + 16 + 6) u; a reciprocal and a product. c is off by u |c| more. So two c
// whose difference is more than 2^-20 (2^-16 times the largest score) + 2^-23
// times their size are in the order of the exact ones, and two sums of two
// where it is more than twice that and 2^-22 times their size. Without a bias
// the experts' keys are the logits themselves, which are exact.
template <int N, int LPT, bool BIAS, bool GROUPED>
__device__ __forceinline__ int choose32(const RouteArgs& a, int64_t t, const float (&l)[N],
                                        float m, char* cs64, int* ids, bool* sure) {
  constexpr float kLog2e = 1.44269504f;
  const int lane = threadIdx.x & 63, seg = seg_of<LPT>(lane), pos = pos_of<LPT>(lane);
  const int e0 = pos * N;
  char* cs = cs64 + seg * N * sizeof(float);
  int key[N];
  bool clear = true;
  float room = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = e0 + i < a.E ? order_key(l[i]) : kNone;
  if (BIAS || GROUPED) {
    float c[N];
    if (a.sigmoid) {
      room = 0x1p-20f;
#pragma unroll
      for (int i = 0; i < N; ++i)
        c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * l[i]));
    } else {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        c[i] = __builtin_amdgcn_exp2f(kLog2e * (l[i] - m));    // (m = -infinity: NaN)
        sum += c[i];
      }
      const float inv = __builtin_amdgcn_rcpf(seg_sum<LPT>(sum));
#pragma unroll
      for (int i = 0; i < N; ++i) c[i] *= inv;
      room = 0x1p-16f * inv;
    }
    if (BIAS) {
      float b[N];
      load_run<N>(a.bias + e0, a.E - e0, 0.0f, b);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        c[i] += b[i];
        key[i] = e0 + i < a.E ? order_key(c[i]) : kNone;
      }
    }
    if (GROUPED) {
      bool nan = false;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        lds_put(cs, e0 + i, c[i]);
        nan |= c[i] != c[i];
      }
      lds_order();
      const int lp = a.lp[LPT == 64 ? 0 : LPT == 32 ? 1 : 2];
      float b1, b2;
      group_best<float>(a, cs, pos, lp, b1, b2);
      const float score = a.best == 2 ? b1 + b2 : b1;
      const int gk = order_key(score), mine = pos >> lp;
      int before = 0;
#pragma unroll 4
      for (int g = 0; g < a.groups; ++g) {
        const int o = LPT == 64 ? __builtin_amdgcn_readlane(gk, g << lp)
                                : __shfl(gk, seg + (g << lp));
        before += o > gk || (o == gk && g < mine);
      }
      const bool valid = mine < a.groups, stays = valid && before < a.top_groups;
      uint64_t keep = __ballot(stays);
      // the last that is kept and the first that is not
      const float low = -seg_max<LPT>(stays ? -score : -INFINITY);
      const float high = seg_max<LPT>(valid && !stays ? score : -INFINITY);
      clear = low - high > 2.0f * room + 0x1p-22f * (fabsf(low) + fabsf(high));
      clear = clear && seg_max<LPT>((int)nan) == 0;
      if constexpr (LPT == 64) {
        if (!clear) keep = scores64<BIAS, GROUPED>(a, t, m, cs64, lp);
        clear = true;
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!kept(a, keep, seg, lp, e0 + i)) key[i] = kNone;
    }
  }
  // The k largest, one after the other, and with a bias more until one is
  // clearly less than the last: lane r takes that of rank r (of several tokens a
  // wave by way of LDS). Of equal keys the lower index is first.
  constexpr bool SORT = N > 1 && N <= 8;      // the lane's own keys, descending
  uint32_t at = 0;                            // and whose they are, 3 bits each
  if constexpr (SORT) {
    int idx[N];
#pragma unroll
    for (int i = 0; i < N; ++i) idx[i] = i;
#pragma unroll
    for (int p = 0; p < N; ++p)
#pragma unroll
      for (int i = p & 1; i + 1 < N; i += 2) {
        const bool swap = key[i + 1] > key[i];
        const int k0 = key[i], i0 = idx[i];
        key[i] = swap ? key[i + 1] : k0;
        idx[i] = swap ? idx[i + 1] : i0;
        key[i + 1] = swap ? k0 : key[i + 1];
        idx[i + 1] = swap ? i0 : idx[i + 1];
      }
#pragma unroll
    for (int i = 0; i < N; ++i) at |= (uint32_t)idx[i] << (3 * i);
  }
  const auto drop = [&](bool mine, int j) {
    if constexpr (SORT) {
#pragma unroll
      for (int i = 0; i + 1 < N; ++i) key[i] = mine ? key[i + 1] : key[i];
      key[N - 1] = mine ? kNone : key[N - 1];
      at >>= mine ? 3 : 0;
    } else {
      const int d = mine ? j : -1;
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = d == i ? kNone : key[i];
    }
  };
  const auto place = [&](int best) {      // of the lane's largest
    if constexpr (SORT) return (int)(at & 7);
    int j = N - 1;
#pragma unroll
    for (int i = N - 2; i >= 0; --i) j = key[i] == best ? i : j;
    return j;
  };
  int id = 0, n = a.k;          // n: found that may be among the k
  bool ties = false, done = false;
  float last = INFINITY;
  int r = 0;
#pragma unroll 1
  for (;; ++r) {
    if (!BIAS && r == a.k) break;
    int bk = key[0];
    if constexpr (!SORT) {
#pragma unroll
      for (int i = 1; i < N; ++i) bk = max(bk, key[i]);
    }
    const int best = seg_max<LPT>(bk);
    if (BIAS) {
      const float v = key_value(best);
      const bool apart = r == 0 || last - v > room + 0x1p-23f * (fabsf(last) + fabsf(v));
      if (!done && r >= a.k && (apart || best == kNone)) {
        done = true;
        n = r;
      }
      ties |= !done && !apart;
      last = v;
      if (LPT == 64 ? done : __ballot(!done) == 0) break;
      if (r == LPT - 1) {      // no lane for more
        clear = clear && done;
        break;
      }
    }
    const uint64_t has = __ballot(bk == best);
    if constexpr (LPT == 64) {
      const int who = __ffsll((unsigned long long)has) - 1;
      const int j = __builtin_amdgcn_readlane(place(best), who);
      if (lane == r) id = who * N + j;
      drop(lane == who, j);
    } else {
      const bool mine = pos == __builtin_ctz((uint32_t)(has >> seg));
      const int j = place(best);
      if (mine) ids[seg + r] = e0 + j;
      drop(mine, j);
    }
  }
  if constexpr (LPT < 64) {
    lds_order();
    id = ids[lane];
  }
  if (BIAS) {
    if (pos >= n) id = 0;
    const bool resolve = ties && clear && a.sigmoid;
    if (ties && !a.sigmoid) clear = false;      // (the scores need the sum over the row)
    if (__ballot(resolve) != 0) {
      // The n found hold the k, but not for sure in their order: theirs in 64 bits.
      const double c = 1.0 / (1.0 + exp(-(double)value_of<N>(l, seg, id))) + (double)a.bias[id];
      const long long mine = order_key(c);
      int before = 0;
#pragma unroll 1
      for (int q = 0; q < r; ++q) {
        const long long o = __shfl(mine, seg + q);
        const int oi = __shfl(id, seg + q);
        before += q < n && (o > mine || (o == mine && oi < id));
      }
      const int to = resolve && pos < n ? before : pos;
      id = __builtin_amdgcn_ds_permute((seg + to) << 2, id);
    }
  }
  *sure = clear;
  return id;
}

template <int N, int LPT, bool BIAS, bool GROUPED>
__global__ __launch_bounds__(kWaves * 64) void route_kernel(RouteArgs a) {
  constexpr int TOKENS = 64 / LPT;
  __shared__ __align__(16) char cs[kWaves][BIAS || GROUPED ? N * 64 * sizeof(double) : 16];
  __shared__ int ids[kWaves][LPT < 64 ? 64 : 1];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int seg = seg_of<LPT>(lane), pos = pos_of<LPT>(lane), e0 = pos * N;
  const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * TOKENS;
  const int64_t T = a.t_dev ? min(a.T, (int64_t)*a.t_dev) : a.T;
  if (t0 >= T) return;
  const int64_t t = t0 + seg / LPT;
  const bool valid = t < T;      // (the lanes of tokens past the last go along)
  float l[N];
  load_logits<N>(a, t, e0, valid ? a.E - e0 : 0, l);
  const float m = a.sigmoid ? 0.0f : row_max<N, LPT>(l);
  bool sure;
  int id = choose32<N, LPT, BIAS, GROUPED>(a, t, l, m, cs[wave], ids[wave], &sure);
  if (BIAS || (GROUPED && LPT < 64)) {
    // the tokens of the wave one after the other, by all of it
    for (uint64_t left = __ballot(valid && !sure && pos == 0); left; left &= left - 1) {
      const int s = __ffsll((unsigned long long)left) - 1;
      const int one = choose64<BIAS, GROUPED>(a, t0 + s / LPT, lane_value(m, s), cs[wave], a.lp[0]);
      // (lane r has that of rank r: to the token's lanes)
      const int moved = __shfl(one, pos);
      if (seg == s) id = moved;
    }
  }
  // the weights, of the k experts alone where that is all they depend on
  const bool chosen = pos < a.k;
  double sr = 0.0, sum;
  const float v = value_of<N>(l, seg, id), lr = chosen ? v : -INFINITY;
  if (a.sigmoid) {
    sr = chosen ? 1.0 / (1.0 + exp(-(double)lr)) : 0.0;
    sum = a.normalize ? lanes_sum(sr, a.k) : 1.0;
  } else {
    // normalised: relative to the chosen ones' largest logit, since a bias may
    // choose experts whose scores are nothing beside the others'
    const float top = a.normalize ? seg_max<LPT>(lr) : m;
    const bool some = top == top && top != -INFINITY;
    sr = some && chosen ? exp((double)lr - (double)top) : 0.0;
    if (lr != lr) sr = lr;
    if (a.normalize) {
      sum = lanes_sum(sr, a.k);
    } else {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (e0 + i < a.E && (some || l[i] != l[i])) sum += exp((double)l[i] - (double)m);
      sum = seg_sum<LPT>(sum);
    }
  }
  if (chosen && valid) {
    a.ids[t * a.k + pos] = id;
    a.probs[t * a.k + pos] = sum == 0.0 ? 0.0f : (float)(sr / sum * (double)a.scale);
  }
}

// 1 / v of a normal v, to a step: the hardware's, and one of Newton's steps
__device__ __forceinline__ float reciprocal(float v) {
  const float r = __builtin_amdgcn_rcpf(v);
  return fmaf(fmaf(-v, r, 1.0f), r, r);
}

// The logits' gradient. With g_r = scale dp_r of the chosen experts,
//   scores' gradient: normalised ds_r = (g_r - sum_q g_q s_q / S) / S, S the
//   sum of the chosen s, else ds_r = g_r; 0 for the others
//   softmax: dl = s (ds - sum ds s), sigmoid: dl = ds s (1 - s).
// Normalised softmax weights are the softmax q over the chosen experts alone:
// dl_r = q_r (g_r - sum g q), nothing for the others; sigmoid ones, with q_r = s_r
// / S, have dl_r = q_r (1 - s_r) (g_r - sum g q).
template <int N>
__global__ __launch_bounds__(kWaves * 64) void route_grad_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63, wave = wave_id(), e0 = lane * N;
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= a.T || (a.t_dev && t >= *a.t_dev)) return;
  const bool all = !a.sigmoid && !a.normalize;
  float l[N];
  if (all) load_logits<N>(a, t, e0, a.E - e0, l);
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
  float total = 0.0f, dr;
  if (all) {
    const float m = row_max<N, 64>(l);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      l[i] = e0 + i < a.E && m != -INFINITY ? expf(l[i] - m) : 0.0f;
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
    // s and 1 - s are z = 1 / (1 + e) and e z with e = exp(-|l|), in one order or
    // the other
    const float e = expf(-fabsf(lr)), z = reciprocal(1.0f + e);
    if (a.normalize) {
      // q relative to the largest score: of logits far below -87 float32 has
      // neither s nor 1 / S (of logits below -709.78 the forward pass' 64 bits have
      // none either, and its weights are 0)
      const float m = wave_max(lr), h = fminf(m, 0.0f);
      float q = id >= 0 && m > -709.7827f ? (lr > 0.0f ? z : expf(lr - h) * z) : 0.0f;
      const float S = wave_sum(q);
      q *= S == 0.0f ? 0.0f : reciprocal(S);
      dr = q * (lr > 0.0f ? e * z : z) * (g - wave_sum(g * q));
    } else {
      dr = g * (e * (z * z));
      if (fabsf(lr) > 80.0f) {      // e below float32's normals, but g e need not be
        const float root = expf(-0.5f * fabsf(lr));
        dr = root * g * (root * (z * z));
      }
    }
  } else {
    const float m = wave_max(lr);
    const float ex = id >= 0 && m == m && m != -INFINITY ? expf(lr - m) : 0.0f;
    const float S = wave_sum(ex);
    const float q = S == 0.0f ? 0.0f : ex / S;
    dr = q * (g - wave_sum(g * q));
  }
  float d[N] = {};
  for (int r = 0; r < a.k; ++r) {
    const int e = __builtin_amdgcn_readlane(id, r) - e0;
    const float v = lane_value(dr, r);
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] += e == i ? v : 0.0f;
  }
  if (all) {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = l[i] * (d[i] - total);
  }
  if (a.dl_bf) store_run<N>((uint16_t*)a.dl + t * a.lddl + e0, a.E - e0, d);
  else store_run<N>((float*)a.dl + t * a.lddl + e0, a.E - e0, d);
}

// f launches, and returns that launch's status
template <typename F>
hipError_t by_experts(int E, F&& f) {
  if (E <= 64) return f(std::integral_constant<int, 1>{});
  if (E <= 128) return f(std::integral_constant<int, 2>{});
  if (E <= 256) return f(std::integral_constant<int, 4>{});
  if (E <= 512) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_route(const RouteArgs& in, hipStream_t s) {
  RouteArgs a = in;
  const bool grouped = a.top_groups < a.groups;
  int lg = 0;      // lanes a group, a power of two
  while ((1 << lg) < a.groups) ++lg;
  for (int i = 0; i < 3; ++i) a.lp[i] = grouped ? max(6 - i - lg, 0) : 6 - i;
  const auto go = [&](auto n, auto lpt) {
    constexpr int N = decltype(n)::value, LPT = decltype(lpt)::value;
    const int64_t each = kWaves * 64 / LPT;
    const unsigned grid = (unsigned)((a.T + each - 1) / each);
    if (a.bias && grouped) route_kernel<N, LPT, true, true><<<grid, kWaves * 64, 0, s>>>(a);
    else if (a.bias) route_kernel<N, LPT, true, false><<<grid, kWaves * 64, 0, s>>>(a);
    else if (grouped) route_kernel<N, LPT, false, true><<<grid, kWaves * 64, 0, s>>>(a);
    else route_kernel<N, LPT, false, false><<<grid, kWaves * 64, 0, s>>>(a);
    return hipGetLastError();
  };
  // Several tokens a wave where there are many and their experts few: they share
  // its instructions, and it takes longer (us, from graphs: 16384 tokens of 64
  // experts, top 6, 6.3, a wave a token 10.2, in groups 11.3, 22.2; 4096 4.3, 4.7;
  // 2048 in groups 6.9, 6.5; 8192 of 128 7.1, 8.0, in groups 12.5, 16.1; 2048 4.5,
  // 4.4; 8192 of 256 by two a wave 12.8, 10.7).
  if (a.E <= 64 && a.k < 16 && a.groups <= 16 && a.T >= 4096)
    return go(std::integral_constant<int, 4>{}, std::integral_constant<int, 16>{});
  if (a.E <= 128 && a.k < 32 && a.groups <= 32 && a.T >= 8192)
    return go(std::integral_constant<int, 4>{}, std::integral_constant<int, 32>{});
  return by_experts(a.E, [&](auto n) { return go(n, std::integral_constant<int, 64>{}); });
}
hipError_t launch_route_grad(const RouteArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((a.T + kWaves - 1) / kWaves);
  return by_experts(a.E, [&](auto n) {
    route_grad_kernel<decltype(n)::value><<<grid, kWaves * 64, 0, s>>>(a);
    return hipGetLastError();
  });
}

}  // namespace sffn
