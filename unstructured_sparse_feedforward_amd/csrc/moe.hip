// A whole mixture-of-experts layer for few tokens:
//
//   l = x W_r^T,  the k experts with the largest l of each token,
//   p = softmax of l over them (or over all experts),
//   y = sum_r p_r (ReLU(x W_g,e(r)) * (x W_u,e(r))) W_d,e(r)
//
// With few tokens the time is that of reading the selected experts'
// weights, so every weight is read once (per 16 or 32 of its expert's
// tokens). The launches:
//   logits  x W_r^T in 64 bits, a wave an expert and token;
//   route   top k and weights, a workgroup a token (for few experts together
//           with the logits; a single token's is part of the next kernel; in
//           place of both, take, where the caller has chosen the experts);
//   hidden  a workgroup has an expert and a slice of its neurons: it computes
//           z for all of the expert's tokens, and u only for the neurons that
//           are active (z > 0) for one of them, as in the rest of the library;
//   down    a workgroup has an expert and a chunk of y's columns, and reads
//           those of the active neurons' rows (in both, with few experts, for
//           a share of the expert's tokens, and here of its neurons);
//   sum     the token's k outputs, weighted, in the order of their ranks (no
//           float atomics: results repeat bit for bit). A launch of its own,
//           2.5 to 4 us: summing in the down kernel's last workgroup a token
//           takes a device-wide fence in all of them, which cost 10, or
//           stores that pass the L2 (one token the same 28.5 us, 256 tokens
//           of 4 over 32 4-bit experts 148 us in place of 135).
//
// Measured, launches included, all weights out of the caches: one token over
// 6 of 64 bf16 experts of 2048 x 1408, a sixth of the neurons active, 28 us
// (46 MB: 9.4 us at 4.9 TB/s; hidden 14, down 6.5, two small launches 6); 32
// tokens over 64 experts of that size in 4 bits 78 us (hidden 37, down 25);
// 64 tokens over 16 bf16 experts of 2048 x 5632, few active, 97 us (hidden 77
// us, 5.0 TB/s: bound by memory; routing 5, down 10, sum 4).
#include "moe.hpp"

namespace sffn {
namespace {

constexpr int NT = 256;
constexpr int kWaves = NT / 64;

// the wave's index, known to be the same in all its lanes
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

__device__ __forceinline__ int tokens(const MoeArgs& a) {
  return a.t_dev ? min(max(*a.t_dev, 0), a.T) : a.T;
}

// A logit as an integer of the same order (NaN above everything, the two
// zeros equal), so that ranks are unique whatever the values: ties and NaN
// go to the lowest expert.
__device__ __forceinline__ long long order_key(double l) {
  if (l != l) return 0x7FF8000000000000ll;
  const long long b = __double_as_longlong(l + 0.0);
  return b < 0 ? b ^ 0x7FFFFFFFFFFFFFFFll : b;
}
__device__ __forceinline__ double key_value(long long k) {
  return __longlong_as_double(k < 0 ? k ^ 0x7FFFFFFFFFFFFFFFll : k);
}

// ---------------------------------------------------------------- router

// The logits, a wave an expert and token, summed in 64 bits in an order that
// depends on d alone (a lane's columns ascending, then the lanes pairwise), so
// that a token's choice of experts is the same in every call. The product of
// two bf16 values has 16 bits: the sums are exact, and logits compare as their
// exact values do, where the products of a logit (zeros aside) lie within a
// factor of 2^37 / d of each other. Beyond that ties are those of the sums.
__device__ __forceinline__ double logit(const MoeArgs& a, int t, int e) {
  const int lane = threadIdx.x & 63;
  const uint16_t* x = a.x + (int64_t)t * a.d;
  const uint16_t* w = a.router + (int64_t)e * a.d;
  double s = 0.0;
#pragma unroll 4
  for (int c = lane * 8; c < a.d; c += 512) {
    float wv[8], xv[8];
    Vec<uint16_t, 8>::cvt(*(const u32x4_t*)(w + c), wv);
    Vec<uint16_t, 8>::cvt(*(const u32x4_t*)(x + c), xv);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fma((double)wv[j], (double)xv[j], s);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
  return s;
}
__global__ __launch_bounds__(NT) void moe_logits_kernel(MoeArgs a) {
  const int e = blockIdx.x * kWaves + wave_id();
  const int t = blockIdx.y;
  if (e >= a.E || t >= tokens(a)) return;
  const double s = logit(a, t, e);
  if ((threadIdx.x & 63) == 0) a.keys[(int64_t)t * a.E + e] = order_key(s);
}

// A token's k experts and their weights by rank (an expert's rank is the
// number of experts before it), from r.keys. Called by all N threads of a
// workgroup; begins and ends with a barrier.
struct Route {
  long long keys[kMoeMaxE];
  int before[kMoeMaxE];
  long long top;
  float wsum[16];
  int expert[kMoeMaxK];
  float p[kMoeMaxK];
};
template <int N>
__device__ __forceinline__ void route(const MoeArgs& a, Route& r) {
  const int tid = threadIdx.x;
  for (int e = tid; e < a.E; e += N) r.before[e] = 0;
  __syncthreads();
  // the comparisons shared out over all threads
  const int parts = max(N / a.E, 1);
  for (int i = tid; i < a.E * parts; i += N) {
    const int e = i % a.E;
    const long long mine = r.keys[e];
    int n = 0;
    for (int o = i / a.E; o < a.E; o += parts) {
      const long long other = r.keys[o];
      n += other > mine || (other == mine && o < e);
    }
    if (n) atomicAdd(&r.before[e], n);   // whole numbers: any order
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += N) {
    const int rank = r.before[e];
    if (rank == 0) r.top = r.keys[e];
    if (rank < a.k) r.expert[rank] = e;
  }
  __syncthreads();
  // exponentials below that of the largest logit; softmax over the k
  // experts or over all
  const double l0 = key_value(r.top);
  float sum = 0.0f;
  for (int i = tid; i < (a.normalize ? a.k : a.E); i += N) {
    const int e = a.normalize ? r.expert[i] : i;
    sum += expf((float)(key_value(r.keys[e]) - l0));
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
  if ((tid & 63) == 0) r.wsum[tid >> 6] = sum;
  __syncthreads();
  if (tid < a.k) {
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < N / 64; ++w) total += r.wsum[w];
    r.p[tid] = expf((float)(key_value(r.keys[r.expert[tid]]) - l0)) / total;
  }
  __syncthreads();
}

// A workgroup a token. LOGITS: it computes them itself, for as many experts
// as it has waves; with more, their 64-bit sums would keep the one CU busy
// (64 experts, d = 2048: 8.3 us, in a kernel of their own over all CUs 3.0
// and 3.5 here).
constexpr int kFusedE = 16;

template <bool LOGITS, int N>
__global__ __launch_bounds__(N) void moe_route_kernel(MoeArgs a) {
  __shared__ Route r;
  const int t = blockIdx.x, tid = threadIdx.x;
  if (t >= tokens(a)) return;
  if (LOGITS) {
    const int e = wave_id();
    if (e < a.E) {
      const double s = logit(a, t, e);
      if ((tid & 63) == 0) r.keys[e] = order_key(s);
    }
  } else {
    for (int e = tid; e < a.E; e += N) r.keys[e] = a.keys[(int64_t)t * a.E + e];
  }
  route<N>(a, r);
  if (tid < a.k) {
    const int i = t * a.k + tid;
    a.expert[i] = r.expert[tid];
    a.weight[i] = r.p[tid];
    if (a.ids) a.ids[i] = r.expert[tid];
    if (a.probs) a.probs[i] = r.p[tid];
  }
}

// Experts and weights given by the caller, a thread a (token, rank) pair: an
// index that is no expert's becomes -1, whose pair no later kernel computes or
// adds; of one that a token has twice the first pair takes both weights, so
// that an expert has a token once (its list of pairs has room for that).
__global__ __launch_bounds__(64) void moe_take_kernel(MoeArgs a) {
  const int i = blockIdx.x * 64 + threadIdx.x;
  const int t = i / a.k, r = i % a.k;
  if (t >= tokens(a)) return;
  const int32_t* ids = a.in_ids + (int64_t)t * a.k;
  const float* p = a.in_probs + (int64_t)t * a.k;
  const int e = ids[r];
  bool mine = e >= 0 && e < a.E;
  float w = 0.0f;
#pragma unroll 8
  for (int q = 0; q < a.k; ++q)
    if (ids[q] == e) {
      if (q < r) mine = false;
      else w += p[q];
    }
  a.expert[i] = mine ? e : -1;
  a.weight[i] = w;
}

// ---------------------------------------------------------------- weights

struct Rows {            // one of an expert's matrices
  const uint8_t* p;      // first row of the expert
  const uint8_t* sc;     // its scales (MXFP4)
  int64_t pitch;         // bytes a row
  int64_t gpitch;        // scale bytes a 128-column group (all experts' rows)
};

// 8 codes times their scale as bf16 pairs: exact (two significant bits). The
// conversion takes the scale's exponent byte as it is (255: NaN).
__device__ __forceinline__ u32x4_t from_codes(uint32_t q, uint32_t sb) {
  const float s = __uint_as_float(sb << 23);
  u32x4_t o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
  return o;
}

__device__ __forceinline__ f32x4_t mfma(const u32x4_t& w, const u32x4_t& v, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w),
                                                 __builtin_bit_cast(bf16x8_t, v), c, 0, 0, 0);
}

// ---------------------------------------------------------------- products with x

// acc[i][n] += rows 16 i .. of row() . x of 16 tokens (xo[n]: the offset of
// token l % 16 for lane l; XL: of token l / 16), over steps part, part +
// parts, .. of d: 64 columns of bf16, 128 of codes.
//
// The rows go through a ring of D slots in LDS of the wave's own (no barrier:
// the wave waits for its own oldest copies): a copy instruction covers whole
// 64- or 128-byte pieces of rows, while loads straight into the matrix
// instruction's lanes, in which neighbours hold different rows, take an access
// each; 64 experts of 2048 x 1408 in 4 bits then kept the address units busy
// for 25 of 27 us. A slot holds 16 rows (two blocks of codes one after the
// other), 16-byte piece c of row r at position c ^ (r / 2) % 8 of 8 (codes: c ^
// (r / 4) % 4 of 4), so that 16 lanes reading one piece of 16 rows meet
// different banks. The instruction's k order is free as long as both operands
// agree: lane l reads piece l / 16 of a row's four of 64 bytes, which are 32
// bf16 values, the instruction's own order, or 128 codes, four instructions'
// worth.
//
// XL (codes, up to kStaged tokens): x goes through the ring too. Loaded
// straight into the instruction's lanes it takes an access for every token
// and 16 bytes, four instructions a step; one copy brings a step's 256 bytes
// of four tokens, 16-byte piece c of token t at position c ^ t of 16. With 32
// tokens over 64 4-bit experts (three each) 77.7 us in place of 81.4. (bf16
// steps have half the x to load for twice the weights: even.)
template <bool MX>
constexpr int kRing = MX ? 3 : 5;      // slots: with four of codes registers spill
constexpr int kSlot = 2048;            // bytes: two copies of 64 lanes x 16
constexpr int kStaged = 4;
template <bool XL>
constexpr int kStep = kSlot + (XL ? 1024 : 0);
template <bool MX>
constexpr int kRingBytes = kRing<MX> * kStep<MX>;

template <bool MX, int MT, int NTK, bool XL, typename F>
__device__ __forceinline__ void dots(const MoeArgs& a, const Rows& w, F&& row,
                                     const uint32_t (&xo)[NTK], char* ring, int lane, int part,
                                     int parts, f32x4_t (&acc)[MT][NTK]) {
  static_assert(MT == (MX ? 2 : 1), "a slot holds two copies");
  static_assert(!XL || (MX && NTK == 1), "staged x is one copy of a step of codes");
  constexpr int D = kRing<MX>, NF = MX ? 4 : 2;    // MFMAs a step and block
  constexpr int SC = MX ? 128 : 64, SB = MX ? 64 : 128;   // columns and row bytes a step
  constexpr int OPS = 2 + (MX ? MT : 0) + (XL ? 1 : NTK * NF);  // loads a step
  const int kq = lane >> 4, l15 = lane & 15;
  // 32-bit offsets from an address that all lanes share
  uint32_t po[2], so[MT], xp[NTK];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = MX ? lane >> 2 : 8 * i + (lane >> 3);
    const int c = MX ? (lane & 3) ^ ((r >> 2) & 3) : (lane & 7) ^ ((r >> 1) & 7);
    po[i] = (uint32_t)row(MX ? 16 * i + r : r) * (uint32_t)w.pitch + c * 16;
  }
  if (MX) {
#pragma unroll
    for (int i = 0; i < MT; ++i) so[i] = (uint32_t)row(16 * i + l15) * 4 + kq;
  }
#pragma unroll
  for (int n = 0; n < NTK; ++n)
    xp[n] = xo[n] + (XL ? (l15 ^ kq) * 16 : kq * (MX ? 64 : 16));
  const uint8_t* xb = (const uint8_t*)a.x;
  u32x4_t xv[XL ? 1 : D][NTK][NF];
  uint32_t sb[D][MT];
  auto load = [&](auto ss, int i) {
    constexpr int s = decltype(ss)::value;
    const int64_t g = part + i * parts;
#pragma unroll
    for (int c = 0; c < 2; ++c) copy16(w.p + g * SB, po[c], ring + s * kStep<XL> + c * 1024);
    if constexpr (MX) {
#pragma unroll
      for (int m = 0; m < MT; ++m) sb[s][m] = *(w.sc + g * w.gpitch + so[m]);
    }
    if constexpr (XL) {
      copy16(xb + g * (SC * 2), xp[0], ring + s * kStep<XL> + kSlot);
    } else {
#pragma unroll
      for (int n = 0; n < NTK; ++n)
#pragma unroll
        for (int f = 0; f < NF; ++f)
          xv[s][n][f] = *(const u32x4_t*)(xb + g * (SC * 2) + f * (MX ? 16 : 64) + xp[n]);
    }
  };
  u32x4_t q[2];
  auto read = [&](auto ss) {
    const char* p = ring + decltype(ss)::value * kStep<XL>;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      q[c] = *(const u32x4_t*)(MX ? p + c * 1024 + l15 * 64 + ((kq ^ ((l15 >> 2) & 3)) << 4)
                                  : p + l15 * 128 + (((c * 4 + kq) ^ ((l15 >> 1) & 7)) << 4));
    if constexpr (XL) {
      const int t = l15 & (kStaged - 1);
#pragma unroll
      for (int f = 0; f < NF; ++f)
        xv[0][0][f] = *(const u32x4_t*)(p + kSlot + t * 256 + (((kq * 4 + f) ^ t) << 4));
    }
    wait_point<wait_imm(63, 0)>();     // read before the slot is written again
  };
  auto multiply = [&](auto ss) {
    constexpr int s = decltype(ss)::value;
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const u32x4_t wv = MX ? from_codes(q[m][f & 3], sb[s][m]) : q[f & 1];
#pragma unroll
        for (int n = 0; n < NTK; ++n) acc[m][n] = mfma(wv, xv[XL ? 0 : s][n][f], acc[m][n]);
      }
  };
  const int G = a.d / SC;
  const int n = G > part ? (G - part + parts - 1) / parts : 0;   // the wave's steps
  int i0 = 0;
  if (n >= 2 * D) {
    // D steps in flight: the oldest has landed when the loads of D - 1 are
    // left. (The first loads are not conditional here: the compiler's own
    // waits for x would otherwise drain every load in flight at the loop's
    // back edge.)
    unroll<D>([&](auto s) {
      load(s, decltype(s)::value);
      order_point();
    });
    for (; i0 + 2 * D <= n; i0 += D)
      unroll<D>([&](auto s) {
        wait_point<wait_imm((D - 1) * OPS, 15)>();
        read(s);
        multiply(s);
        load(s, i0 + decltype(s)::value + D);
      });
  } else {
    unroll<D>([&](auto s) {
      if (decltype(s)::value < n) load(s, decltype(s)::value);
      order_point();   // the waits count the loads step by step
    });
  }
  for (; i0 < n; i0 += D)
    unroll<D>([&](auto s) {
      const int i = i0 + decltype(s)::value;
      if (i >= n) return;
      if (i + D <= n) wait_point<wait_imm((D - 1) * OPS, 15)>();
      else wait_point<wait_imm(0, 15)>();
      read(s);
      multiply(s);
      if (i + D < n) load(s, i + D);
    });
}

// ---------------------------------------------------------------- hidden

// Rows of a product with x that a wave takes at a time, in blocks of 16:
// codes are a quarter of the bytes, and two blocks halve the loads of x.
template <bool MX>
constexpr int kBlocks = MX ? 2 : 1;
// most neurons of a workgroup: every wave one tile
template <bool MX>
constexpr int kSlice = kWaves * 16 * kBlocks<MX>;

// LDS of a pass of 16 NTK tokens
template <bool MX, int NTK>
struct Shared {
  static constexpr int MT = kBlocks<MX>, SL = kSlice<MX>;
  float z[16 * NTK][SL + 4];           // gate pre-activations (padded rows)
  int act[SL];                         // active neurons of the slice, ascending
  uint8_t on[SL];
  int na;
};

// The waves' rings. (Dynamic LDS: for reads of a static object the compiler
// waits for every copy into LDS in flight.) A wave's ring, when its copies
// have all landed, also holds its share of a product.
extern __shared__ __align__(16) char rings[];

// The products of tiles of 16 MT rows with the pass's tokens: the waves share
// out the tiles, and d where the tiles are fewer than the waves. row(i) is
// the row of position i. Leaves the shares in the rings, joined by share_sum.
template <bool MX, int NTK>
__device__ __forceinline__ f32x4_t& share_of(int wave, int i, int t, int lane) {
  return *(f32x4_t*)(rings + wave * kRingBytes<MX> + ((i * NTK + t) * 64 + lane) * 16);
}
template <bool MX, int NTK, bool XL, typename F>
__device__ __forceinline__ int share_products(const MoeArgs& a, const Rows& w,
                                              const uint32_t (&xo)[NTK], int tiles, F&& row) {
  constexpr int MT = kBlocks<MX>;
  const int lane = threadIdx.x & 63;
  const int wave = wave_id();
  const int lg = tiles <= 1 ? 0 : tiles <= 2 ? 1 : 2;
  const int parts = kWaves >> lg, tile = wave >> (2 - lg), part = wave & (parts - 1);
  if (tile < tiles) {
    f32x4_t acc[MT][NTK] = {};
    dots<MX, MT, NTK, XL>(a, w, [&](int i) { return row(tile * MT * 16 + i); }, xo,
                      rings + wave * kRingBytes<MX>, lane, part, parts, acc);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < NTK; ++t) share_of<MX, NTK>(wave, i, t, lane) = acc[i][t];
  }
  return parts;
}
template <bool MX, int NTK>
__device__ __forceinline__ f32x4_t share_sum(int parts, int block, int t, int l) {
  constexpr int MT = kBlocks<MX>;
  const int w0 = block / MT * parts;
  f32x4_t s = share_of<MX, NTK>(w0, block % MT, t, l);
  for (int p = 1; p < parts; ++p) s += share_of<MX, NTK>(w0 + p, block % MT, t, l);
  return s;
}

__device__ __forceinline__ uint64_t below(int lane) { return lane ? ~0ull >> (64 - lane) : 0ull; }

// A unit's (token, rank) pairs in ascending order; returns their number. A
// unit is an expert, or a pair, whose expert's pairs it has if it is the
// first of them (else none). *before: the pairs of the experts before it.
// Called by all NT threads.
struct Lists {
  int pair[kMoeMaxT];
  int wsum[kWaves];
  int wless[kWaves];
};
__device__ __forceinline__ int unit_pairs(const MoeArgs& a, int unit, Lists& ls, int* expert,
                                          int* before) {
  const int lane = threadIdx.x & 63;
  const int wave = wave_id();
  const int np = tokens(a) * a.k;
  const bool pairs = a.by_pair;
  if (pairs && unit >= np) return 0;
  const int e = pairs ? a.expert[unit] : unit;
  if (e < 0) return 0;
  *expert = e;
  int n = 0, less = 0;
  for (int i0 = 0; i0 < np; i0 += NT) {
    const int i = i0 + threadIdx.x;
    const int f = i < np ? a.expert[i] : a.E;
    const bool mine = f == e;
    const uint64_t b = __ballot(mine), l = __ballot(f < e);
    if (i0) __syncthreads();
    if (lane == 0) {
      ls.wsum[wave] = __popcll(b);
      ls.wless[wave] = __popcll(l);
    }
    __syncthreads();
    int at = n + __popcll(b & below(lane));
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) at += ls.wsum[w];
      n += ls.wsum[w];
      less += ls.wless[w];
    }
    if (mine) ls.pair[at] = i;
  }
  *before = less;
  __syncthreads();
  if (pairs && n > 0 && ls.pair[0] != unit) n = 0;
  return n;
}

// 16 NTK of the unit's tokens (list positions p0 ..) through the slice's
// neurons j0 .. j0 + nbe: their h, and in `any` the neurons active for one.
template <bool MX, bool GATED, int NTK, bool XL>
__device__ __forceinline__ void pass(const MoeArgs& a, Shared<MX, NTK>& sh, const Lists& ls,
                                     const Rows& wg, const Rows& wu, int j0, int nbe, int n,
                                     int p0, int place, bool more, uint8_t* any) {
  constexpr int MT = kBlocks<MX>;
  const int lane = threadIdx.x & 63;
  const int wave = wave_id();
  const int tid = threadIdx.x;
  const int nt = min(n - p0, 16 * NTK);   // tokens of this pass
  const int P = a.T * a.k;
  uint32_t xo[NTK];
#pragma unroll
  for (int i = 0; i < NTK; ++i) {
    const int tk = i * 16 + (XL ? lane >> 4 : lane & 15);
    xo[i] = (uint32_t)(ls.pair[p0 + min(tk, nt - 1)] / a.k) * (uint32_t)(a.d * 2);
  }

  if (tid < kSlice<MX>) sh.on[tid] = 0;
  const int blocks = nbe / 16;
  int parts = share_products<MX, NTK, XL>(a, wg, xo, (blocks + MT - 1) / MT,
                                      [&](int i) { return j0 + min(i, nbe - 1); });
  __syncthreads();
  for (int e = tid; e < blocks * NTK * 64; e += NT) {
    const int block = e / (NTK * 64), t = (e >> 6) % NTK, l = e & 63;
    const f32x4_t s = share_sum<MX, NTK>(parts, block, t, l);
    const int tk = t * 16 + (l & 15), j = block * 16 + 4 * (l >> 4);
    *(f32x4_t*)&sh.z[tk][j] = s;
    if (tk < nt) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (s[q] > 0.0f) sh.on[j + q] = any[j + q] = 1;   // every writer stores the same
      // non-gated: h is z itself; gated: a neuron that only another pass
      // of the workgroup finds active has h = 0 here
      if (!GATED || more) {
        float* o = a.h + (int64_t)(j0 + j) * P + place + p0 + tk;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q * P] = !GATED && s[q] > 0.0f ? s[q] : 0.0f;
      }
    }
  }
  __syncthreads();
  if (!GATED) return;
  // the neurons active for some token of the pass, ascending
  if (wave == 0) {
    int base = 0;
    for (int c = 0; c < nbe; c += 64) {
      const bool p = c + lane < nbe && sh.on[c + lane];
      const uint64_t b = __ballot(p);
      if (p) sh.act[base + __popcll(b & below(lane))] = c + lane;
      base += __popcll(b);
    }
    if (lane == 0) sh.na = base;
  }
  __syncthreads();
  const int na = sh.na;
  if (na == 0) return;
  parts = share_products<MX, NTK, XL>(a, wu, xo, (na + 16 * MT - 1) / (16 * MT),
                                  [&](int i) { return j0 + sh.act[min(i, na - 1)]; });
  __syncthreads();
  // h of the active neurons; the others' is not read
  for (int e = tid; e < (na + 15) / 16 * NTK * 64; e += NT) {
    const int block = e / (NTK * 64), t = (e >> 6) % NTK, l = e & 63;
    const f32x4_t u = share_sum<MX, NTK>(parts, block, t, l);
    const int tk = t * 16 + (l & 15);
    if (tk < nt) {
      float* o = a.h + (int64_t)j0 * P + place + p0 + tk;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = block * 16 + 4 * (l >> 4) + q;
        if (i < na) {
          const int j = sh.act[i];
          const float z = sh.z[tk][j];
          o[(int64_t)j * P] = z > 0.0f ? z * u[q] : 0.0f;
        }
      }
    }
  }
}

// The routing of a single token, for at most kOneE experts: lane l has the
// keys of experts l and 64 + l, each wave compares them with its share of the
// experts, and the shares are added. Returns the expert of rank `rank`, in
// *place the number of chosen experts of lower index; `give`: write the
// routing for the kernels to come. Called by all threads; holds a barrier.
// (Saves a launch: one token over 64 bf16 experts 28.4 us, routed in a kernel
// of its own 31.5; over 128 4-bit ones 24.7 and 29.3.)
constexpr int kOneE = 128;
__device__ __forceinline__ int route_one(const MoeArgs& a, int rank, bool give,
                                         int (&share)[kWaves][kOneE], int* place) {
  const int lane = threadIdx.x & 63;
  const int wave = wave_id();
  long long key[2];
  int before[2] = {};
  // (below every logit's key, infinities included)
#pragma unroll
  for (int i = 0; i < 2; ++i)
    key[i] = 64 * i + lane < a.E ? a.keys[64 * i + lane] : (long long)0x8000000000000000ull;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = min(a.E - 64 * i, 64);
    for (int o = wave; o < m; o += kWaves) {
      const uint32_t lo = __builtin_amdgcn_readlane((int)key[i], o);
      const uint32_t hi = __builtin_amdgcn_readlane((int)(key[i] >> 32), o);
      const long long other = (long long)((uint64_t)hi << 32 | lo);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        before[j] += other > key[j] || (other == key[j] && 64 * i + o < 64 * j + lane);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) share[wave][64 * j + lane] = before[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    before[j] = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) before[j] += share[w][64 * j + lane];
  }
  int e = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint64_t b = __ballot(before[j] == rank && 64 * j + lane < a.E);
    if (b) e = 64 * j + __ffsll((unsigned long long)b) - 1;
  }
  const uint64_t c0 = __ballot(before[0] < a.k && lane < a.E);
  const uint64_t c1 = __ballot(before[1] < a.k && 64 + lane < a.E);
  *place = __popcll(c0 & (e < 64 ? below(e) : ~0ull)) + __popcll(e < 64 ? 0ull : c1 & below(e - 64));
  if (give && wave == 0) {
    long long top = max(key[0], key[1]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = max(top, __shfl_xor(top, o));
    const double l0 = key_value(top);
    float ex[2], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool counts = 64 * j + lane < a.E && (before[j] < a.k || !a.normalize);
      ex[j] = counts ? expf((float)(key_value(key[j]) - l0)) : 0.0f;
      sum += ex[j];
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (64 * j + lane < a.E && before[j] < a.k) {
        a.expert[before[j]] = 64 * j + lane;
        a.weight[before[j]] = ex[j] / sum;
        if (a.ids) a.ids[before[j]] = 64 * j + lane;
        if (a.probs) a.probs[before[j]] = ex[j] / sum;
      }
  }
  return __builtin_amdgcn_readfirstlane(e);
}

// ONE: a single token, whose routing every workgroup finds for itself.
template <bool MX, bool GATED, bool ONE, int NTK>
__global__ __launch_bounds__(NT, NTK == 1 ? 4 : 2) void moe_hidden_kernel(MoeArgs a) {
  __shared__ Lists ls;
  __shared__ uint8_t any[kSlice<MX>];
  __shared__ union {
    int share[kWaves][kOneE];
    Shared<MX, 1> s1;
    Shared<MX, NTK> s;
  } sh;
  const int tid = threadIdx.x;
  const int slice = blockIdx.x, unit = blockIdx.y, z = blockIdx.z;
  int e, n = 1, place;
  if (tid < kSlice<MX>) any[tid] = 0;
  if (ONE) {
    if (tokens(a) == 0) return;
    e = route_one(a, unit, slice == 0 && unit == 0, sh.share, &place);
    if (tid == 0) ls.pair[0] = unit;
    __syncthreads();
  } else {
    n = unit_pairs(a, unit, ls, &e, &place);
    if (n <= 16 * NTK * z) return;
  }

  const int j0 = slice * a.nb;
  const int nbe = min(a.nb, a.F - j0);
  const int64_t pitch = MX ? a.d / 2 : (int64_t)a.d * 2;
  const int64_t row0 = (int64_t)e * a.F;
  const int64_t gp = (int64_t)a.E * a.F * 4;
  const Rows wg = {(const uint8_t*)a.wg + row0 * pitch, MX ? a.sg + row0 * 4 : nullptr, pitch, gp};
  const Rows wu = {GATED ? (const uint8_t*)a.wu + row0 * pitch : nullptr,
                   MX && GATED ? a.su + row0 * 4 : nullptr, pitch, gp};
  const bool more = n > 16 * NTK * a.zh;
  for (int p0 = 16 * NTK * z; p0 < n; p0 += 16 * NTK * a.zh) {
    if (MX && n - p0 <= kStaged)
      pass<MX, GATED, 1, MX>(a, sh.s1, ls, wg, wu, j0, nbe, n, p0, place, more, any);
    else if (n - p0 <= 16)
      pass<MX, GATED, 1, false>(a, sh.s1, ls, wg, wu, j0, nbe, n, p0, place, more, any);
    else
      pass<MX, GATED, NTK, false>(a, sh.s, ls, wg, wu, j0, nbe, n, p0, place, more, any);
    __syncthreads();
  }
  if (tid < nbe) a.on[((int64_t)z * a.Y + unit) * a.F + j0 + tid] = any[tid];
}

// ---------------------------------------------------------------- down

constexpr int kFl = 4;           // times 8 flags a thread
constexpr int kSeg = kFl * 8 * NT;   // neurons whose active ones are listed at a time (8192)

// A lane loads CPL columns of 8 neurons (16 bytes of bf16, 8 of codes) and
// turns them into CPL operands, one a column: operand q of lane l holds
// column CPL (l % 16) + q at k = neurons 8 (l / 16) .. + 7, and the results
// of a lane are 4 CPL consecutive columns of token l % 16. (A chunk is 256
// bytes of a bf16 row, 128 of codes: the rows are scattered, and shorter
// pieces cost more accesses for the same bytes. 32 tokens over 64 4-bit
// experts: 80 us, 8 columns a lane and twice the workgroups 86.)
template <bool MX>
constexpr int kCpl = MX ? 16 : 8;

// (Registers for two workgroups a CU: with three, bf16 spills; 32 tokens of 6
// over 64 experts of 2048 x 1408, half the neurons active, 200 us, 205.)
template <bool MX>
__global__ __launch_bounds__(NT, 2) void moe_down_kernel(MoeArgs a) {
  constexpr int CPL = kCpl<MX>, COLS = 16 * CPL;
  __shared__ uint16_t act[kSeg];
  __shared__ int wsum[kWaves];
  __shared__ f32x4_t red[kWaves / 2][CPL][64];
  __shared__ Lists ls;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = wave_id();
  const int kq = lane >> 4, l15 = lane & 15;
  const int chunk = blockIdx.x, unit = blockIdx.y;
  // the workgroup's blocks of 16 tokens, p_first and every 16 zd from there
  // on, and its range of neurons
  const int p_first = ((int)blockIdx.z & (a.zd - 1)) * 16;
  const int range = (int)blockIdx.z >> (31 - __builtin_clz(a.zd));
  const int f_begin = range * a.fs, f_end = min(a.F, f_begin + a.fs);
  // the flags of the neurons active for the tokens at p0, from s0 on, 8 x kFl
  // a thread (F and fs are multiples of 32)
  uint64_t fl[kFl];
  auto flags = [&](int p0, int s0) {
    const int z = (p0 >> (a.ntk + 3)) & (a.zh - 1);   // ntk is 1 or 2
    const uint8_t* on = a.on + ((int64_t)z * a.Y + unit) * a.F;
    const int f0 = s0 + tid * (8 * kFl);
#pragma unroll
    for (int v = 0; v < kFl; ++v) fl[v] = f0 < f_end ? *(const uint64_t*)(on + f0 + 8 * v) : 0;
  };
  flags(p_first, f_begin);   // (a unit without tokens has none that mean anything)
  int e, place;
  const int n = unit_pairs(a, unit, ls, &e, &place);
  if (n <= p_first) return;
  const int ncol = min(COLS, a.d - chunk * COLS);   // (the last chunk of codes may be half)
  const int col = chunk * COLS + min(CPL * l15, ncol - CPL);
  const int64_t pitch = MX ? a.d / 2 : (int64_t)a.d * 2;
  const int64_t gp = (int64_t)a.E * a.F * 4;
  // a row's place as a 32-bit offset from an address that all lanes share
  const uint8_t* wp = (const uint8_t*)a.wd + (int64_t)e * a.F * pitch;
  const uint32_t cb = MX ? col / 2 : col * 2, rp = (uint32_t)pitch;
  // (its scales: one or two 128-column groups)
  const uint8_t* sp = MX ? a.sd + (int64_t)e * a.F * 4 + (col >> 7) * gp + ((col >> 5) & 3) : nullptr;

  for (int p0 = p_first; p0 < n; p0 += 16 * a.zd) {
    const int nt = min(n - p0, 16);
    f32x4_t acc[CPL] = {};
    for (int s0 = f_begin; s0 < f_end; s0 += kSeg) {
      // list the segment's active neurons
      if (s0 > f_begin || p0 > p_first) flags(p0, s0);
      const int f0 = s0 + tid * (8 * kFl);
      int mine = 0;
#pragma unroll
      for (int v = 0; v < kFl; ++v) mine += __popcll(fl[v]);
      int pre = mine;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(pre, o);
        if (lane >= o) pre += v;
      }
      __syncthreads();                 // the last segment's list is done with
      if (lane == 63) wsum[wave] = pre;
      __syncthreads();
      int at = pre - mine, na = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (w < wave) at += wsum[w];
        na += wsum[w];
      }
#pragma unroll
      for (int v = 0; v < kFl; ++v) {
        if (!fl[v]) continue;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if ((fl[v] >> (8 * q)) & 1) act[at++] = (uint16_t)(f0 + 8 * v + q);
      }
      __syncthreads();
      // 32 neurons a step, the steps shared out over the waves, the next
      // step's loads in flight
      const uint32_t ho = (uint32_t)(place + p0 + min(l15, nt - 1)) * 4;
      const uint32_t hp4 = (uint32_t)(a.T * a.k) * 4;
      u32x2_t q[2][8];
      uint32_t sb[2][8];
      u32x4_t raw[2][8];
      float hv[2][8];
      auto load = [&](auto bb, int ks) {
        constexpr int b = decltype(bb)::value;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t r = act[min(ks + kq * 8 + j, na - 1)];
          if constexpr (MX) {
            q[b][j] = *(const u32x2_t*)(wp + (r * rp + cb));
            sb[b][j] = sp[r * 4];
          } else {
            raw[b][j] = *(const u32x4_t*)(wp + (r * rp + cb));
          }
          hv[b][j] = *(const float*)((const uint8_t*)a.h + (r * hp4 + ho));
        }
      };
      auto step = [&](auto bb, int ks) {
        constexpr int b = decltype(bb)::value;
        u32x4_t v[8][CPL / 8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < CPL / 8; ++i) {
            if constexpr (MX) v[j][i] = from_codes(q[b][j][i], sb[b][j]);
            else v[j][i] = raw[b][j];
          }
        // h in three bf16 parts, whose sum has the 24 bits of a float32: the
        // matrix instructions take bf16, and one rounding of h to it would
        // be the layer's largest error by far
        u32x4_t hp[3];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float x = ks + kq * 8 + j < na ? hv[b][j] : 0.0f;
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            const __bf16 xb = (__bf16)x;
            const uint32_t bits = __builtin_bit_cast(uint16_t, xb);
            hp[p][j / 2] = j & 1 ? hp[p][j / 2] | bits << 16 : bits;
            // an infinite or NaN h is all in its first part
            x = fabsf((float)xb) < INFINITY ? x - (float)xb : 0.0f;
          }
        }
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          // low (c even) or high halves of neurons 2 i and 2 i + 1
          const uint32_t sel = (c & 1) ? 0x07060302u : 0x05040100u;
          u32x4_t o;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = __builtin_amdgcn_perm(v[2 * i + 1][c / 8][(c % 8) >> 1],
                                         v[2 * i][c / 8][(c % 8) >> 1], sel);
#pragma unroll
          for (int p = 2; p >= 0; --p) acc[c] = mfma(o, hp[p], acc[c]);
        }
      };
      constexpr int S = kWaves * 32;
      if (wave * 32 < na) load(Int<0>{}, wave * 32);
      for (int ks = wave * 32; ks < na; ks += 2 * S) {
        if (ks + S < na) load(Int<1>{}, ks + S);
        step(Int<0>{}, ks);
        if (ks + S < na) {
          if (ks + 2 * S < na) load(Int<0>{}, ks + 2 * S);
          step(Int<1>{}, ks + S);
        }
      }
    }
    // the waves' sums: the upper half's through LDS into the lower half's,
    // theirs through LDS into the result
#pragma unroll
    for (int half = 1; half >= 0; --half) {
      if (wave / (kWaves / 2) == half) {
#pragma unroll
        for (int q = 0; q < CPL; ++q) {
          f32x4_t& m = red[wave % (kWaves / 2)][q][lane];
          m = half ? acc[q] : acc[q] + m;
        }
      }
      __syncthreads();
    }
    for (int i = tid; i < CPL * 64; i += NT) {
      const int l = i & 63, q0 = (i >> 6) / 4 * 4, r = (i >> 6) % 4;
      // row r of operands q0 .. q0 + 3: four consecutive columns
      const int tk = l & 15, c = 4 * CPL * (l >> 4) + CPL * r + q0;
      f32x4_t s;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        s[q] = red[0][q0 + q][l][r];
#pragma unroll
        for (int w = 1; w < kWaves / 2; ++w) s[q] += red[w][q0 + q][l][r];
      }
      if (tk < nt && c < ncol)
        *(f32x4_t*)(a.part + ((int64_t)range * a.T * a.k + ls.pair[p0 + tk]) * a.d +
                    chunk * COLS + c) = s;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- sum

// y of a token: a wave 256 columns, the k outputs in the order of their ranks
// (GIVEN: those of its pairs that have an expert)
template <bool GIVEN>
__global__ __launch_bounds__(64) void moe_sum_kernel(MoeArgs a) {
  const int t = blockIdx.y, lane = threadIdx.x;
  if (t >= tokens(a)) return;
  const int c = blockIdx.x * 256 + lane * 4;
  if (c >= a.d) return;
  const float* p = a.weight + (int64_t)t * a.k;
  const float* q = a.part + (int64_t)t * a.k * a.d + c;
  f32x4_t s = {};
#pragma unroll 8
  for (int r = 0; r < a.k; ++r) {
    if (GIVEN && a.expert[(int64_t)t * a.k + r] < 0) continue;
    f32x4_t v = *(const f32x4_t*)(q + (int64_t)r * a.d);
    for (int i = 1; i < a.split; ++i)
      v += *(const f32x4_t*)(q + ((int64_t)i * a.T * a.k + r) * a.d);
    s += v * p[r];
  }
  *(f32x4_t*)(a.y + (int64_t)t * a.d + c) = s;
}

template <bool MX, bool GATED>
hipError_t launch_hidden(const MoeArgs& a, hipStream_t s) {
  const dim3 grid((a.F + a.nb - 1) / a.nb, a.Y, a.zh);
  constexpr size_t lds = kWaves * kRingBytes<MX>;
  if (a.one) moe_hidden_kernel<MX, GATED, true, 1><<<grid, NT, lds, s>>>(a);
  else if (a.ntk == 1) moe_hidden_kernel<MX, GATED, false, 1><<<grid, NT, lds, s>>>(a);
  else moe_hidden_kernel<MX, GATED, false, 2><<<grid, NT, lds, s>>>(a);
  return hipGetLastError();
}

}  // namespace

void moe_plan(bool mx, MoeArgs* a) {
  const int pairs = a->T * a->k;
  a->one = a->T == 1 && a->E <= kOneE && !a->in_ids;
  // Units of the fewer of pairs and experts: of 6 of 64 bf16 experts of 2048 x
  // 1408, 2, 4 and 8 tokens take 41.2, 53.1 and 75.7 us, with a unit for every
  // expert 43.5, 56.8 and 78.7; of 8 of 128 4-bit ones of 2048 x 768, 2, 8 and 15
  // tokens 31.5, 43.0 and 60.5, and 36.2, 46.3 and 61.8.
  a->by_pair = pairs < a->E || a->one;
  a->Y = a->by_pair ? pairs : a->E;
  const int least = mx ? 32 : 16;
  int nb = mx ? kSlice<true> : kSlice<false>;
  // Neurons a workgroup: the most (64 of bf16, 128 of codes) where that leaves
  // eight workgroups a CU, with codes, a quarter of the bytes, four (bf16: 64
  // tokens over 16 experts of 5632 neurons 142 us, by four a CU 146; codes: 32
  // tokens over 64 experts 81, by eight 86.8). Else half as many, and a quarter
  // only where half leaves less than two workgroups a CU, so that x and the
  // start of the rings are paid for less often (4 tokens of 6 over 64 experts:
  // bf16 32 neurons 53.1, 16 58.6, 64 55.5; codes 64 neurons 39.6, 32 43.0; one
  // token to 8 of 32 experts of 2816 neurons: 32 neurons 41.1, 16 46.5; to 4 of
  // 16, d = 4096: 16 43.2, 32 46.5). Several tokens' long rows keep the first
  // border for the quarter as well (16 tokens of 2 over 16 bf16 experts of 2816
  // neurons: d = 4096 124 us, by the second border 130; d = 2560 89.5, 84.7; 40 of
  // 4 over 28 4-bit ones of 1440, d = 3584: 81.7, 84.6).
  const int longest = nb, most = mx ? 1024 : 2048;
  const int fewest = a->d >= 3584 && !a->one ? most : 512;
  while (nb > least &&
         (int64_t)a->Y * ((a->F + nb - 1) / nb) < (nb == longest ? most : fewest))
    nb /= 2;
  a->nb = nb;
  // Two blocks of 16 tokens a pass where the experts have more than that: a
  // mean of 12 tokens costs the same either way (96 tokens of 8 over 64 bf16
  // experts of 2048 x 1408: 254, 252 us), 8 tokens 206 and 211, 16 tokens 319
  // and 301.
  a->ntk = pairs <= 12 * a->E ? 1 : 2;
  const int cols = 16 * (mx ? kCpl<true> : kCpl<false>);
  a->chunks = (a->d + cols - 1) / cols;
  // Where workgroups are few, an expert's blocks of tokens go to several, and
  // in the down kernel ranges of at least 1024 neurons do (their outputs are
  // added in the sum kernel): 128 tokens to one bf16 expert of 2048 x 5632 86
  // us, without 374; one token to 2 of 8 28.8, without 31.7. Ranges up to
  // 256 workgroups (64 tokens over 16 experts of 5632 neurons: 99.1 us, up to
  // 512 99.9), with several blocks of tokens 512 (128 tokens of 2 over 4
  // experts of 2816: 107.8, up to 256 112.7).
  int blocks = 1;      // of 16 tokens, the mean of an expert, up to a power of two
  while (!a->by_pair && 16 * blocks * a->E < pairs) blocks *= 2;
  a->zh = a->Y * ((a->F + nb - 1) / nb) < 1024 ? (blocks + a->ntk - 1) / a->ntk : 1;
  a->zd = a->chunks * a->Y < 512 ? blocks : 1;
  a->split = 1;
  while (a->chunks * a->Y * a->zd * a->split < (blocks > 1 ? 512 : 256) &&
         a->F / (2 * a->split) >= 1024)
    a->split *= 2;
  a->fs = ((a->F + a->split - 1) / a->split + 31) / 32 * 32;
}

hipError_t launch_moe(bool mx, const MoeArgs& a, hipStream_t s) {
  if (a.in_ids) {
    moe_take_kernel<<<(a.T * a.k + 63) / 64, 64, 0, s>>>(a);
  } else if (!a.one && a.E <= kFusedE) {
    moe_route_kernel<true, kFusedE * 64><<<a.T, kFusedE * 64, 0, s>>>(a);
  } else {
    moe_logits_kernel<<<dim3((a.E + kWaves - 1) / kWaves, a.T), NT, 0, s>>>(a);
    if (!a.one) moe_route_kernel<false, NT><<<a.T, NT, 0, s>>>(a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool gated = a.wu != nullptr;
  e = mx ? (gated ? launch_hidden<true, true>(a, s) : launch_hidden<true, false>(a, s))
         : (gated ? launch_hidden<false, true>(a, s) : launch_hidden<false, false>(a, s));
  if (e != hipSuccess) return e;
  const dim3 grid(a.chunks, a.Y, a.zd * a.split);
  if (mx) moe_down_kernel<true><<<grid, NT, 0, s>>>(a);
  else moe_down_kernel<false><<<grid, NT, 0, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 sum((a.d + 255) / 256, a.T);
  if (a.in_ids) moe_sum_kernel<true><<<sum, 64, 0, s>>>(a);
  else moe_sum_kernel<false><<<sum, 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace sffn
