// A whole mixture-of-experts layer for few tokens:
//
//   l = x W_r^T,  the k experts with the largest l of each token,
//   p = softmax of l over them (or over all experts),
//   y = sum_r p_r (ReLU(x W_g,e(r)) * (x W_u,e(r))) W_d,e(r)
//
// With few tokens the time is that of reading the selected experts'
// weights, so every weight is read once, by one workgroup: a workgroup has
// an expert and a slice of its neurons, and computes those neurons' gate,
// up and down products for all of the expert's tokens. The layout is the
// layer's (row j of each matrix belongs to neuron j), so the three products
// of a slice read three runs of rows. Gate comes first; up and down are
// read only for neurons that are active (z > 0) for one of the tokens, as
// in the rest of the library.
//
// Three launches: the logits; the experts, which leave each (token, rank)'s
// partial output of each slice; the weighted sum over ranks and slices, in
// a fixed order (no atomics: results repeat bit for bit).
#include "moe.hpp"

namespace sffn {
namespace {

constexpr int NT = 256;
constexpr int kWaves = NT / 64;

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

// ---------------------------------------------------------------- logits

// One wave an expert and kLogitT tokens. The sums are 64-bit: two experts'
// logits then compare as their exact values do (the product of two bf16
// values has 16 bits), whatever the order of summation.
constexpr int kLogitT = 4;

__global__ __launch_bounds__(NT) void moe_logits_kernel(MoeArgs a) {
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int T = tokens(a);
  const int t0 = blockIdx.y * kLogitT;
  if (e >= a.E || t0 >= T) return;
  const uint16_t* w = a.router + (int64_t)e * a.d;
  double s[kLogitT] = {};
#pragma unroll 2
  for (int c = lane * 8; c < a.d; c += 512) {
    float wv[8];
    Vec<uint16_t, 8>::cvt(*(const u32x4_t*)(w + c), wv);
#pragma unroll
    for (int i = 0; i < kLogitT; ++i) {
      float xv[8];
      const int t = min(t0 + i, T - 1);
      Vec<uint16_t, 8>::cvt(*(const u32x4_t*)(a.x + (int64_t)t * a.d + c), xv);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i] = fma((double)wv[j], (double)xv[j], s[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kLogitT; ++i) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) s[i] += __shfl_xor(s[i], o);
    if (lane == 0 && t0 + i < T) a.keys[(int64_t)(t0 + i) * a.E + e] = order_key(s[i]);
  }
}

// ---------------------------------------------------------------- weights

struct Rows {            // one of an expert's matrices
  const uint8_t* p;      // first row of the expert
  const uint8_t* sc;     // its scales (MXFP4)
  int64_t pitch;         // bytes a row
  int64_t gpitch;        // scale bytes a 128-column group (all experts' rows)
};

// the scale 2^(b - 127) of a scale byte
__device__ __forceinline__ float scale_of(uint32_t b) {
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}

// 8 elements of a row as bf16 pairs: bf16 values as they are, or 8 codes
// times their scale (exact: two significant bits).
__device__ __forceinline__ u32x4_t from_codes(uint32_t q, uint32_t sb) {
  const float s = scale_of(sb);
  u32x4_t o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
  if (__builtin_expect(sb == 255u, 0)) o = u32x4_t{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
  return o;
}

__device__ __forceinline__ f32x4_t mfma(const u32x4_t& w, const u32x4_t& v, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w),
                                                 __builtin_bit_cast(bf16x8_t, v), c, 0, 0, 0);
}

// ---------------------------------------------------------------- products with x

// acc[i][n] += rows r[i] (16 of them, one a lane's row) . x of 16 tokens,
// over this wave's share of d. The instruction's k order is free as long as
// both operands agree: lane l takes 32 (bf16) or 16 (codes) contiguous bytes
// of row l % 16, so that the four lanes of a row cover 128 or 64 bytes.
template <bool MX, int MT, int NTK>
__device__ __forceinline__ void dots(const MoeArgs& a, const Rows& w, const int (&r)[MT],
                                     const uint16_t* const (&xt)[NTK], int lane, int wave,
                                     f32x4_t (&acc)[MT][NTK]) {
  const int kq = lane >> 4;
  if constexpr (MX) {
    const uint8_t* p[MT];
    const uint8_t* ps[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      p[i] = w.p + (int64_t)r[i] * w.pitch + kq * 16;
      ps[i] = w.sc + (int64_t)r[i] * 4 + kq;
    }
    const int G = a.d / 128;
#pragma unroll 2
    for (int g = wave; g < G; g += kWaves) {
      u32x4_t q[MT];
      uint32_t sb[MT];
      u32x4_t xv[NTK][4];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        q[i] = *(const u32x4_t*)(p[i] + (int64_t)g * 64);
        sb[i] = ps[i][g * w.gpitch];
      }
#pragma unroll
      for (int n = 0; n < NTK; ++n)
#pragma unroll
        for (int f = 0; f < 4; ++f)
          xv[n][f] = *(const u32x4_t*)(xt[n] + g * 128 + kq * 32 + f * 8);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const u32x4_t wv = from_codes(q[i][f], sb[i]);
#pragma unroll
          for (int n = 0; n < NTK; ++n) acc[i][n] = mfma(wv, xv[n][f], acc[i][n]);
        }
    }
  } else {
    const uint8_t* p[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) p[i] = w.p + (int64_t)r[i] * w.pitch + kq * 32;
    const int G = a.d / 64;
#pragma unroll 4
    for (int g = wave; g < G; g += kWaves) {
      u32x4_t wv[MT][2], xv[NTK][2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
#pragma unroll
        for (int i = 0; i < MT; ++i) wv[i][f] = *(const u32x4_t*)(p[i] + (int64_t)g * 128 + f * 16);
#pragma unroll
        for (int n = 0; n < NTK; ++n)
          xv[n][f] = *(const u32x4_t*)(xt[n] + g * 64 + kq * 16 + f * 8);
      }
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int n = 0; n < NTK; ++n) acc[i][n] = mfma(wv[i][f], xv[n][f], acc[i][n]);
    }
  }
}

// ---------------------------------------------------------------- experts

// LDS of a workgroup for passes of 16 NTK tokens.
template <int NTK>
struct Shared {
  static constexpr int kTok = 16 * NTK;
  static constexpr int kZ = kMoeSlice + 4;    // padded rows: no bank conflicts
  static constexpr int kH = kMoeSlice + 8;
  f32x4_t red[kWaves][2][NTK][64];     // the waves' shares of a 32-neuron product
  float z[kTok][kZ];                   // gate pre-activations of the pass
  __align__(16) uint16_t hi[kTok][kH]; // h of the active neurons, bf16 high ...
  __align__(16) uint16_t lo[kTok][kH]; // ... and low parts
  int act[kMoeSlice];                  // active neurons of the slice, ascending
  uint8_t on[kMoeSlice];
  int na;
};

struct Lists {
  int tok[kMoeMaxT];                   // the expert's tokens, ascending
  int pair[kMoeMaxT];                  // token * k + rank
  int rank[kMoeMaxT];                  // of each token (k: not selected)
  int wsum[kWaves];
};

// 16 NTK of the expert's tokens (list positions p0 ..) through the slice's
// neurons j0 .. j0 + nbe.
template <bool MX, bool GATED, int NTK>
__device__ __forceinline__ void pass(const MoeArgs& a, Shared<NTK>& sh, const Lists& ls,
                                     const Rows& wg, const Rows& wu, const Rows& wd, int j0,
                                     int nbe, int n, int p0, int slice) {
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int tid = threadIdx.x;
  const int nt = min(n - p0, 16 * NTK);   // tokens of this pass
  const uint16_t* xt[NTK];
#pragma unroll
  for (int i = 0; i < NTK; ++i)
    xt[i] = a.x + (int64_t)ls.tok[p0 + min(i * 16 + (lane & 15), nt - 1)] * a.d;

  if (tid < kMoeSlice) sh.on[tid] = 0;
  // gate: 32 neurons at a time, the waves' shares of d joined in LDS
  for (int c = 0; c < nbe; c += 32) {
    f32x4_t acc[2][NTK] = {};
    const int r[2] = {j0 + c + (lane & 15), j0 + c + 16 + (lane & 15)};
    dots<MX, 2, NTK>(a, wg, r, xt, lane, wave, acc);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < NTK; ++t) sh.red[wave][i][t][lane] = acc[i][t];
    __syncthreads();
    for (int e = tid; e < 2 * NTK * 64; e += NT) {
      const int i = e / (NTK * 64), t = (e >> 6) % NTK, l = e & 63;
      f32x4_t s = sh.red[0][i][t][l];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += sh.red[w][i][t][l];
      const int tk = t * 16 + (l & 15), j = c + i * 16 + 4 * (l >> 4);
      *(f32x4_t*)&sh.z[tk][j] = s;
      if (tk < nt) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (s[q] > 0.0f) sh.on[j + q] = 1;   // every writer stores the same
      }
    }
  }
  __syncthreads();
  // the neurons active for some token of the pass, ascending
  if (wave == 0) {
    int base = 0;
    for (int c = 0; c < nbe; c += 64) {
      const bool p = c + lane < nbe && sh.on[c + lane];
      const uint64_t b = __ballot(p);
      if (p) sh.act[base + __popcll(b & (lane ? ~0ull >> (64 - lane) : 0ull))] = c + lane;
      base += __popcll(b);
    }
    if (lane == 0) sh.na = base;
  }
  __syncthreads();
  const int na = sh.na;
  const int nap = (na + 31) / 32 * 32;

  // h = z u of the active neurons, as bf16 high and low parts: their sum
  // has 16 significant bits, so the down product sees h to 2^-17
  for (int c = 0; c < nap; c += 32) {
    f32x4_t acc[2][NTK] = {};
    if constexpr (GATED) {
      const int r[2] = {j0 + sh.act[min(c + (lane & 15), na - 1)],
                        j0 + sh.act[min(c + 16 + (lane & 15), na - 1)]};
      dots<MX, 2, NTK>(a, wu, r, xt, lane, wave, acc);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < NTK; ++t) sh.red[wave][i][t][lane] = acc[i][t];
      __syncthreads();
    }
    for (int e = tid; e < 2 * NTK * 64; e += NT) {
      const int i = e / (NTK * 64), t = (e >> 6) % NTK, l = e & 63;
      f32x4_t u = {1.0f, 1.0f, 1.0f, 1.0f};
      if constexpr (GATED) {
        u = sh.red[0][i][t][l];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) u += sh.red[w][i][t][l];
      }
      const int tk = t * 16 + (l & 15), j = c + i * 16 + 4 * (l >> 4);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float h = 0.0f;
        if (j + q < na) {
          const float z = sh.z[tk][sh.act[j + q]];
          h = z > 0.0f ? z * u[q] : 0.0f;
        }
        const __bf16 hh = (__bf16)h;
        const float hf = (float)hh;
        // an infinite or NaN h is all in its high part
        const __bf16 hl = (__bf16)(fabsf(hf) < INFINITY ? h - hf : 0.0f);
        sh.hi[tk][j + q] = __builtin_bit_cast(uint16_t, hh);
        sh.lo[tk][j + q] = __builtin_bit_cast(uint16_t, hl);
      }
    }
  }
  __syncthreads();

  // down: a wave has 128 columns at a time. A lane loads 8 columns of 8
  // neurons and turns them into 8 operands, one a column: operand q of lane
  // l holds column 8 (l % 16) + q at k = neurons 8 (l / 16) .. + 7, and the
  // results of a lane are 32 consecutive columns of token l % 16.
  const int kq = lane >> 4;
  for (int c0 = wave * 128; c0 < a.d; c0 += kWaves * 128) {
    f32x4_t acc[8][NTK] = {};
    const int col = c0 + 8 * (lane & 15);
    for (int ks = 0; ks < nap; ks += 32) {
      u32x4_t v[8];
      if constexpr (MX) {
        uint32_t q[8], sb[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = j0 + sh.act[min(ks + kq * 8 + j, na - 1)];
          q[j] = *(const uint32_t*)(wd.p + (int64_t)r * wd.pitch + col / 2);
          sb[j] = wd.sc[(c0 / 128) * wd.gpitch + (int64_t)r * 4 + ((lane & 15) >> 2)];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = from_codes(q[j], sb[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = j0 + sh.act[min(ks + kq * 8 + j, na - 1)];
          v[j] = *(const u32x4_t*)(wd.p + (int64_t)r * wd.pitch + col * 2);
        }
      }
      u32x4_t hh[NTK], hl[NTK];
#pragma unroll
      for (int t = 0; t < NTK; ++t) {
        hh[t] = *(const u32x4_t*)&sh.hi[t * 16 + (lane & 15)][ks + kq * 8];
        hl[t] = *(const u32x4_t*)&sh.lo[t * 16 + (lane & 15)][ks + kq * 8];
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        // low (q even) or high halves of neurons 2 i and 2 i + 1
        const uint32_t sel = (q & 1) ? 0x07060302u : 0x05040100u;
        u32x4_t o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = __builtin_amdgcn_perm(v[2 * i + 1][q >> 1], v[2 * i][q >> 1], sel);
#pragma unroll
        for (int t = 0; t < NTK; ++t) {
          acc[q][t] = mfma(o, hh[t], acc[q][t]);
          acc[q][t] = mfma(o, hl[t], acc[q][t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NTK; ++t) {
      const int tk = t * 16 + (lane & 15);
      if (tk >= nt) continue;
      float* o = a.part + ((int64_t)slice * a.T * a.k + ls.pair[p0 + tk]) * a.d + c0 + 32 * kq;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *(f32x4_t*)(o + 8 * i) = f32x4_t{acc[0][t][i], acc[1][t][i], acc[2][t][i], acc[3][t][i]};
        *(f32x4_t*)(o + 8 * i + 4) =
            f32x4_t{acc[4][t][i], acc[5][t][i], acc[6][t][i], acc[7][t][i]};
      }
    }
  }
}

template <bool MX, bool GATED, int NTK>
__global__ __launch_bounds__(NT) void moe_experts_kernel(MoeArgs a) {
  __shared__ Lists ls;
  __shared__ Shared<NTK> sh;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int e = blockIdx.y;
  const int slice = blockIdx.x;
  const int T = tokens(a);
  // the expert's rank for each token: the experts that come before it
  for (int t = wave; t < T; t += kWaves) {
    const long long* keys = a.keys + (int64_t)t * a.E;
    const long long mine = keys[e];
    int before = 0;
    for (int o = 0; o < a.E; o += 64) {
      const int f = o + lane;
      bool b = false;
      if (f < a.E) {
        const long long other = keys[f];
        b = other > mine || (other == mine && f < e);
      }
      before += __popcll(__ballot(b));
    }
    if (lane == 0) {
      ls.rank[t] = before;
      if (slice == 0 && before < a.k) {
        a.chosen[t * a.k + before] = mine;
        if (a.ids) a.ids[t * a.k + before] = e;
      }
    }
  }
  __syncthreads();
  // list its tokens, one a thread, in ascending order
  const int t = threadIdx.x;
  const bool mine = t < T && ls.rank[t] < a.k;
  const uint64_t b = __ballot(mine);
  if (lane == 0) ls.wsum[wave] = __popcll(b);
  __syncthreads();
  int at = __popcll(b & (lane ? ~0ull >> (64 - lane) : 0ull)), n = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) at += ls.wsum[w];
    n += ls.wsum[w];
  }
  if (mine) {
    ls.tok[at] = t;
    ls.pair[at] = t * a.k + ls.rank[t];
  }
  if (n == 0) return;
  __syncthreads();

  const int j0 = slice * a.nb;
  const int nbe = min(a.nb, a.F - j0);
  const int64_t pitch = MX ? a.d / 2 : (int64_t)a.d * 2;
  const int64_t row0 = (int64_t)e * a.F;
  const int64_t gp = (int64_t)a.E * a.F * 4;
  const Rows wg = {(const uint8_t*)a.wg + row0 * pitch, MX ? a.sg + row0 * 4 : nullptr, pitch, gp};
  const Rows wu = {GATED ? (const uint8_t*)a.wu + row0 * pitch : nullptr,
                   MX && GATED ? a.su + row0 * 4 : nullptr, pitch, gp};
  const Rows wd = {(const uint8_t*)a.wd + row0 * pitch, MX ? a.sd + row0 * 4 : nullptr, pitch, gp};
  for (int p0 = 0; p0 < n; p0 += 16 * NTK) {
    pass<MX, GATED, NTK>(a, sh, ls, wg, wu, wd, j0, nbe, n, p0, slice);
    __syncthreads();
  }
}

// ---------------------------------------------------------------- sum

// y of a token's 64 columns: 16 groups of 16 lanes share out the k S
// partial outputs and are added in LDS.
__global__ __launch_bounds__(NT) void moe_sum_kernel(MoeArgs a) {
  __shared__ float p[kMoeMaxK];
  __shared__ f32x4_t red[16][16];
  __shared__ float wsum[kWaves];
  const int t = blockIdx.y;
  if (t >= tokens(a)) return;
  const int tid = threadIdx.x;
  const double top = key_value(a.chosen[(int64_t)t * a.k]);
  if (tid < a.k) p[tid] = expf((float)(key_value(a.chosen[(int64_t)t * a.k + tid]) - top));
  float total = 0.0f;
  if (!a.normalize) {
    for (int e = tid; e < a.E; e += NT)
      total += expf((float)(key_value(a.keys[(int64_t)t * a.E + e]) - top));
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) total += __shfl_xor(total, o);
    if ((tid & 63) == 0) wsum[tid >> 6] = total;
  }
  __syncthreads();
  total = 0.0f;
  if (a.normalize) {
    for (int r = 0; r < a.k; ++r) total += p[r];
  } else {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) total += wsum[w];
  }
  if (blockIdx.x == 0 && a.probs && tid < a.k) a.probs[t * a.k + tid] = p[tid] / total;
  const int g = tid >> 4, c = blockIdx.x * 64 + (tid & 15) * 4;
  f32x4_t s = {};
  const int64_t stride = (int64_t)a.T * a.k * a.d;
  const float* base = a.part + (int64_t)t * a.k * a.d + c;
#pragma unroll 4
  for (int i = g; i < a.k * a.S; i += 16) {
    const int r = i % a.k, sl = i / a.k;
    s += *(const f32x4_t*)(base + sl * stride + (int64_t)r * a.d) * p[r];
  }
  red[g][tid & 15] = s;
  __syncthreads();
  if (tid < 16) {
    f32x4_t v = red[0][tid];
#pragma unroll
    for (int i = 1; i < 16; ++i) v += red[i][tid];
    *(f32x4_t*)(a.y + (int64_t)t * a.d + c) = v / total;
  }
}

template <bool MX, bool GATED>
hipError_t launch_experts(const MoeArgs& a, hipStream_t s) {
  const dim3 grid(a.S, a.E);
  if (a.T <= 16) moe_experts_kernel<MX, GATED, 1><<<grid, NT, 0, s>>>(a);
  else moe_experts_kernel<MX, GATED, 2><<<grid, NT, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

void moe_slices(int T, int F, int E, int k, int* nb, int* S) {
  // as many neurons a workgroup as leave two workgroups a CU over the
  // experts that T tokens can reach: fewer partial outputs to write and add
  const int64_t reach = (int64_t)T * k < E ? (int64_t)T * k : E;
  int b = kMoeSlice;
  while (b > 32 && reach * ((F + b - 1) / b) < 512) b /= 2;
  *nb = b;
  *S = (F + b - 1) / b;
}

hipError_t launch_moe(bool mx, const MoeArgs& a, hipStream_t s) {
  moe_logits_kernel<<<dim3((a.E + kWaves - 1) / kWaves, (a.T + kLogitT - 1) / kLogitT), NT, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool gated = a.wu != nullptr;
  e = mx ? (gated ? launch_experts<true, true>(a, s) : launch_experts<true, false>(a, s))
         : (gated ? launch_experts<false, true>(a, s) : launch_experts<false, false>(a, s));
  if (e != hipSuccess) return e;
  moe_sum_kernel<<<dim3(a.d / 64, a.T), NT, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace sffn
