// The residual's addition and the root-mean-square norm of the sum,
//
//   s = x + res  (rounded to res's type, and kept),
//   r = 1 / sqrt(mean s^2 + eps),   y = s r w,
//
// with y in float32, bf16 or MXFP8, and its gradient: with xh = s r and
// g = dy w,
//
//   ds = r (g - xh mean(g xh)) + ds_in,    dw = sum over rows of dy xh.
//
// A row is read once and stays in registers between the sum of its squares
// and the result. Sums are float32, those of results in float32 and MXFP8
// float64.
#include "mx.hpp"
#include "norm.hpp"
#include "rowio.hpp"

namespace sffn {
namespace {

// A row is L lanes' (a wave's 64, or a workgroup's), who hold V pieces of CH
// consecutive elements each: piece v of lane l is at column (v L + l) CH.
constexpr int CH = 8;
template <int L>
struct Row {
  static constexpr int NT = L == 64 ? 256 : L;     // threads a workgroup
  static constexpr int ROWS = NT / L;              // rows a workgroup
};

template <typename E>
__device__ __forceinline__ void store_piece(E* p, int left, const float* v) {
  if (left >= CH) {
    store8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (j < left) st(p + j, v[j]);
  }
}

// The lane's pieces of a row of a matrix of either type, as they are in
// memory (a: float32 0 .. 3 or all of bf16, b: float32 4 .. 7), and their
// values: apart, so that a load is waited for only where its values are used.
struct Piece {
  u32x4_t a, b;
};
template <int L, int V>
__device__ __forceinline__ void load_row(const void* p, int64_t at, int bf, int cols, int l,
                                         Piece (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * L + l) * CH, left = cols - c;
    if (bf) {
      const uint16_t* q = (const uint16_t*)p + at + c;
      if (left >= CH) {
        v[i].a = *(const u32x4u_t*)q;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[i].a[j] = (2 * j < left ? (uint32_t)q[2 * j] : 0u) |
                      (2 * j + 1 < left ? (uint32_t)q[2 * j + 1] << 16 : 0u);
      }
    } else {
      const uint32_t* q = (const uint32_t*)p + at + c;
      if (left >= CH) {
        v[i].a = *(const u32x4w_t*)q;
        v[i].b = *(const u32x4w_t*)(q + 4);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i].a[j] = j < left ? q[j] : 0u;
          v[i].b[j] = 4 + j < left ? q[4 + j] : 0u;
        }
      }
    }
  }
}
template <int V>
__device__ __forceinline__ void values(const Piece (&v)[V], int bf, float (&o)[V][CH]) {
  if (bf) {
#pragma unroll
    for (int i = 0; i < V; ++i) Vec<uint16_t, 8>::cvt(v[i].a, o[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[i][j] = __uint_as_float(v[i].a[j]);
        o[i][4 + j] = __uint_as_float(v[i].b[j]);
      }
  }
}
template <int L, int V>
__device__ __forceinline__ void store_row(void* p, int64_t at, int bf, int cols, int l,
                                          const float (&v)[V][CH]) {
  if (bf) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * L + l) * CH;
      store_piece((uint16_t*)p + at + c, cols - c, v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * L + l) * CH;
      store_piece((float*)p + at + c, cols - c, v[i]);
    }
  }
}

// The sum of v over the row's lanes, in all of them, in an order that depends
// on L alone. share: a value a wave (unused for L = 64). Of a workgroup's
// calls, two in turn need two shares or a barrier between them.
template <int L, typename T>
__device__ __forceinline__ T row_sum(T v, T* share) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0) share[threadIdx.x >> 6] = v;
    __syncthreads();
    v = share[0];
#pragma unroll
    for (int w = 1; w < L / 64; ++w) v += share[w];
  }
  return v;
}

// The lane's pieces of a row as MXFP8. 32 / CH lanes have a block, 128 / CH
// the four whose scales are a dword.
template <int L, int V>
__device__ __forceinline__ void store_mx8(const NormArgs& a, int64_t row, int l,
                                          const float (&v)[V][CH]) {
  const int Kp = (int)mx_padded(a.cols);
  uint8_t* codes = (uint8_t*)a.out + row * Kp;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * L + l) * CH;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < CH; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < 32 / CH; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    const uint32_t sb = scale_byte<Fp8>(m);
    if (c < Kp) *(u32x2_t*)(codes + c) = Fp8::pack8(v[i], sb);
    uint32_t d = sb << (8 * (l / (32 / CH) % 4));
    d |= (uint32_t)__shfl_xor((int)d, 32 / CH);
    d |= (uint32_t)__shfl_xor((int)d, 64 / CH);
    if (l % (128 / CH) == 0 && c < Kp)
      *(uint32_t*)(a.out_sc + ((int64_t)(c / 128) * a.rows + row) * 4) = d;
  }
}

// WIDE (results in float32 and MXFP8): the sum and the products in 64 bits, y
// rounded once, so that a result in 8 bits is that of the formula but where y
// lies within half a step of float32 of a border, and not four of them. It costs
// most for MXFP8 from bf16, which is bound by its instructions (8192 x 2048 29.9
// us, in 32 bits 28.0; without a residual 20.9, 18.4; from float32 45.5, 45.5).
// r by quotients and a root in 64 bits, in place of 1 / cols from the host and
// rsqrt, took 33.2 and 23.7 us (31.1 and 21.7 otherwise the same). A bf16
// result's own rounding is 2^15 times what 64 bits would gain.
template <int L, int V, bool WIDE>
__global__ __launch_bounds__(Row<L>::NT) void norm_kernel(NormArgs a) {
  typedef std::conditional_t<WIDE, double, float> T;
  __shared__ T share[WIDE ? 1 : 2][16];
  const int l = threadIdx.x % L;
  const int64_t row = (int64_t)blockIdx.x * Row<L>::ROWS + threadIdx.x / L;
  if (row >= a.rows || (a.n_dev && row >= *a.n_dev)) return;   // (all lanes of a row)
  Piece ps[V], pr[V], pw[V];
  float s[V][CH], t[V][CH];
  load_row<L, V>(a.x, row * a.ldx, a.x_bf, a.cols, l, ps);
  if (a.res) load_row<L, V>(a.res, row * a.ldr, a.r_bf, a.cols, l, pr);
  if (a.weight) load_row<L, V>(a.weight, 0, a.w_bf, a.cols, l, pw);
  values(ps, a.x_bf, s);
  if (a.res) {
    values(pr, a.r_bf, t);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        s[i][j] += t[i][j];
        if (a.r_bf) s[i][j] = bf16lo(bf16_bits(s[i][j]));
      }
    store_row<L, V>(a.res_out, row * a.ldro, a.r_bf, a.cols, l, s);
  }
  T q = 0;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < CH; ++j) q = fma((T)s[i][j], (T)s[i][j], q);
  T r = row_sum<L>(q, share[0]);
  float rstd;
  if constexpr (WIDE) {
    r = rsqrt(fma(r, a.inv_cols, (double)a.eps));
    rstd = (float)r;
  } else {
    r = r / (float)a.cols + a.eps;
    // (a wave's lanes have one r; as bits, 2^-100 to infinity)
    const uint32_t bits = __builtin_amdgcn_readfirstlane(__float_as_uint(r));
    if (__builtin_expect(bits - 0x0D800000u >= 0x7F800000u - 0x0D800000u, 0)) {
      // Squares that float32 does not hold: again those of s m. (Any other mean is
      // off by at most 2^-150, half of float32's smallest step, of each square.)
      // m of small ones stays with s, since r may be above float32; m of large ones
      // goes to r, since s m would lose the row's smallest. (No other row's result
      // changes; us with and without this, 8192 x 2048 bf16 26.1, 26.0, 1024 x
      // 16384 33.7, 33.1.)
      const bool small = r < 1.0f;
      const float m = small ? 0x1p100f : 0x1p-100f;
      q = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          q = fmaf(s[i][j] * m, s[i][j] * m, q);
          if (small) s[i][j] *= m;
        }
      r = 1.0f / sqrtf(row_sum<L>(q, share[1]) / (float)a.cols + a.eps * m * m);
      rstd = r * m;
      if (!small) r = rstd;
    } else {
      r = 1.0f / sqrtf(r);
      rstd = r;
    }
  }
  if (a.rstd && l == 0) a.rstd[row] = rstd;
  if (a.weight) values(pw, a.w_bf, t);
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < CH; ++j)
      s[i][j] = (float)(a.weight ? (T)s[i][j] * r * (T)t[i][j] : (T)s[i][j] * r);
    // columns past the last are 0 in MXFP8: s is 0, but r may be infinite
    const int left = a.cols - (i * L + l) * CH;
    if (WIDE && left < CH) {
#pragma unroll
      for (int j = 0; j < CH; ++j)
        if (j >= left) s[i][j] = 0.0f;
    }
  }
  if (WIDE && a.out_kind == kMx8) store_mx8<L, V>(a, row, l, s);
  else store_row<L, V>(a.out, row * a.ldo, !WIDE, a.cols, l, s);
}

// dw of kSlab columns over all rows, by a workgroup of NT threads: four lanes
// have 8 columns each of a row (of cols >= 8; the last ones' run is moved to end
// with the row), so a wave 16 rows; 8 rows of a lane are loaded at a time.
constexpr int kSlab = 32;
template <int NT>
__device__ __forceinline__ void columns_dw(const NormGradArgs& a, int slab, float* red) {
  constexpr int STEP = NT / 4, U = 8;
  const int c = slab * kSlab + (threadIdx.x & 3) * CH, c0 = min(c, a.cols - CH);
  float dw[CH] = {};
  for (int64_t r0 = threadIdx.x >> 2; r0 < a.rows; r0 += STEP * U) {
    Piece s[U][1], g[U][1];
    float r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = min(r0 + u * STEP, a.rows - 1);
      load_row<1, 1>(a.s, row * a.lds + c0, a.s_bf, CH, 0, s[u]);
      load_row<1, 1>(a.dy, row * a.lddy + c0, a.dy_bf, CH, 0, g[u]);
      r[u] = a.rstd[row];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r0 + u * STEP >= a.rows) break;
      float sv[1][CH], gv[1][CH];
      values(s[u], a.s_bf, sv);
      values(g[u], a.dy_bf, gv);
#pragma unroll
      for (int j = 0; j < CH; ++j) dw[j] = fmaf(gv[0][j], sv[0][j] * r[u], dw[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < CH; ++j) {
#pragma unroll
    for (int o = 4; o < 64; o <<= 1) dw[j] += __shfl_xor(dw[j], o);
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane < 4) {
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (c0 + j >= c) red[wave * kSlab + c0 + j - slab * kSlab] = dw[j];
  }
  __syncthreads();
  const int col = slab * kSlab + threadIdx.x;
  if (threadIdx.x < kSlab && col < a.cols) {
    float v = red[threadIdx.x];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) v += red[w * kSlab + threadIdx.x];
    a.dw[col] = v;
  }
}

// A workgroup's rows are blockIdx.x ROWS + .., and every gridDim.x ROWS from
// there on: it sums its rows' dy xh in registers, its waves' sums through LDS,
// and writes one row of the workspace.
//
// ONE: little enough to be read a second time: the first a.slabs workgroups
// form dw, which needs no row's sum, from columns of their own, the others ds
// of a row each, and there is no second launch (777 x 1003 bf16: a call 14.5
// us, 10 so).
template <int L, int V, bool ONE>
__global__ __launch_bounds__(Row<L>::NT) void norm_grad_kernel(NormGradArgs a) {
  constexpr int ROWS = Row<L>::ROWS, NT = Row<L>::NT;
  __shared__ float share[2][16];
  __shared__ float red[ONE ? NT / 64 * kSlab : ROWS > 1 ? (ROWS - 1) * L * V * CH : 1];
  const int l = threadIdx.x % L, mine = threadIdx.x / L;
  const int block = ONE ? (int)blockIdx.x - a.slabs : (int)blockIdx.x;
  if (ONE && block < 0) {
    columns_dw<NT>(a, blockIdx.x, red);
    return;
  }
  // The next row's loads are issued before this row's sum is waited for, and
  // the weights are kept (of rows over 8192 both would take more registers than
  // 16 waves have).
  constexpr bool AHEAD = L * V <= 1024;
  float w[V][CH], dw[V][CH] = {};
  auto load_weight = [&] {
    if (a.weight) {
      Piece p[V];
      load_row<L, V>(a.weight, 0, a.w_bf, a.cols, l, p);
      values(p, a.w_bf, w);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < CH; ++j) w[i][j] = 1.0f;
    }
  };
  if (AHEAD) load_weight();
  Piece ps[V], pg[V], pd[V];
  float r = 0.0f;
  auto load = [&](int64_t row) {
    load_row<L, V>(a.s, row * a.lds, a.s_bf, a.cols, l, ps);
    load_row<L, V>(a.dy, row * a.lddy, a.dy_bf, a.cols, l, pg);
    if (a.ds_in) load_row<L, V>(a.ds_in, row * a.lddi, a.di_bf, a.cols, l, pd);
    r = a.rstd[row];
  };
  const int64_t step = (int64_t)(ONE ? gridDim.x - a.slabs : gridDim.x) * ROWS;
  int64_t row = (int64_t)block * ROWS + mine;    // (with L > 64 a workgroup has one row)
  int turn = 0;
  if (AHEAD && row < a.rows) load(row);
  for (; row < a.rows; row += step) {
    if (!AHEAD) {
      load(row);
      load_weight();
    }
    float s[V][CH], g[V][CH], q = 0.0f;
    values(ps, a.s_bf, s);
    values(pg, a.dy_bf, g);
    const float r0 = r;
    Piece p0[AHEAD ? V : 1];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (AHEAD) p0[i] = pd[i];
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        s[i][j] *= r0;
        dw[i][j] = fmaf(g[i][j], s[i][j], dw[i][j]);
        g[i][j] *= w[i][j];
        q = fmaf(g[i][j], s[i][j], q);
      }
    }
    if (AHEAD && row + step < a.rows) load(row + step);
    const float c = row_sum<L>(q, share[turn]) / (float)a.cols;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < CH; ++j) s[i][j] = r0 * (g[i][j] - s[i][j] * c);
    if (a.ds_in) {
      if constexpr (AHEAD) values(p0, a.di_bf, g);
      else values(pd, a.di_bf, g);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < CH; ++j) s[i][j] += g[i][j];
    }
    store_row<L, V>(a.ds, row * a.ldds, a.ds_bf, a.cols, l, s);
  }
  if (ONE || !a.dw) return;
  if constexpr (ROWS > 1) {
    if (mine > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < CH; ++j) red[((mine - 1) * V * CH + i * CH + j) * L + l] = dw[i][j];
    }
    __syncthreads();
    if (mine > 0) return;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int m = 0; m < ROWS - 1; ++m) dw[i][j] += red[(m * V * CH + i * CH + j) * L + l];
  }
  store_row<L, V>(a.part, (int64_t)blockIdx.x * a.cols, 0, a.cols, l, dw);
}

// dw from the workgroups' sums: 64 columns a workgroup, its 16 waves share out
// the rows of the workspace (in an order that depends on the sizes alone).
constexpr int kDwWaves = 16;
__global__ __launch_bounds__(kDwWaves * 64) void norm_dw_kernel(NormGradArgs a) {
  __shared__ float red[kDwWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < a.cols) {
#pragma unroll 8
    for (int p = wave; p < a.parts; p += kDwWaves) s += a.part[(int64_t)p * a.cols + c];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < a.cols) {
#pragma unroll
    for (int w = 1; w < kDwWaves; ++w) s += red[w][lane];
    a.dw[c] = s;
  }
}

template <int L, int V>
hipError_t norm(const NormArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((a.rows + Row<L>::ROWS - 1) / Row<L>::ROWS);
  if (a.out_kind != kBF16) norm_kernel<L, V, true><<<grid, Row<L>::NT, 0, s>>>(a);
  else norm_kernel<L, V, false><<<grid, Row<L>::NT, 0, s>>>(a);
  return hipGetLastError();
}
template <int L, int V>
hipError_t norm_grad(const NormGradArgs& a, hipStream_t s) {
  if constexpr (L * V * CH <= 8192) {
    if (a.parts == 0) {
      const unsigned rows = (unsigned)((a.rows + Row<L>::ROWS - 1) / Row<L>::ROWS);
      if (a.slabs == 0 || !a.in_place) {
        norm_grad_kernel<L, V, true><<<a.slabs + rows, Row<L>::NT, 0, s>>>(a);
        return hipGetLastError();
      }
      // The slabs read every row of dy and s, which ds would overwrite under
      // them: all of dw first, then the rows, in launches of their own.
      norm_grad_kernel<L, V, true><<<a.slabs, Row<L>::NT, 0, s>>>(a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      NormGradArgs b = a;
      b.slabs = 0;
      norm_grad_kernel<L, V, true><<<rows, Row<L>::NT, 0, s>>>(b);
      return hipGetLastError();
    }
  }
  norm_grad_kernel<L, V, false><<<a.parts, Row<L>::NT, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

// Threads for a row by its columns, 8 a thread up to a workgroup's most: the
// fewer a thread, the more rows a CU has in flight (us, from graphs, out of the
// caches: 8192 x 2048 bf16 in, out and stream 27.4, by 64 threads of 32 columns
// 30.5, by 512 of 4 34; 4096 x 4096 27.9, 256 of 16 29.7). A wave or more a
// row: 64 threads of 16 columns for 777 x 1003 6.5, 128 of 8 5.9.
int norm_threads(int64_t cols) {
  return cols <= 512 ? 64 : cols <= 1024 ? 128 : cols <= 2048 ? 256 : cols <= 4096 ? 512 : 1024;
}
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  switch (norm_threads(a.cols)) {
    case 64: return norm<64, 1>(a, s);
    case 128: return norm<128, 1>(a, s);
    case 256: return norm<256, 1>(a, s);
    case 512: return norm<512, 1>(a, s);
    default: return a.cols <= 8192 ? norm<1024, 1>(a, s) : norm<1024, 2>(a, s);
  }
}

// Whether one launch forms ds and dw: up to 2^21 elements, whose second reading
// is from the caches, and 2048 rows, which a workgroup sums in little time (us,
// from graphs: 777 x 1003 bf16 7.3, two launches 9.3; 1024 x 2048 float32 11.5,
// 13.4; 2000 x 256 10.4, 9.3, where the second launch costs the host 4 more; 4096
// x 512 25.6, 12.9; 2048 x 2048 bf16 14.7, 13.6).
static bool norm_grad_one(int64_t rows, int64_t cols) {
  return cols >= CH && cols <= 8192 && rows <= 2048 && rows * cols <= (int64_t)1 << 21;
}
int norm_grad_slabs(int64_t cols) { return (int)((cols + kSlab - 1) / kSlab); }

// The gradient's workgroups, each of which writes its sums for dw: as many as
// keep the memory busy (8192 x 2048: float32 53 us, by 256 52, 1024 56; bf16 31,
// 40, 33; 4096 x 4096 47, by 512 49; 16384 x 64 13.5, by 512 15.4).
int norm_grad_parts(int64_t rows, int64_t cols) {
  if (norm_grad_one(rows, cols)) return 0;
  const int64_t each = cols <= 1024 ? 4 : 1;      // rows a workgroup at a time
  const int64_t most = cols <= 512 ? 768 : cols <= 2048 ? 512 : 256;
  return (int)min((rows + each - 1) / each, most);
}

// Its threads: up to 1024 columns a wave has a row, and no barrier (8192 x 1000
// float32 32.6 us, by 128 threads 36.2; 777 x 1003 9.3, 10.4).
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.rows == 0) {}      // (dw is then 0)
  else if (a.cols <= 512) e = norm_grad<64, 1>(a, s);
  else if (a.cols <= 1024) e = norm_grad<64, 2>(a, s);
  else if (a.cols <= 2048) e = norm_grad<256, 1>(a, s);
  else if (a.cols <= 4096) e = norm_grad<512, 1>(a, s);
  else if (a.cols <= 8192) e = norm_grad<512, 2>(a, s);
  else e = norm_grad<1024, 2>(a, s);
  if (e != hipSuccess || !a.dw || (a.parts == 0 && a.rows > 0)) return e;
  norm_dw_kernel<<<(unsigned)((a.cols + 63) / 64), kDwWaves * 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace sffn
