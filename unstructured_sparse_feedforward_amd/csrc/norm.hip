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
// and the result. Sums are float32.
#include "mx.hpp"
#include "norm.hpp"
#include "rowio.hpp"

namespace sffn {
namespace {

// A row is L lanes' (a wave's 64, or a workgroup's), who hold V pieces of CH
// consecutive elements each: piece v of lane l is at column (v L + l) CH.
template <int L>
struct Row {
  static constexpr int NT = L < 256 ? 256 : L;     // threads a workgroup
  static constexpr int ROWS = NT / L;              // rows a workgroup
};

template <int CH, typename E>
__device__ __forceinline__ void load_piece(const E* p, int left, float* v) {
  if (left >= CH) {
    if constexpr (CH == 8) load8(p, v);
    else load4(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < CH; ++j) v[j] = j < left ? ld(p + j) : 0.0f;
  }
}
template <int CH, typename E>
__device__ __forceinline__ void store_piece(E* p, int left, const float* v) {
  if (left >= CH) {
    if constexpr (CH == 8) store8(p, v);
    else store4(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (j < left) st(p + j, v[j]);
  }
}

// the lane's pieces of a row of a matrix of either type
template <int L, int V, int CH>
__device__ __forceinline__ void load_row(const void* p, int64_t at, int bf, int cols, int l,
                                         float (&v)[V][CH]) {
  if (bf) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * L + l) * CH;
      load_piece<CH>((const uint16_t*)p + at + c, cols - c, v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * L + l) * CH;
      load_piece<CH>((const float*)p + at + c, cols - c, v[i]);
    }
  }
}
template <int L, int V, int CH>
__device__ __forceinline__ void store_row(void* p, int64_t at, int bf, int cols, int l,
                                          const float (&v)[V][CH]) {
  if (bf) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * L + l) * CH;
      store_piece<CH>((uint16_t*)p + at + c, cols - c, v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * L + l) * CH;
      store_piece<CH>((float*)p + at + c, cols - c, v[i]);
    }
  }
}

// The sum of v over the row's lanes, in all of them, in an order that depends
// on L alone. share: a float a wave (unused for L = 64). Of a workgroup's
// calls, two in turn need two shares or a barrier between them.
template <int L>
__device__ __forceinline__ float row_sum(float v, float* share) {
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
template <int L, int V, int CH>
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
    if (c < Kp) {
      if constexpr (CH == 8) *(u32x2_t*)(codes + c) = Fp8::pack8(v[i], sb);
      else *(uint32_t*)(codes + c) = Fp8::pack4(v[i], sb);
    }
    uint32_t d = sb << (8 * (l / (32 / CH) % 4));
    d |= (uint32_t)__shfl_xor((int)d, 32 / CH);
    d |= (uint32_t)__shfl_xor((int)d, 64 / CH);
    if (l % (128 / CH) == 0 && c < Kp)
      *(uint32_t*)(a.out_sc + ((int64_t)(c / 128) * a.rows + row) * 4) = d;
  }
}

template <int L, int V, int CH>
__global__ __launch_bounds__(Row<L>::NT) void norm_kernel(NormArgs a) {
  __shared__ float share[16];
  const int l = threadIdx.x % L;
  const int64_t row = (int64_t)blockIdx.x * Row<L>::ROWS + threadIdx.x / L;
  if (row >= a.rows || (a.n_dev && row >= *a.n_dev)) return;   // (all lanes of a row)
  float s[V][CH], t[V][CH];
  load_row<L, V, CH>(a.x, row * a.ldx, a.x_bf, a.cols, l, s);
  if (a.res) {
    load_row<L, V, CH>(a.res, row * a.ldr, a.r_bf, a.cols, l, t);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        s[i][j] += t[i][j];
        if (a.r_bf) s[i][j] = bf16lo(bf16_bits(s[i][j]));
      }
    store_row<L, V, CH>(a.res_out, row * a.ldro, a.r_bf, a.cols, l, s);
  }
  if (a.weight) load_row<L, V, CH>(a.weight, 0, a.w_bf, a.cols, l, t);
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < CH; ++j) q = fmaf(s[i][j], s[i][j], q);
  const float r = 1.0f / sqrtf(row_sum<L>(q, share) / (float)a.cols + a.eps);
  if (a.rstd && l == 0) a.rstd[row] = r;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      s[i][j] *= r;
      // (columns past the last are 0 there: s is 0, and r may be infinite)
      if (a.weight) s[i][j] *= t[i][j];
      if ((i * L + l) * CH + j >= a.cols) s[i][j] = 0.0f;
    }
  if (a.out_kind == kMx8) store_mx8<L, V, CH>(a, row, l, s);
  else store_row<L, V, CH>(a.out, row * a.ldo, a.out_kind == kBF16, a.cols, l, s);
}

// A workgroup's rows are blockIdx.x ROWS + .., and every gridDim.x ROWS from
// there on: it sums its rows' dy xh in registers, its waves' sums through LDS,
// and writes one row of the workspace.
template <int L, int V, int CH>
__global__ __launch_bounds__(Row<L>::NT) void norm_grad_kernel(NormGradArgs a) {
  constexpr int ROWS = Row<L>::ROWS;
  __shared__ float share[2][16];
  __shared__ float red[ROWS > 1 ? (ROWS - 1) * L * V * CH : 1];
  const int l = threadIdx.x % L, mine = threadIdx.x / L;
  float w[V][CH], dw[V][CH] = {};
  if (a.weight) {
    load_row<L, V, CH>(a.weight, 0, a.w_bf, a.cols, l, w);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < CH; ++j) w[i][j] = 1.0f;
  }
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.rows; r0 += (int64_t)gridDim.x * ROWS) {
    const int64_t row = r0 + mine;
    if (L == 64 && row >= a.rows) break;      // (with L > 64 a workgroup has one row)
    float s[V][CH], g[V][CH], t[V][CH];
    load_row<L, V, CH>(a.s, row * a.lds, a.s_bf, a.cols, l, s);
    load_row<L, V, CH>(a.dy, row * a.lddy, a.dy_bf, a.cols, l, g);
    if (a.ds_in) load_row<L, V, CH>(a.ds_in, row * a.lddi, a.di_bf, a.cols, l, t);
    const float r = a.rstd[row];
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        s[i][j] *= r;
        dw[i][j] = fmaf(g[i][j], s[i][j], dw[i][j]);
        g[i][j] *= w[i][j];
        q = fmaf(g[i][j], s[i][j], q);
      }
    const float c = row_sum<L>(q, share[turn]) / (float)a.cols;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        s[i][j] = r * (g[i][j] - s[i][j] * c);
        if (a.ds_in) s[i][j] += t[i][j];
      }
    store_row<L, V, CH>(a.ds, row * a.ldds, a.ds_bf, a.cols, l, s);
  }
  if (!a.dw) return;
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
  store_row<L, V, CH>(a.part, (int64_t)blockIdx.x * a.cols, 0, a.cols, l, dw);
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

template <int L, int V, int CH>
hipError_t norm(const NormArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((a.rows + Row<L>::ROWS - 1) / Row<L>::ROWS);
  norm_kernel<L, V, CH><<<grid, Row<L>::NT, 0, s>>>(a);
  return hipGetLastError();
}
template <int L, int V, int CH>
hipError_t norm_grad(const NormGradArgs& a, hipStream_t s) {
  norm_grad_kernel<L, V, CH><<<a.parts, Row<L>::NT, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  if (a.cols <= 512) return norm<64, 1, 8>(a, s);
  if (a.cols <= 1024) return norm<64, 2, 8>(a, s);
  if (a.cols <= 2048) return norm<64, 4, 8>(a, s);
  if (a.cols <= 4096) return norm<256, 2, 8>(a, s);
  if (a.cols <= 8192) return norm<256, 4, 8>(a, s);
  return norm<512, 4, 8>(a, s);
}

int norm_grad_parts(int64_t rows, int64_t cols) {
  const int64_t each = cols <= 2048 ? 4 : 1;      // rows a workgroup at a time
  return (int)min((rows + each - 1) / each, (int64_t)512);
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.rows == 0) {}      // (dw is then 0)
  else if (a.cols <= 512) e = norm_grad<64, 1, 8>(a, s);
  else if (a.cols <= 1024) e = norm_grad<64, 2, 8>(a, s);
  else if (a.cols <= 2048) e = norm_grad<64, 4, 8>(a, s);
  else if (a.cols <= 4096) e = norm_grad<256, 2, 8>(a, s);
  else if (a.cols <= 8192) e = norm_grad<256, 4, 8>(a, s);
  else e = norm_grad<512, 4, 8>(a, s);
  if (e != hipSuccess || !a.dw) return e;
  norm_dw_kernel<<<(unsigned)((a.cols + 63) / 64), kDwWaves * 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace sffn
