// Products of two MXFP4 matrices, out = a b^T, by the scaled matrix
// instructions: every product of two elements is exact, the block scales
// enter inside the instruction, and the sums are float32.
#include "mx.hpp"

namespace sffn {
namespace {

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
constexpr int kFp4 = 4;   // operand format field of the f8f6f4 instructions

// 16 bytes (32 elements) of an operand; the instruction reads the first
// four registers of a 4-bit operand.
__device__ __forceinline__ i32x8_t frag(const i32x4_t v) {
  return i32x8_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) {
  *p = v == v ? (uint16_t)f32_to_bf16(v) : (uint16_t)0x7FC0;
}

// ---------------------------------------------------------------- few rows

// M <= 16 MT rows of a: one workgroup for 16 rows of b, whose waves share
// out K by 128-wide groups and add their sums in LDS. The rows of b are the
// instruction's first operand: lane l holds row l % 16, k = 32 (l / 16) ..
// + 31, and of the result four consecutive n of row m = l % 16.
constexpr int kFewWaves = 8;

template <int MT, typename O>
__global__ __launch_bounds__(kFewWaves * 64) void mx_few_kernel(MxGemmArgs g) {
  __shared__ f32x4_t red[kFewWaves][MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int64_t rb = mx_padded(g.K) / 2;
  const int G = (int)(rb / 64);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t n = min(n0 + (lane & 15), g.N - 1);
  const int kq = lane >> 4;
  const uint8_t* pb = g.b + n * rb + kq * 16;
  const uint8_t* pbs = g.b_sc + n * 4 + kq;
  const uint8_t* pa[MT];
  const uint8_t* pas[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = min((int64_t)(i * 16 + (lane & 15)), g.M - 1);
    pa[i] = g.a + m * rb + kq * 16;
    pas[i] = g.a_sc + m * 4 + kq;
  }
  f32x4_t acc[MT] = {};
#pragma unroll 4
  for (int t = wave; t < G; t += kFewWaves) {
    const i32x4_t bv = *(const i32x4_t*)(pb + (int64_t)t * 64);
    const int bs = pbs[(int64_t)t * g.N * 4];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const i32x4_t av = *(const i32x4_t*)(pa[i] + (int64_t)t * 64);
      const int as = pas[i][(int64_t)t * g.M * 4];
      acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(bv), frag(av), acc[i], kFp4,
                                                                kFp4, 0, bs, 0, as);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) red[wave][i][lane] = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < MT * 64; e += kFewWaves * 64) {
    const int i = e >> 6, l = e & 63;
    f32x4_t s = red[0][i][l];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += red[w][i][l];
    const int64_t m = i * 16 + (l & 15);
    if (m >= g.M) continue;
    const int64_t nn = n0 + 4 * (l >> 4);
    O* o = (O*)g.out + m * g.ldo + nn;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (nn + j < g.N) put(o + j, s[j]);
  }
}

// ---------------------------------------------------------------- tiles of 64

// A 64 x 64 tile a workgroup, its four waves sharing out K as above; the
// operands go from memory to registers. Lane l holds row l % 32 of an
// operand's 32-row block and k = 32 (l / 32) .. + 31 of a 64-wide step.
template <typename O>
__global__ __launch_bounds__(256) void mx_mid_kernel(MxGemmArgs g) {
  __shared__ float red[4][64 * 64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int64_t rb = mx_padded(g.K) / 2;
  const int G = (int)(rb / 64);
  const int64_t n0 = (int64_t)blockIdx.x * 64, m0 = (int64_t)blockIdx.y * 64;
  const int hi = lane >> 5;
  const uint8_t *pa[2], *pb[2], *pas[2], *pbs[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = min(m0 + i * 32 + (lane & 31), g.M - 1);
    const int64_t n = min(n0 + i * 32 + (lane & 31), g.N - 1);
    pa[i] = g.a + m * rb + hi * 16;
    pb[i] = g.b + n * rb + hi * 16;
    pas[i] = g.a_sc + m * 4;
    pbs[i] = g.b_sc + n * 4;
  }
  f32x16_t acc[2][2] = {};
#pragma unroll 2
  for (int t = wave; t < G; t += 4) {
    int as[2], bs[2];
    i32x4_t av[2][2], bv[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      as[i] = *(const int*)(pas[i] + (int64_t)t * g.M * 4);
      bs[i] = *(const int*)(pbs[i] + (int64_t)t * g.N * 4);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        av[i][s] = *(const i32x4_t*)(pa[i] + (int64_t)t * 64 + s * 32);
        bv[i][s] = *(const i32x4_t*)(pb[i] + (int64_t)t * 64 + s * 32);
      }
    }
    // the block of substep s is 2 s + hi: shifted so that byte 2 s is it
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      as[i] = (int)((uint32_t)as[i] >> (8 * hi));
      bs[i] = (int)((uint32_t)bs[i] >> (8 * hi));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            frag(av[i][0]), frag(bv[j][0]), acc[i][j], kFp4, kFp4, 0, as[i], 0, bs[j]);
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            frag(av[i][1]), frag(bv[j][1]), acc[i][j], kFp4, kFp4, 2, as[i], 2, bs[j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        red[wave][(i * 32 + 8 * (e / 4) + 4 * hi + e % 4) * 64 + j * 32 + (lane & 31)] =
            acc[i][j][e];
  __syncthreads();
  for (int e = threadIdx.x; e < 64 * 64; e += 256) {
    const int64_t m = m0 + e / 64, n = n0 + e % 64;
    if (m < g.M && n < g.N)
      put((O*)g.out + m * g.ldo + n, red[0][e] + red[1][e] + red[2][e] + red[3][e]);
  }
}

template <typename O>
hipError_t launch(const MxGemmArgs& g, hipStream_t s) {
  if (g.M <= 64) {
    const unsigned grid = (unsigned)((g.N + 15) / 16);
    if (g.M <= 16) mx_few_kernel<1, O><<<grid, kFewWaves * 64, 0, s>>>(g);
    else if (g.M <= 32) mx_few_kernel<2, O><<<grid, kFewWaves * 64, 0, s>>>(g);
    else mx_few_kernel<4, O><<<grid, kFewWaves * 64, 0, s>>>(g);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((g.N + 63) / 64), (unsigned)((g.M + 63) / 64));
  mx_mid_kernel<O><<<grid, 256, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_gemm(Dtype out_dt, const MxGemmArgs& g, hipStream_t s) {
  return out_dt == kBF16 ? launch<uint16_t>(g, s) : launch<float>(g, s);
}

}  // namespace sffn
