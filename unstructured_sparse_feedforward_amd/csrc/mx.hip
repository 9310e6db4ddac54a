// MXFP4: quantisation of float32 and bf16 matrices to microscaled 4-bit
// floating point, and back. Every 32 consecutive elements of a row share a
// power-of-two scale 2^e, e = floor(log2 max|x|) - 2 (the exponent of the
// block's largest magnitude less that of the largest element, 6 = 1.5 * 4);
// an element is the e2m1 value nearest to x 2^-e (ties to the even code,
// saturated at 6). e comes from the exponent bits of the largest magnitude,
// so no logarithm is taken and the result is exact; the division and the
// rounding are one conversion instruction for two elements.
//
// Both directions are bound by memory: 2 or 4 bytes read and 17/32 byte
// written per element, against about three vector instructions.
#include "mx.hpp"

namespace sffn {
namespace {

constexpr int NT = 256;

// scale byte (e + 127) of a block whose largest magnitude has these bits.
// 255 (NaN): the block holds an infinity or a NaN. Subnormal and zero
// magnitudes land on the smallest scale.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int b = (int)(amax >> 23);
  return b == 255 ? 255u : (uint32_t)max(b - 2, 0);
}

// The conversions take a scale's exponent byte as it is (0 is 2^-127, 255
// NaN). 8 elements of a block as codes, the first in the lowest nibble.
__device__ __forceinline__ float scale_of(uint32_t sb) { return __uint_as_float(sb << 23); }
__device__ __forceinline__ uint32_t pack8(const float* v, uint32_t sb) {
  if (sb == 255u) return 0u;
  const float s = scale_of(sb);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
  return q;
}

__device__ __forceinline__ float ld(const float* p) { return *p; }
__device__ __forceinline__ float ld(const uint16_t* p) { return bf16lo(*p); }

// 8 elements in 16-byte loads that need no more than the elements' own
// alignment (the hardware's unaligned access)
typedef f32x4_t f32x4u_t __attribute__((aligned(4)));
typedef u32x4_t u32x4u_t __attribute__((aligned(2)));
__device__ __forceinline__ void load8(const float* p, float* v) {
  const f32x4_t a = *(const f32x4u_t*)p, b = *(const f32x4u_t*)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
}
__device__ __forceinline__ void load8(const uint16_t* p, float* v) {
  Vec<uint16_t, 8>::cvt(*(const u32x4u_t*)p, v);
}

// Rows as they are stored. A lane holds 8 consecutive elements, four lanes
// a block, a wave 512 columns (four 128-column groups) of kQRows rows; a
// workgroup's waves take consecutive rows, so that the scales of a group,
// four bytes a row, leave through LDS as runs of 16 * 4 bytes.
constexpr int kQRows = 4;                // rows a wave
constexpr int kQWg = kQRows * NT / 64;   // rows a workgroup

template <typename E>
__global__ __launch_bounds__(NT) void mx_quantize_kernel(const E* __restrict__ x, int64_t R,
                                                         int64_t K, int64_t ldx,
                                                         uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales) {
  __shared__ __align__(16) uint8_t sc[4][kQWg][4];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * kQWg;
  const int64_t c = (int64_t)blockIdx.y * 512 + lane * 8;
  const int64_t Kp = mx_padded(K);
  float v[kQRows][8];
#pragma unroll
  for (int i = 0; i < kQRows; ++i) {
    const int64_t r = r0 + wave * kQRows + i;
    const E* p = x + r * ldx + c;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (r < R) {
      if (c + 8 <= K) {
        load8(p, v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < K) v[i][j] = ld(p + j);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kQRows; ++i) {
    const int64_t r = r0 + wave * kQRows + i;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2));
    const uint32_t sb = scale_byte(m);
    if (r < R && c < Kp) *(uint32_t*)(codes + r * (Kp / 2) + c / 2) = pack8(v[i], sb);
    if ((lane & 3) == 0) sc[lane >> 4][wave * kQRows + i][(lane >> 2) & 3] = (uint8_t)sb;
  }
  __syncthreads();
  // the scales of 4 groups x kQWg rows, a dword each
  if (threadIdx.x < 4 * kQWg) {
    const int g = threadIdx.x / kQWg, rl = threadIdx.x % kQWg;
    const int64_t gg = (int64_t)blockIdx.y * 4 + g;
    if (gg < Kp / 128 && r0 + rl < R)
      *(uint32_t*)(scales + (gg * R + r0 + rl) * 4) = *(const uint32_t*)sc[g][rl];
  }
}

// The transpose of a stored matrix: output row c is column c of x [K, R],
// its blocks run down x's rows. A lane owns one column and a wave 32 rows
// of 64 columns, so a block's maximum is a lane's own and every load of a
// wave is one run of 64 elements. The workgroup's 8 waves cover 256 rows
// (two groups); their codes leave through LDS, 128 contiguous bytes for
// each of the 64 output rows.
constexpr int kTWaves = 8;

template <typename E>
__global__ __launch_bounds__(kTWaves * 64) void mx_quantize_t_kernel(
    const E* __restrict__ x, int64_t R, int64_t K, int64_t ldx, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales) {
  // 16-byte pieces, one a (column, wave), the piece index swizzled by the column
  __shared__ u32x4_t q[64][kTWaves];
  __shared__ __align__(16) uint8_t sc[2][64][4];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * 64;
  const int64_t k0 = (int64_t)blockIdx.y * (kTWaves * 32) + wave * 32;
  const int64_t Kp = mx_padded(K);
  const int64_t c = c0 + lane;
  float v[32];
  const E* p = x + k0 * ldx + c;
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = (c < R && k0 + j < K) ? ld(p + j * ldx) : 0.0f;
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  const uint32_t sb = scale_byte(m);
  u32x4_t o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = pack8(v + 8 * j, sb);
  q[lane][wave ^ (lane & 7)] = o;
  sc[wave >> 2][lane][wave & 3] = (uint8_t)sb;
  __syncthreads();
  {
    const int rl = threadIdx.x >> 3, piece = threadIdx.x & 7;
    const int64_t kk = (int64_t)blockIdx.y * (kTWaves * 32) + piece * 32;
    if (c0 + rl < R && kk < Kp)
      *(u32x4_t*)(codes + (c0 + rl) * (Kp / 2) + kk / 2) = q[rl][piece ^ (rl & 7)];
  }
  if (threadIdx.x < 128) {
    const int g = threadIdx.x >> 6, rl = threadIdx.x & 63;
    const int64_t gg = (int64_t)blockIdx.y * 2 + g;
    if (gg < Kp / 128 && c0 + rl < R)
      *(uint32_t*)(scales + (gg * R + c0 + rl) * 4) = *(const uint32_t*)sc[g][rl];
  }
}

__device__ __forceinline__ void store8(float* p, const float* v) {
  *(f32x4u_t*)p = f32x4_t{v[0], v[1], v[2], v[3]};
  *(f32x4u_t*)(p + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);   // NaN stays NaN
}
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
  *(u32x4u_t*)p = o;
}
__device__ __forceinline__ void st(float* p, float v) { *p = v; }
__device__ __forceinline__ void st(uint16_t* p, float v) { *p = (uint16_t)bf16_bits(v); }

// The values the codes stand for; the lanes' columns as in
// mx_quantize_kernel. A bf16 value is exact too (two significant bits)
// down to bf16's subnormals. Scale 255 makes the block NaN.
template <typename E>
__global__ __launch_bounds__(NT) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales,
                                                           int64_t R, int64_t K,
                                                           E* __restrict__ out, int64_t ldo) {
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * kQWg + wave * kQRows;
  const int64_t c = (int64_t)blockIdx.y * 512 + lane * 8;
  if (c >= K) return;
  const int64_t Kp = mx_padded(K);
  uint32_t q[kQRows], sb[kQRows];
#pragma unroll
  for (int i = 0; i < kQRows; ++i) {
    const int64_t r = r0 + i < R ? r0 + i : R - 1;
    q[i] = *(const uint32_t*)(codes + r * (Kp / 2) + c / 2);
    sb[i] = scales[((c >> 7) * R + r) * 4 + ((c >> 5) & 3)];
  }
#pragma unroll
  for (int i = 0; i < kQRows; ++i) {
    if (r0 + i >= R) break;
    const float s = scale_of(sb[i]);
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], s, 0);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], s, 1);
    const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], s, 2);
    const f32x2_t e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], s, 3);
    const float v[8] = {a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
    E* o = out + (r0 + i) * ldo + c;
    if (c + 8 <= K) {
      store8(o, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < K) st(o + j, v[j]);
    }
  }
}

}  // namespace

hipError_t launch_mx_quantize(Dtype dt, const void* x, int64_t rows, int64_t cols, int64_t ldx,
                              bool transposed, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  if (transposed) {
    // rows of x are the contracted axis
    const int64_t R = cols, K = rows;
    const dim3 grid((unsigned)((R + 63) / 64),
                    (unsigned)((mx_padded(K) + kTWaves * 32 - 1) / (kTWaves * 32)));
    if (dt == kBF16)
      mx_quantize_t_kernel<uint16_t><<<grid, kTWaves * 64, 0, s>>>((const uint16_t*)x, R, K, ldx,
                                                                   codes, scales);
    else
      mx_quantize_t_kernel<float><<<grid, kTWaves * 64, 0, s>>>((const float*)x, R, K, ldx, codes,
                                                                scales);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((rows + kQWg - 1) / kQWg), (unsigned)((mx_padded(cols) + 511) / 512));
  if (dt == kBF16)
    mx_quantize_kernel<uint16_t><<<grid, NT, 0, s>>>((const uint16_t*)x, rows, cols, ldx, codes,
                                                     scales);
  else
    mx_quantize_kernel<float><<<grid, NT, 0, s>>>((const float*)x, rows, cols, ldx, codes,
                                                  scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(Dtype dt, const uint8_t* codes, const uint8_t* scales,
                                int64_t rows, int64_t cols, void* out, int64_t ldo,
                                hipStream_t s) {
  const dim3 grid((unsigned)((rows + kQWg - 1) / kQWg), (unsigned)((cols + 511) / 512));
  if (dt == kBF16)
    mx_dequantize_kernel<uint16_t><<<grid, NT, 0, s>>>(codes, scales, rows, cols,
                                                       (uint16_t*)out, ldo);
  else
    mx_dequantize_kernel<float><<<grid, NT, 0, s>>>(codes, scales, rows, cols, (float*)out,
                                                    ldo);
  return hipGetLastError();
}

}  // namespace sffn
