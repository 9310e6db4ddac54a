// MXFP4 and MXFP8: quantisation of float32 and bf16 matrices to microscaled
// 4- or 8-bit floating point, and back. Every 32 consecutive elements of a row
// share a power-of-two scale 2^e, e = floor(log2 max|x|) - TOP, TOP the
// exponent of the format's largest element (2 for e2m1, whose largest is 6 =
// 1.5 * 4; 8 for e4m3, 448 = 1.75 * 256); an element is the value of the
// format nearest to x 2^-e (ties to the even code, saturated at the
// largest). e comes from the exponent bits of the largest magnitude, so no
// logarithm is taken and the result is exact; the division and the rounding
// are one conversion instruction for two elements of 4 bits, two for one of
// 8.
//
// Both directions are bound by memory: 2 or 4 bytes read and 17/32 (33/32)
// byte written per element, against about three vector instructions.
#include "mx.hpp"
#include "rowio.hpp"

namespace sffn {
namespace {

constexpr int NT = 256;

// Rows as they are stored. A lane holds 8 consecutive elements, four lanes
// a block, a wave 512 columns (four 128-column groups) of kQRows rows; a
// workgroup's waves take consecutive rows, so that the scales of a group,
// four bytes a row, leave through LDS as runs of 16 * 4 bytes.
constexpr int kQRows = 4;                // rows a wave
constexpr int kQWg = kQRows * NT / 64;   // rows a workgroup

template <typename F, typename E>
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
    const uint32_t sb = scale_byte<F>(m);
    if (r < R && c < Kp)
      *(typename F::Codes8*)(codes + (r * Kp + c) * F::BITS / 8) = F::pack8(v[i], sb);
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
  const uint32_t sb = scale_byte<Fp4>(m);
  u32x4_t o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = Fp4::pack8(v + 8 * j, sb);
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

// The values the codes stand for; the lanes' columns as in
// mx_quantize_kernel. A bf16 value is exact too (two or four significant
// bits) down to bf16's subnormals. Scale 255 makes the block NaN.
template <typename F, typename E>
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
  typename F::Codes8 q[kQRows];
  uint32_t sb[kQRows];
#pragma unroll
  for (int i = 0; i < kQRows; ++i) {
    const int64_t r = r0 + i < R ? r0 + i : R - 1;
    q[i] = *(const typename F::Codes8*)(codes + (r * Kp + c) * F::BITS / 8);
    sb[i] = scales[((c >> 7) * R + r) * 4 + ((c >> 5) & 3)];
  }
#pragma unroll
  for (int i = 0; i < kQRows; ++i) {
    if (r0 + i >= R) break;
    float v[8];
    F::unpack8(q[i], sb[i], v);
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

template <typename F>
hipError_t launch_quantize(Dtype dt, const void* x, int64_t rows, int64_t cols, int64_t ldx,
                           uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const dim3 grid((unsigned)((rows + kQWg - 1) / kQWg), (unsigned)((mx_padded(cols) + 511) / 512));
  if (dt == kBF16)
    mx_quantize_kernel<F><<<grid, NT, 0, s>>>((const uint16_t*)x, rows, cols, ldx, codes, scales);
  else
    mx_quantize_kernel<F><<<grid, NT, 0, s>>>((const float*)x, rows, cols, ldx, codes, scales);
  return hipGetLastError();
}

template <typename F>
hipError_t launch_dequantize(Dtype dt, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                             int64_t cols, void* out, int64_t ldo, hipStream_t s) {
  const dim3 grid((unsigned)((rows + kQWg - 1) / kQWg), (unsigned)((cols + 511) / 512));
  if (dt == kBF16)
    mx_dequantize_kernel<F><<<grid, NT, 0, s>>>(codes, scales, rows, cols, (uint16_t*)out, ldo);
  else
    mx_dequantize_kernel<F><<<grid, NT, 0, s>>>(codes, scales, rows, cols, (float*)out, ldo);
  return hipGetLastError();
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
  return launch_quantize<Fp4>(dt, x, rows, cols, ldx, codes, scales, s);
}

hipError_t launch_mx8_quantize(Dtype dt, const void* x, int64_t rows, int64_t cols, int64_t ldx,
                               uint8_t* codes, uint8_t* scales, hipStream_t s) {
  return launch_quantize<Fp8>(dt, x, rows, cols, ldx, codes, scales, s);
}

hipError_t launch_mx_dequantize(Dtype dt, const uint8_t* codes, const uint8_t* scales,
                                int64_t rows, int64_t cols, void* out, int64_t ldo,
                                hipStream_t s) {
  return launch_dequantize<Fp4>(dt, codes, scales, rows, cols, out, ldo, s);
}

hipError_t launch_mx8_dequantize(Dtype dt, const uint8_t* codes, const uint8_t* scales,
                                 int64_t rows, int64_t cols, void* out, int64_t ldo,
                                 hipStream_t s) {
  return launch_dequantize<Fp8>(dt, codes, scales, rows, cols, out, ldo, s);
}

}  // namespace sffn
