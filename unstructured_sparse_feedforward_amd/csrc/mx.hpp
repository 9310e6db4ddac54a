// MXFP4 matrices, shared by the quantiser (mx.hip), the product
// (mx_gemm.hip) and the expert layer (moe.hip).
//
// A matrix [R, K] (blocks of 32 along K) is kept as
//   codes  [R, Kp / 2] bytes, Kp = K rounded up to 128: element k of a row
//          in byte k / 2, the even one in the low nibble;
//   scales [Kp / 128, R, 4] bytes: byte b of (g, r) is the scale exponent
//          plus 127 (255: NaN) of the block at k = 128 g + 32 b of row r.
// The padding elements' codes are 0. The scales of consecutive rows are
// consecutive dwords, so that a GEMM fetches those of a tile's rows for one
// 128-wide k step as one run, and a lane has the four of its row in a
// register (the scaled MFMAs select a byte of it).
#pragma once

#include "sffn_internal.hpp"

namespace sffn {

__host__ __device__ __forceinline__ int64_t mx_padded(int64_t K) { return (K + 127) / 128 * 128; }

hipError_t launch_mx_quantize(Dtype dt, const void* x, int64_t rows, int64_t cols, int64_t ldx,
                              bool transposed, uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_mx_dequantize(Dtype dt, const uint8_t* codes, const uint8_t* scales,
                                int64_t rows, int64_t cols, void* out, int64_t ldo, hipStream_t s);

// out[m, n] = sum_k a[m, k] b[n, k], stored as float32 or bf16
struct MxGemmArgs {
  const uint8_t* a;
  const uint8_t* a_sc;
  const uint8_t* b;
  const uint8_t* b_sc;
  int64_t M, N, K;
  void* out;
  int64_t ldo;
};
hipError_t launch_mx_gemm(Dtype out_dt, const MxGemmArgs& g, hipStream_t s);

}  // namespace sffn
