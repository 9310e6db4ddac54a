// C ABI of the MXFP4 and MXFP8 calls (sffn_mx_*, sffn_mx8_*): argument validation and launches.
// See include/sffn.h for the contract of every entry point.
#include "mx.hpp"
#include "sffn.h"

namespace {

using namespace sffn;

constexpr int64_t kMaxRows = (int64_t)1 << 27;     // 32-bit grid sizes of the quantiser
constexpr int64_t kMaxGemmRows = (int64_t)1 << 21; // 64-row tiles within a grid's y extent
constexpr int64_t kMaxK = (int64_t)1 << 22;

bool aligned(const void* p, size_t a) { return p != nullptr && (uintptr_t)p % a == 0; }
bool float_type(int32_t dt) { return dt == SFFN_F32 || dt == SFFN_BF16; }
size_t elem(int32_t dt) { return dt == SFFN_BF16 ? 2 : 4; }
Dtype dt_of(int32_t dt) { return dt == SFFN_BF16 ? kBF16 : kF32; }
bool matrix_ok(const uint8_t* codes, const uint8_t* scales) {
  return aligned(codes, 16) && aligned(scales, 4);
}
sffn_status done(hipError_t e) { return e == hipSuccess ? SFFN_OK : SFFN_E_HIP; }

// the calls of both formats
typedef hipError_t Dequantize(Dtype, const uint8_t*, const uint8_t*, int64_t, int64_t, void*,
                              int64_t, hipStream_t);
typedef hipError_t Gemm(Dtype, const MxGemmArgs&, hipStream_t);

sffn_status bytes(int bits, int64_t rows, int64_t cols, size_t* code_bytes, size_t* scale_bytes) {
  if (!code_bytes || !scale_bytes || rows < 0 || cols < 0 || rows > kMaxRows || cols > kMaxK)
    return SFFN_E_ARG;
  const size_t Kp = (size_t)mx_padded(cols);
  *code_bytes = (size_t)rows * Kp * bits / 8;
  *scale_bytes = (size_t)rows * (Kp / 32);
  return SFFN_OK;
}

sffn_status dequantize(Dequantize* f, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                       int64_t cols, void* out, int32_t dtype, int64_t ldo, hipStream_t stream) {
  if (!float_type(dtype)) return SFFN_E_ARG;
  if (rows < 0 || cols < 0 || rows > kMaxRows || cols > kMaxK || ldo < cols) return SFFN_E_ARG;
  if (rows == 0 || cols == 0) return SFFN_OK;
  if (!aligned(out, elem(dtype)) || !matrix_ok(codes, scales)) return SFFN_E_ARG;
  return done(f(dt_of(dtype), codes, scales, rows, cols, out, ldo, stream));
}

sffn_status matmul(Gemm* f, const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                   const uint8_t* b_codes, const uint8_t* b_scales, int64_t N, int64_t K,
                   void* out, int32_t out_dtype, int64_t ldo, hipStream_t stream) {
  if (!float_type(out_dtype)) return SFFN_E_ARG;
  if (M < 0 || N < 0 || K < 0 || M > kMaxGemmRows || N > kMaxGemmRows || K > kMaxK || ldo < N)
    return SFFN_E_ARG;
  if (M == 0 || N == 0) return SFFN_OK;
  if (!aligned(out, elem(out_dtype))) return SFFN_E_ARG;
  if (K > 0 && (!matrix_ok(a_codes, a_scales) || !matrix_ok(b_codes, b_scales))) return SFFN_E_ARG;
  const MxGemmArgs g = {a_codes, a_scales, b_codes, b_scales, M, N, K, out, ldo};
  return done(f(dt_of(out_dtype), g, stream));
}

}  // namespace

extern "C" {

sffn_status sffn_mx_bytes(int64_t rows, int64_t cols, size_t* code_bytes, size_t* scale_bytes) {
  return bytes(4, rows, cols, code_bytes, scale_bytes);
}

sffn_status sffn_mx8_bytes(int64_t rows, int64_t cols, size_t* code_bytes, size_t* scale_bytes) {
  return bytes(8, rows, cols, code_bytes, scale_bytes);
}

sffn_status sffn_mx_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                             int32_t transposed, uint8_t* codes, uint8_t* scales,
                             hipStream_t stream) {
  if (!float_type(dtype) || (transposed != 0 && transposed != 1)) return SFFN_E_ARG;
  if (rows < 0 || cols < 0 || ldx < cols) return SFFN_E_ARG;
  if ((transposed ? cols : rows) > kMaxRows || (transposed ? rows : cols) > kMaxK)
    return SFFN_E_ARG;
  if (rows == 0 || cols == 0) return SFFN_OK;
  if (!aligned(x, elem(dtype)) || !matrix_ok(codes, scales)) return SFFN_E_ARG;
  return done(launch_mx_quantize(dt_of(dtype), x, rows, cols, ldx, transposed == 1, codes, scales,
                                 stream));
}

sffn_status sffn_mx8_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols,
                              int64_t ldx, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (!float_type(dtype)) return SFFN_E_ARG;
  if (rows < 0 || cols < 0 || ldx < cols || rows > kMaxRows || cols > kMaxK) return SFFN_E_ARG;
  if (rows == 0 || cols == 0) return SFFN_OK;
  if (!aligned(x, elem(dtype)) || !matrix_ok(codes, scales)) return SFFN_E_ARG;
  return done(launch_mx8_quantize(dt_of(dtype), x, rows, cols, ldx, codes, scales, stream));
}

sffn_status sffn_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                               int64_t cols, void* out, int32_t dtype, int64_t ldo,
                               hipStream_t stream) {
  return dequantize(launch_mx_dequantize, codes, scales, rows, cols, out, dtype, ldo, stream);
}

sffn_status sffn_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int64_t cols, void* out, int32_t dtype, int64_t ldo,
                                hipStream_t stream) {
  return dequantize(launch_mx8_dequantize, codes, scales, rows, cols, out, dtype, ldo, stream);
}

sffn_status sffn_mx_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                           const uint8_t* b_codes, const uint8_t* b_scales, int64_t N, int64_t K,
                           void* out, int32_t out_dtype, int64_t ldo, hipStream_t stream) {
  return matmul(launch_mx_gemm, a_codes, a_scales, M, b_codes, b_scales, N, K, out, out_dtype,
                ldo, stream);
}

sffn_status sffn_mx8_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                            const uint8_t* b_codes, const uint8_t* b_scales, int64_t N, int64_t K,
                            void* out, int32_t out_dtype, int64_t ldo, hipStream_t stream) {
  return matmul(launch_mx8_gemm, a_codes, a_scales, M, b_codes, b_scales, N, K, out, out_dtype,
                ldo, stream);
}

}  // extern "C"
