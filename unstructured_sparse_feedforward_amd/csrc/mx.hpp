// MXFP4 matrices, shared by the quantiser (mx.hip), the products (mx_gemm.hip,
// mx8_gemm.hip) and the expert layer (moe.hip), and the copies into LDS of the
// products and the layer.
//
// A matrix [R, K] (blocks of 32 along K) is kept as
//   codes  [R, Kp / 2] bytes, Kp = K rounded up to 128: element k of a row
//          in byte k / 2, the even one in the low nibble;
//   scales [Kp / 128, R, 4] bytes: byte b of (g, r) is the scale exponent
//          plus 127 (255: NaN) of the block at k = 128 g + 32 b of row r.
// The padding elements' codes are 0, and so are the scale bytes of blocks that
// are all padding. (The product multiplies those too. Masking their scales in
// its kernels cost 1 to 7% of every product: 8192 x 8192 x 8192 256 to 269 us,
// 1 x 5632 x 2048 3.27 to 3.38.) The scales of consecutive rows are
// consecutive dwords, so that a GEMM fetches those of a tile's rows for one
// 128-wide k step as one run, and a lane has the four of its row in a
// register (the scaled MFMAs select a byte of it).
#pragma once

#include "sffn_internal.hpp"

namespace sffn {

__host__ __device__ __forceinline__ int64_t mx_padded(int64_t K) { return (K + 127) / 128 * 128; }

// ---------------------------------------------------------------- copies into LDS

// s_waitcnt immediate (vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt
// 11:8); a field at its maximum does not wait.
constexpr int wait_imm(int vm, int lgkm) {
  return (vm & 0xF) | ((vm >> 4) << 14) | (7 << 4) | (lgkm << 8);
}

// A point that neither the compiler nor its scheduler moves memory accesses
// across, and a wait there.
__device__ __forceinline__ void order_point() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
template <int IMM>
__device__ __forceinline__ void wait_point() {
  order_point();
  __builtin_amdgcn_s_waitcnt(IMM);
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

typedef __attribute__((address_space(3))) void lds_void;

// 16 (4) bytes a lane from base + voff into LDS at lds + 16 (4) x lane: a
// buffer load over a raw resource of the whole 32-bit range. Every offset
// formed here is inside the operand.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, -1, 0x00020000);
}
__device__ __forceinline__ void copy16(const uint8_t* base, uint32_t voff, char* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(base), (lds_void*)lds, 16, voff, 0, 0, 0);
}
__device__ __forceinline__ void copy4(const uint8_t* base, uint32_t voff, char* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(base), (lds_void*)lds, 4, voff, 0, 0, 0);
}

// Compile-time loop: f(Int<0>), .., f(Int<N - 1>).
template <int V>
struct Int {
  static constexpr int value = V;
};
template <int N, int K = 0, typename F>
__device__ __forceinline__ void unroll(F&& f) {
  if constexpr (K < N) {
    f(Int<K>{});
    unroll<N, K + 1>(f);
  }
}

// ---------------------------------------------------------------- launchers

hipError_t launch_mx_quantize(Dtype dt, const void* x, int64_t rows, int64_t cols, int64_t ldx,
                              bool transposed, uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_mx_dequantize(Dtype dt, const uint8_t* codes, const uint8_t* scales,
                                int64_t rows, int64_t cols, void* out, int64_t ldo, hipStream_t s);

// The same for MXFP8 (e4m3 elements): codes [R, Kp] bytes, element k of a row
// in byte k, the scales as above.
hipError_t launch_mx8_quantize(Dtype dt, const void* x, int64_t rows, int64_t cols, int64_t ldx,
                               uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_mx8_dequantize(Dtype dt, const uint8_t* codes, const uint8_t* scales,
                                 int64_t rows, int64_t cols, void* out, int64_t ldo,
                                 hipStream_t s);

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
// a in MXFP8, b in MXFP4
hipError_t launch_mx8_gemm(Dtype out_dt, const MxGemmArgs& g, hipStream_t s);

}  // namespace sffn
