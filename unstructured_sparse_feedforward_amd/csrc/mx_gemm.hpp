// What the products of microscaled matrices share (mx_gemm.hip,
// mx8_gemm.hip): operand fragments, stores, the accumulators' reads.
#pragma once

#include "mx.hpp"

namespace sffn {

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
constexpr int kFp8 = 0, kFp4 = 4;   // operand format fields of the f8f6f4 instructions

// 16 bytes (32 elements) of a 4-bit operand, of whose registers the
// instruction reads the first four.
__device__ __forceinline__ i32x8_t frag(const i32x4_t v) {
  return i32x8_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) {
  *p = __builtin_bit_cast(uint16_t, (__bf16)v);   // to nearest even; NaN stays NaN
}

constexpr int kNXcd = 8;
constexpr int kCus = 256;
constexpr int kGroupM = 4;

// An accumulator at the point of use. 256 of them are in AGPRs: read there,
// one by one, or the compiler moves (and converts) them all before the
// epilogue's branch, which spills. (The compiler adds no wait states between
// a matrix instruction and inline asm that reads its result: see
// settle_sums.)
template <int MI>
__device__ __forceinline__ float sum_of(float a) {
  if constexpr (MI < 4) return a;
  float v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
  return v;
}

// Before the first sum_of after a matrix instruction: its result may be read 20
// wait states later (with an 8-bit operand, 16 passes) at the earliest; 24 here.
template <int MI>
__device__ __forceinline__ void settle_sums() {
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (MI == 4) asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace sffn
