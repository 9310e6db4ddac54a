// Rows of float32 or bf16 elements in 16- and 32-byte pieces that need no
// more than the elements' own alignment, and the two microscaled formats an
// element can be turned into.
#pragma once

#include "sffn_internal.hpp"

namespace sffn {

__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);   // to nearest even; NaN stays NaN
}

__device__ __forceinline__ float ld(const float* p) { return *p; }
__device__ __forceinline__ float ld(const uint16_t* p) { return bf16lo(*p); }
__device__ __forceinline__ void st(float* p, float v) { *p = v; }
__device__ __forceinline__ void st(uint16_t* p, float v) { *p = (uint16_t)bf16_bits(v); }

// (the hardware's unaligned access)
typedef f32x4_t f32x4u_t __attribute__((aligned(4)));
typedef u32x4_t u32x4u_t __attribute__((aligned(2)));
typedef u32x4_t u32x4w_t __attribute__((aligned(4)));
typedef u32x2_t u32x2u_t __attribute__((aligned(2)));

// 8 elements
__device__ __forceinline__ void load8(const float* p, float* v) {
  const f32x4_t a = *(const f32x4u_t*)p, b = *(const f32x4u_t*)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
}
__device__ __forceinline__ void load8(const uint16_t* p, float* v) {
  const u32x4_t a = *(const u32x4u_t*)p;     // (a reference would claim its own alignment)
  Vec<uint16_t, 8>::cvt(a, v);
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *(f32x4u_t*)p = f32x4_t{v[0], v[1], v[2], v[3]};
  *(f32x4u_t*)(p + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
  *(u32x4u_t*)p = o;
}

// 4 elements
__device__ __forceinline__ void load4(const float* p, float* v) {
  const f32x4_t a = *(const f32x4u_t*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = a[i];
}
__device__ __forceinline__ void load4(const uint16_t* p, float* v) {
  const u32x2_t a = *(const u32x2u_t*)p;
  Vec<uint16_t, 4>::cvt(a, v);
}
__device__ __forceinline__ void store4(float* p, const float* v) {
  *(f32x4u_t*)p = f32x4_t{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void store4(uint16_t* p, const float* v) {
  *(u32x2u_t*)p = u32x2_t{bf16_bits(v[0]) | (bf16_bits(v[1]) << 16),
                          bf16_bits(v[2]) | (bf16_bits(v[3]) << 16)};
}

// A microscaled format: TOP, the exponent of the largest element; the codes
// of 8 elements of a block, the first in the lowest bits, and back. A scale
// is kept as its exponent plus 127, `sb`; 255: the block holds an infinity
// or a NaN, and its codes are 0.

// The scale byte of a block whose largest magnitude has these bits.
// Subnormal and zero magnitudes land on the smallest scale.
template <typename F>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int b = (int)(amax >> 23);
  return b == 255 ? 255u : (uint32_t)max(b - F::TOP, 0);
}

// The conversions take a scale's exponent byte as it is (0 is 2^-127, 255
// NaN).
__device__ __forceinline__ float scale_of(uint32_t sb) { return __uint_as_float(sb << 23); }

// e2m1: the largest is 6 = 1.5 * 4
struct Fp4 {
  static constexpr int TOP = 2, BITS = 4;
  typedef uint32_t Codes8;
  __device__ static __forceinline__ Codes8 pack8(const float* v, uint32_t sb) {
    if (sb == 255u) return 0u;
    const float s = scale_of(sb);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
    return q;
  }
  __device__ static __forceinline__ void unpack8(Codes8 q, uint32_t sb, float* v) {
    const float s = scale_of(sb);
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 0);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 1);
    const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 2);
    const f32x2_t e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 3);
    v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
    v[4] = d[0]; v[5] = d[1]; v[6] = e[0]; v[7] = e[1];
  }
};

// e4m3: the largest is 448 = 1.75 * 256. A block's largest magnitude is
// below 512 scales, and the conversion gives NaN above 464: so the clamp.
// The division is a multiplication by 2^(127 - sb), exact but for results
// below float32's smallest normal, which are 0 in 8 bits.
struct Fp8 {
  static constexpr int TOP = 8, BITS = 8;
  typedef u32x2_t Codes8;
  __device__ static __forceinline__ uint32_t pack4(const float* v, uint32_t sb) {
    if (sb == 255u) return 0u;
    const float inv = __uint_as_float((254u - sb) << 23);
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __builtin_amdgcn_fmed3f(v[i] * inv, -448.0f, 448.0f);
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
  }
  __device__ static __forceinline__ Codes8 pack8(const float* v, uint32_t sb) {
    return Codes8{pack4(v, sb), pack4(v + 4, sb)};
  }
  __device__ static __forceinline__ void unpack8(Codes8 q, uint32_t sb, float* v) {
    const float s = scale_of(sb);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[i], s, false);
      const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[i], s, true);
      v[4 * i] = a[0]; v[4 * i + 1] = a[1]; v[4 * i + 2] = b[0]; v[4 * i + 3] = b[1];
    }
  }
};

}  // namespace sffn
