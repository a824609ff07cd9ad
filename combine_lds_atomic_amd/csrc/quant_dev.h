// Block-128 e4m3 quantisation, shared by the kernels that write 8-bit rows:
// dispatch (from bfloat16 tokens), the norm and the SwiGLU product (from
// float32).
#pragma once

#include "moe_internal.h"

namespace moe {

// The scale of a 128-element block from the largest |x| of the block, given
// as the integer bit pattern of a non-negative float: amax / 448 (IEEE
// division).  A block of zeros has scale 0, and so has one whose quotient is
// below half of float32's smallest number (amax < 3.2e-43).  Compared as
// integers, infinity and NaN are above every finite value, so a block that
// holds one gets that scale.
__device__ __forceinline__ float block_scale(int amax_bits) { return __uint_as_float((uint32_t)amax_bits) / 448.0f; }

// Four quotients as e4m3fn bytes, little end first.  v_cvt_pk_fp8_f32 converts
// two floats to OCP e4m3fn per instruction, rounded to nearest even; what is up
// to 464 rounds to 448, and all above becomes NaN.
__device__ __forceinline__ uint32_t fp8x4(const float (&q)[4]) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
  return (uint32_t)w;
}

// Four quotients v[i] / scale (IEEE division) of bfloat16 values, for a scale
// above 0.  No block of bfloat16 values has a scale below 2.0e-43, whose
// quotients are at most 450; the exhaustive sweep test checks the bytes against
// the oracle's encoder on every bfloat16 pair x <= amax.
__device__ __forceinline__ uint32_t quant4(const float* v, float scale) {
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = v[i] / scale;
  return fp8x4(q);
}

// The same for float32 values, saturated, and zero bytes where the scale is 0.
// Quotients pass 448 by a rounding where the scale is a normal number, and by
// up to a half where it is a subnormal one of few bits: only those are held to
// 448 (a select for every value took 2% of the norm's time).
__device__ __forceinline__ uint32_t quant4_scaled(const float* v, float scale) {
  if (scale == 0.0f) return 0u;
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = v[i] / scale;
  if (__builtin_expect(scale < 0x1p-126f, 0)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = fminf(fmaxf(q[i], -448.0f), 448.0f);
  }
  return fp8x4(q);
}

__device__ __forceinline__ int abs_bits(float v) { return (int)(__float_as_uint(v) & 0x7FFFFFFFu); }

// Two floats as bfloat16 (round to nearest even; NaN stays NaN), first low.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return f32_to_bf16_rne(a) | (f32_to_bf16_rne(b) << 16);
}

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// Eight e4m3 values (two dwords) as bf16, exactly.
__device__ __forceinline__ v8bf widen8(uint32_t a, uint32_t b) {
  union {
    v2bf p[4];
    v8bf v;
  } u;
  u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return u.v;
}

}  // namespace moe
