// Block-128 e4m3 quantisation shared by the kernels that write 8-bit rows.
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

// Four quotients v[i] / scale (IEEE division) of float32 values as e4m3fn
// bytes, little end first, rounded to nearest even and saturated.  Zero bytes
// where the scale is 0.
//
// v_cvt_pk_fp8_f32 rounds what is up to 464 to 448 and turns all above into
// NaN.  Quotients pass 448 by a rounding where the scale is a normal number,
// and by up to a half where it is a subnormal one of few bits: only those are
// held to 448 (a select for every value took 2% of the norm's time).
__device__ __forceinline__ uint32_t quant4_scaled(const float* v, float scale) {
  if (scale == 0.0f) return 0u;
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = v[i] / scale;
  if (__builtin_expect(scale < 0x1p-126f, 0)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = fminf(fmaxf(q[i], -448.0f), 448.0f);
  }
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
  return (uint32_t)w;
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
