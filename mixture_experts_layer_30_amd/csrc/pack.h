// Blocks of 32 values in 8 bits: e4m3 codes with a power of two as the block's scale.
//
// The scale is the least 2^e with max |v| <= 448 * 2^e (448 is the largest e4m3 value), at
// least 2^-127, kept as the byte e + 127.  A power of two divides exactly, so a value is
// rounded once, to the nearest e4m3 value (half a step: 2^-4 of it), and the codes are the
// same however the division is done.  With 448 = 1.75 * 2^8 and max |v| = 1.m * 2^k, e is
// k - 8, and one more where 1.m > 1.75: integer operations on the bits of the maximum.
// A value that is not finite becomes NaN and has no part in the maximum.
#pragma once

#include "rows.h"

namespace moe {

// max(m, |v|), without the values that are not finite
__device__ __forceinline__ float abs_max(float m, float v) {
  const float a = fabsf(v);
  return a < __builtin_inff() ? fmaxf(m, a) : m;
}

__device__ __forceinline__ int scale_byte(float most) {
  const int b = (int)__float_as_uint(most);
  const int e = (b >> 23) - 8 + ((b & 0x7fffff) > 0x600000 ? 1 : 0);
  return e > 0 ? e : 0;
}

// 1 / scale, for the bytes that scale_byte gives (0 .. 247)
__device__ __forceinline__ float inverse_scale(int byte) {
  return __uint_as_float((uint32_t)(254 - byte) << 23);
}

__device__ __forceinline__ float scale_of(int byte) {
  return __uint_as_float(byte ? (uint32_t)byte << 23 : 0x00400000u);   // 2^-127 is subnormal
}

// 8 values as codes (code j in byte j)
__device__ __forceinline__ uint2 pack_e4m3x8(const float* v, float inv) {
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    q[j] = fabsf(v[j]) < __builtin_inff() ? v[j] * inv : __builtin_nanf("");
  uint2 r;
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  r.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  r.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], w, true);
  return r;
}

__device__ __forceinline__ void unpack_e4m3x8(uint2 c, float scale, float* v) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true);
  const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false);
  const f32x2 e = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true);
  v[0] = a.x * scale; v[1] = a.y * scale; v[2] = b.x * scale; v[3] = b.y * scale;
  v[4] = d.x * scale; v[5] = d.y * scale; v[6] = e.x * scale; v[7] = e.y * scale;
}

// the largest over a quad of lanes
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kQuadXor1, 0xF, 0xF, false)));
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kQuadXor2, 0xF, 0xF, false)));
}

}  // namespace moe
