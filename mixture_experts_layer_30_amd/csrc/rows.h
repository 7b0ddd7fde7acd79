// Loads and stores of 8 neighbours of a row, and sums across a wavefront's lanes.
#pragma once

#include "common.h"

namespace moe {

// 8 consecutive elements as fp32 (p 16-byte aligned)
template <class S>
__device__ __forceinline__ void load8f(const typename S::T* p, float* v);
template <>
__device__ __forceinline__ void load8f<BF16>(const uint16_t* p, float* v) {
  const u32x4 r = *reinterpret_cast<const u32x4*>(p);
  const uint32_t q[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(q[j] << 16);
    v[2 * j + 1] = __uint_as_float(q[j] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8f<F32>(const float* p, float* v) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0];
  const f32x4 b = reinterpret_cast<const f32x4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

template <class S>
__device__ __forceinline__ void store8f(typename S::T* p, const float* v);
template <>
__device__ __forceinline__ void store8f<BF16>(uint16_t* p, const float* v) {
  u32x4 r;
  r.x = pack_bf16x2(v[0], v[1]);
  r.y = pack_bf16x2(v[2], v[3]);
  r.z = pack_bf16x2(v[4], v[5]);
  r.w = pack_bf16x2(v[6], v[7]);
  *reinterpret_cast<u32x4*>(p) = r;
}
template <>
__device__ __forceinline__ void store8f<F32>(float* p, const float* v) {
  reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
  reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
}

// DPP controls (gfx9 encoding): quad permutations and row mirrors
constexpr int kQuadXor1 = 0xB1;     // quad_perm [1,0,3,2]
constexpr int kQuadXor2 = 0x4E;     // quad_perm [2,3,0,1]
constexpr int kRowHalfMirror = 0x141;
constexpr int kRowMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false);
  return v + __int_as_float(o);
}

// Sum of v over the wavefront, in every lane (every lane active).
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<kQuadXor1>(v);
  v = dpp_add<kQuadXor2>(v);
  v = dpp_add<kRowHalfMirror>(v);
  v = dpp_add<kRowMirror>(v);
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
  const float r1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
  const float r2 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32));
  const float r3 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
  return (r0 + r1) + (r2 + r3);
}

}  // namespace moe
