// wave_ops.h -- reductions over the 64 lanes of a wavefront by DPP and
// permlane exchanges, and the order keys of a top-k, shared by the library's
// kernels (gfx950).
#pragma once

#include "device_common.h"

namespace skinny {

namespace {

__device__ __forceinline__ float fbits(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t ubits(float f) { return __builtin_bit_cast(uint32_t, f); }

template <int CTRL>
__device__ __forceinline__ float dpp_mov(float x) {
  return fbits(__builtin_amdgcn_update_dpp(0u, ubits(x), CTRL, 0xF, 0xF, false));
}

// DPP controls: row_mirror (l ^ 15 in a row of 16), row_half_mirror (l ^ 7),
// quad_perm [2,3,0,1] (l ^ 2), quad_perm [1,0,3,2] (l ^ 1)
constexpr int kDppRowMirror = 0x140;
constexpr int kDppRowHalfMirror = 0x141;
constexpr int kDppXor2 = 0x4E;
constexpr int kDppXor1 = 0xB1;

// Order keys: the float's bits with the magnitude bits of negative values
// flipped, read as a signed integer, and -0 mapped to +0's key; for non-NaN
// values the key order is IEEE order and equal keys are IEEE-equal values.
__device__ __forceinline__ int order_key(float x) {
  uint32_t b = ubits(x);
  if (b == 0x80000000u) b = 0u;  // -0 ranks with +0
  return (int)(b ^ ((uint32_t)((int)b >> 31) & 0x7fffffffu));
}

// the float whose order key is `key` (-0 comes back as +0)
__device__ __forceinline__ float key_value(int key) {
  return fbits((uint32_t)key ^ ((uint32_t)(key >> 31) & 0x7fffffffu));
}

template <int CTRL>
__device__ __forceinline__ int dpp_mov_i(int x) {
  return (int)__builtin_amdgcn_update_dpp(0u, (uint32_t)x, CTRL, 0xF, 0xF, false);
}

__device__ __forceinline__ int wave_max_i32(int v) {
  v = max(v, dpp_mov_i<kDppXor1>(v));
  v = max(v, dpp_mov_i<kDppXor2>(v));
  v = max(v, dpp_mov_i<kDppRowHalfMirror>(v));
  v = max(v, dpp_mov_i<kDppRowMirror>(v));
  auto r16 = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
  v = max((int)r16[0], (int)r16[1]);
  auto r32 = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
  v = max((int)r32[0], (int)r32[1]);
  return v;
}

__device__ __forceinline__ int wave_min_i32(int v) {
  v = min(v, dpp_mov_i<kDppXor1>(v));
  v = min(v, dpp_mov_i<kDppXor2>(v));
  v = min(v, dpp_mov_i<kDppRowHalfMirror>(v));
  v = min(v, dpp_mov_i<kDppRowMirror>(v));
  auto r16 = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
  v = min((int)r16[0], (int)r16[1]);
  auto r32 = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
  v = min((int)r32[0], (int)r32[1]);
  return v;
}

__device__ __forceinline__ float wave_max_f32(float v) {
  v = fmaxf(v, dpp_mov<kDppXor1>(v));
  v = fmaxf(v, dpp_mov<kDppXor2>(v));
  v = fmaxf(v, dpp_mov<kDppRowHalfMirror>(v));
  v = fmaxf(v, dpp_mov<kDppRowMirror>(v));
  auto r16 = __builtin_amdgcn_permlane16_swap(ubits(v), ubits(v), false, false);
  v = fmaxf(fbits(r16[0]), fbits(r16[1]));
  auto r32 = __builtin_amdgcn_permlane32_swap(ubits(v), ubits(v), false, false);
  return fmaxf(fbits(r32[0]), fbits(r32[1]));
}

__device__ __forceinline__ float wave_sum_f32(float v) {
  v += dpp_mov<kDppXor1>(v);
  v += dpp_mov<kDppXor2>(v);
  v += dpp_mov<kDppRowHalfMirror>(v);
  v += dpp_mov<kDppRowMirror>(v);
  auto r16 = __builtin_amdgcn_permlane16_swap(ubits(v), ubits(v), false, false);
  v = fbits(r16[0]) + fbits(r16[1]);
  auto r32 = __builtin_amdgcn_permlane32_swap(ubits(v), ubits(v), false, false);
  return fbits(r32[0]) + fbits(r32[1]);
}

// order of a wave's LDS writes and its later reads by other lanes (the LDS
// works in order; this keeps the compiler from moving them)
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace

}  // namespace skinny
