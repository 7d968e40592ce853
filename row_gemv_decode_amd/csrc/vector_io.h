// vector_io.h -- loads and stores of a few consecutive values from and to rows
// that start at any element, shared by the kernels of a batch of requests
// (gfx950).  Global accesses of 8 and 16 bytes take any alignment here, so a
// vector's place in its row never depends on where the row lies.
#pragma once

#include "device_common.h"

namespace skinny {

namespace {

typedef uint32_t u32x4_align4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_align2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_align4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32x2_align2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x2_align1 __attribute__((ext_vector_type(2), aligned(1)));

// Workgroup `index` of `count` in an order in which the workgroups that share an XCD
// (every eighth one), and with it an L2, have consecutive places.
__device__ __forceinline__ uint32_t xcd_place(uint32_t index, uint32_t count) {
  const uint32_t xcd = index & 7, most = count >> 3, more = count & 7;
  return xcd * most + min(xcd, more) + (index >> 3);
}

template <int K>
constexpr int kind_size() { return K == CK_F32 ? 4 : 2; }

__device__ __forceinline__ int kind_bytes(int kind) { return kind == CK_F32 ? 4 : 2; }

template <int K>
__device__ __forceinline__ float value_at(const void* p, int64_t i) {
  if constexpr (K == CK_F32) {
    return ((const float*)p)[i];
  } else if constexpr (K == CK_F16) {
    return (float)((const _Float16*)p)[i];
  } else {
    return f32_from_bits((uint32_t)((const uint16_t*)p)[i] << 16);
  }
}

// the stored bits of N values (4 or 8): dwords in memory order.  (A vector, not an
// array: arrays of these that are copied as a whole ended up in scratch memory.)
template <int K, int N>
struct Raw {
  static constexpr int kWords = N * kind_size<K>() / 4;
  uint32_t w __attribute__((ext_vector_type(kWords)));
};

template <int K, int N>
__device__ __forceinline__ Raw<K, N> load_raw(const void* p, int64_t i) {
  Raw<K, N> r;
  constexpr int W = Raw<K, N>::kWords;
  const char* at = (const char*)p + i * kind_size<K>();
  if constexpr (W == 2) {
    const u32x2 v = *(const u32x2_align2*)at;
    r.w[0] = v[0], r.w[1] = v[1];
  } else {
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
      u32x4 v;
      if constexpr (K == CK_F32) {
        v = *(const u32x4_align4*)(at + 16 * q);
      } else {
        v = *(const u32x4_align2*)(at + 16 * q);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) r.w[4 * q + e] = v[e];
    }
  }
  return r;
}

template <int K, int N>
__device__ __forceinline__ void unpack_raw(const Raw<K, N>& r, float (&x)[N]) {
#pragma unroll
  for (int q = 0; q < Raw<K, N>::kWords; ++q) {
    const uint32_t w = r.w[q];
    if constexpr (K == CK_F32) {
      x[q] = f32_from_bits(w);
    } else if constexpr (K == CK_F16) {
      const h2_t hh = as_h2(w);
      x[2 * q] = (float)hh[0];
      x[2 * q + 1] = (float)hh[1];
    } else {
      x[2 * q] = f32_from_bits(w << 16);
      x[2 * q + 1] = f32_from_bits(w & 0xffff0000u);
    }
  }
}

// two values in a dword of a 16-bit type, rounded to nearest even
template <int K>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (K == CK_F16) {
    const h2_t v = {(_Float16)a, (_Float16)b};
    return h2_bits(v);
  } else {
    const b2_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
}

// STREAM: past the caches' replacement order.  What a launch writes, the next one
// mostly reads on another XCD, so nothing is gained by keeping it; rows that start in
// the middle of a cache line gain most (2000 x 7681 norm 33.1 -> 24.1 us).
template <bool STREAM>
__device__ __forceinline__ void put8(u32x2 v, char* at) {
  if constexpr (STREAM) {
    __builtin_nontemporal_store(v, (u32x2_align1*)at);
  } else {
    *(u32x2_align1*)at = v;
  }
}
template <bool STREAM>
__device__ __forceinline__ void put16(u32x4 v, char* at) {
  if constexpr (STREAM) {
    __builtin_nontemporal_store(v, (u32x4_align2*)at);
  } else {
    *(u32x4_align2*)at = v;
  }
}

template <int K, int N, bool STREAM = false>
__device__ __forceinline__ void store_vec(void* p, int64_t i, const float (&x)[N]) {
  char* at = (char*)p + i * kind_size<K>();
  if constexpr (K == CK_F32) {
#pragma unroll
    for (int q = 0; q < N / 4; ++q)
      put16<STREAM>(u32x4{__builtin_bit_cast(uint32_t, x[4 * q]), __builtin_bit_cast(uint32_t, x[4 * q + 1]),
                          __builtin_bit_cast(uint32_t, x[4 * q + 2]), __builtin_bit_cast(uint32_t, x[4 * q + 3])},
                    at + 16 * q);
  } else if constexpr (N == 4) {
    put8<STREAM>(u32x2{pack2<K>(x[0], x[1]), pack2<K>(x[2], x[3])}, at);
  } else {
#pragma unroll
    for (int q = 0; q < N / 8; ++q)
      put16<STREAM>(u32x4{pack2<K>(x[8 * q], x[8 * q + 1]), pack2<K>(x[8 * q + 2], x[8 * q + 3]),
                          pack2<K>(x[8 * q + 4], x[8 * q + 5]), pack2<K>(x[8 * q + 6], x[8 * q + 7])},
                    at + 16 * q);
  }
}

}  // namespace

}  // namespace skinny
