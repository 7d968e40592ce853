// window_kernel.h -- the matrix-core inner step of the decode window's 4-bit
// GEMV (w4.hip) and MoE layer (moe.hip), for gfx950 (MI355X).
//
// One wave multiplies 16 rows of A (the window's tokens) by tiles of 16 weight
// columns, k in units of 128, on v_mfma_f32_16x16x32_{f16,bf16}: lane l holds
// row (or column) l & 15 and, with h = l >> 4, the eight elements 8h .. 8h + 7
// of each block of 32; of the 16 x 16 result it holds column l & 15, rows
// 4h .. 4h + 3.  All 16 rows cost the same as one, and a row's sums do not
// depend on the other rows, so row i of any window equals the one-row call bit
// for bit.  A weight is read once for the whole window, straight from HBM to
// registers: no weight is used by two waves, so LDS would only add a copy.
//
// 4-bit weights (one scale, and optionally one zero point, per group of G
// elements along k; W = s * (q - z)):
//   * Lane (column, h) loads 16 bytes, the 32 codes of block h of its unit:
//     one wave load covers 16 columns x 64 bytes.  A 4 x 4 exchange between
//     the four lane groups and the four registers (two v_permlane32_swap, two
//     v_permlane16_swap) then gives every lane group its eight codes of each
//     block, so one MFMA sees one block of 32, hence one scale per column.
//   * A code becomes the exact 16-bit float 16 + q by placing its four bits at
//     the top of 16.0's mantissa: a shift and an and-or per pair of codes, no
//     conversion.  The pairs that fall out of a dword are codes (0,4), (1,5),
//     (2,6), (3,7); A's eight elements are permuted alike (four v_perm, shared
//     by all columns of the wave).
//   * Over one group the matrix core sums acc = sum (16 + q) a and, with a
//     constant 1 as weight, sa = sum a, both exact products added in fp32; the
//     group's contribution is s * (acc - (16 + z) * sa) in fp32.  So no weight
//     is rounded, and the correction costs one MFMA per block for all columns.
//     Against subtracting the zero point from every code this takes one VALU
//     instruction per weight instead of two or more.
#pragma once

#include "device_common.h"
#include "window.h"

namespace skinny {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// weights of a window kernel: the rows' own 16-bit type, or 4-bit codes in
// groups of 32, 64 or 128
constexpr int kWFull = 0;

constexpr int kUnit = 128;  // elements of k per step

template <int TK>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (TK == CK_F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, a), __builtin_bit_cast(h8_t, b), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8_t, a), __builtin_bit_cast(b8_t, b), c, 0, 0,
                                                   0);
  }
}

template <int TK>
__device__ __forceinline__ float half_f32(uint16_t bits) {
  if constexpr (TK == CK_F16) {
    return (float)half_from_bits(bits);
  } else {
    return f32_from_bits((uint32_t)bits << 16);
  }
}

template <int TK>
__device__ __forceinline__ uint16_t f32_half(float v) {  // round to nearest even
  if constexpr (TK == CK_F16) {
    return __builtin_bit_cast(uint16_t, (_Float16)v);
  } else {
    return __builtin_bit_cast(uint16_t, (__bf16)v);
  }
}

// eight codes of one dword as 16 + q, in the pair order (0,4) (1,5) (2,6) (3,7)
template <int TK>
__device__ __forceinline__ u32x4 codes16(uint32_t w) {
  constexpr uint32_t base = TK == CK_F16 ? 0x4C004C00u : 0x41804180u;
  constexpr uint32_t mask = TK == CK_F16 ? 0x03C003C0u : 0x00780078u;
  constexpr int top = TK == CK_F16 ? 6 : 3;  // where the code's low bit goes
  u32x4 b;
  b[0] = ((w << top) & mask) | base;
  b[1] = (TK == CK_F16 ? (w << 2) & mask : (w >> 1) & mask) | base;
  b[2] = ((w >> (8 - top)) & mask) | base;
  b[3] = ((w >> (12 - top)) & mask) | base;
  return b;
}

// A's eight consecutive elements in the same pair order
__device__ __forceinline__ u32x4 pair_order(u32x4 a) {
  const uint32_t a0 = a[0], a1 = a[1], a2 = a[2], a3 = a[3];
  u32x4 p;
  p[0] = __builtin_amdgcn_perm(a2, a0, 0x05040100u);
  p[1] = __builtin_amdgcn_perm(a2, a0, 0x07060302u);
  p[2] = __builtin_amdgcn_perm(a3, a1, 0x05040100u);
  p[3] = __builtin_amdgcn_perm(a3, a1, 0x07060302u);
  return p;
}

// register i of lane group h  <->  register h of lane group i
__device__ __forceinline__ u32x4 exchange4(u32x4 v) {
  auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

// One lane's view of a weight matrix [n][k]: its column's row of codes (or
// 16-bit weights), scales and zero points.  WQ: kWFull, or the group length.
template <int WQ>
struct WCol {
  const uint8_t* codes;    // this column's codes, at block h of unit 0
  const uint16_t* scales;  // [k / WQ]
  const uint8_t* zeros;    // [k / WQ], or null: 8 everywhere
};
template <>
struct WCol<kWFull> {
  const uint16_t* w;  // this column's weights, at element 8h of unit 0
};

template <int WQ>
__device__ __forceinline__ WCol<WQ> w_col(const void* codes, const void* scales, const void* zeros, int64_t j,
                                          int64_t k, int h) {
  WCol<WQ> c;
  if constexpr (WQ == kWFull) {
    c.w = (const uint16_t*)codes + j * k + 8 * h;
  } else {
    c.codes = (const uint8_t*)codes + j * (k >> 1) + 16 * h;
    c.scales = (const uint16_t*)scales + j * (k / WQ);
    c.zeros = zeros == nullptr ? nullptr : (const uint8_t*)zeros + j * (k / WQ);
  }
  return c;
}

// The loaded, not yet decoded weights of one (column, unit)
template <int WQ>
struct WRaw {
  u32x4 codes;
  uint16_t scale;  // of lane group h's block
  uint8_t zero;
};
template <>
struct WRaw<kWFull> {
  u32x4 w[4];
};

// Load unit u.  kPart: the last unit of a k that is no multiple of 128 (k is
// one of 32): blocks past k are not read.
template <int WQ, bool kPart>
__device__ __forceinline__ void load_unit(WRaw<WQ>& r, const WCol<WQ>& c, int u, int k, int h) {
  if constexpr (WQ == kWFull) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!kPart || u * kUnit + 32 * i < k)
        r.w[i] = __builtin_nontemporal_load((const u32x4*)(c.w + (int64_t)u * kUnit + 32 * i));
  } else {
    const int kk = u * kUnit + 32 * h;  // this lane group's block
    const bool in = !kPart || kk < k;
    r.codes = u32x4{0u, 0u, 0u, 0u};
    r.scale = 0;
    r.zero = 8;
    if (in) {
      r.codes = __builtin_nontemporal_load((const u32x4*)(c.codes + (int64_t)u * (kUnit / 2)));
      r.scale = c.scales[kk / WQ];
      if (c.zeros != nullptr) r.zero = c.zeros[kk / WQ];
    }
  }
}

// A's four fragments of unit u from a row of 16-bit values (base: element 8h
// of the lane's row); kPart as above, blocks past k stay unset and unused
template <bool kPart>
__device__ __forceinline__ void load_a_unit(u32x4 (&a)[4], const uint16_t* base, int u, int k) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!kPart || u * kUnit + 32 * i < k) a[i] = *(const u32x4*)(base + (int64_t)u * kUnit + 32 * i);
}

// tot[c] += A(unit) . W(unit) for CT column tiles; A is the sum of NP planes.
template <int TK, int WQ, int CT, int NP, bool kPart>
__device__ __forceinline__ void mul_unit(const WRaw<WQ> (&w)[CT], const u32x4 (&a)[NP][4], f32x4 (&tot)[CT], int u,
                                         int k) {
  if constexpr (WQ == kWFull) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kPart && u * kUnit + 32 * i >= k) break;
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int c = 0; c < CT; ++c) tot[c] = mfma16<TK>(a[p][i], w[c].w[i], tot[c]);
    }
  } else {
    constexpr int NB = WQ / 32;  // blocks per group
    u32x4 q[CT], sz[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      q[c] = exchange4(w[c].codes);
      // every lane needs the scale (and zero) of each group of the unit: lane
      // group h loaded those of block h, swaps broadcast them
      const uint32_t own = (uint32_t)w[c].scale | ((uint32_t)w[c].zero << 16);
      if constexpr (NB == 4) {
        sz[c][0] = own;
      } else if constexpr (NB == 2) {
        auto s = __builtin_amdgcn_permlane32_swap(own, own, false, false);
        sz[c][0] = s[0];
        sz[c][1] = s[1];
      } else {
        auto s = __builtin_amdgcn_permlane32_swap(own, own, false, false);
        auto lo = __builtin_amdgcn_permlane16_swap(s[0], s[0], false, false);
        auto hi = __builtin_amdgcn_permlane16_swap(s[1], s[1], false, false);
        sz[c] = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    }
    constexpr uint32_t one = TK == CK_F16 ? 0x3C003C00u : 0x3F803F80u;
    const u32x4 ones = {one, one, one, one};
#pragma unroll
    for (int g = 0; g < 4 / NB; ++g) {
      if (kPart && u * kUnit + 32 * g * NB >= k) break;
      f32x4 sa = {0.0f, 0.0f, 0.0f, 0.0f};
      f32x4 acc[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = g * NB; i < g * NB + NB; ++i) {
        u32x4 ap[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          ap[p] = pair_order(a[p][i]);
          sa = mfma16<TK>(ap[p], ones, sa);
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const uint32_t qi = q[c][i];
          const u32x4 b = codes16<TK>(qi);
#pragma unroll
          for (int p = 0; p < NP; ++p) acc[c] = mfma16<TK>(ap[p], b, acc[c]);
        }
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const uint32_t szg = sz[c][g];
        const float s = half_f32<TK>((uint16_t)(szg & 0xffffu));
        const float z = -16.0f - (float)(szg >> 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) tot[c][e] = __builtin_fmaf(s, __builtin_fmaf(z, sa[e], acc[c][e]), tot[c][e]);
      }
    }
  }
}

// store one fp32 value as the output kind (uniform runtime kind)
__device__ __forceinline__ void store_kind(void* base, int64_t idx, float v, int kind) {
  if (kind == CK_F32) {
    ((float*)base)[idx] = v;
  } else if (kind == CK_F16) {
    ((_Float16*)base)[idx] = (_Float16)v;
  } else {
    ((__bf16*)base)[idx] = (__bf16)v;
  }
}

}  // namespace

}  // namespace skinny
