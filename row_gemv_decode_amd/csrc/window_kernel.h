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

// weights of a window kernel (WQ): the rows' own 16-bit type, or 4-bit codes in
// groups of 32, 64 or 128, plus kZeros when the weight has zero points
constexpr int kWFull = 0;
constexpr int kZeros = 1;
template <int WQ>
constexpr int group_len() { return WQ & ~kZeros; }

// blocks of 32 in a unit, a wave's step along k: 64 bytes of codes or 128 bytes
// of 16-bit weights of each column
template <int WQ>
constexpr int unit_blocks() { return WQ == kWFull ? 2 : 4; }
template <int WQ>
constexpr int unit_len() { return 32 * unit_blocks<WQ>(); }

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

// The two constants of codes16 where one instruction can take both: the mask
// in a scalar register, the base in a vector register (a VOP3 instruction here
// takes one scalar operand and no literal; with both as literals the compiler
// needs an and and an or).
struct CodeBits {
  uint32_t mask, base;
};
template <int TK>
__device__ __forceinline__ CodeBits code_bits() {
  CodeBits c = {TK == CK_F16 ? 0x03C003C0u : 0x00780078u, TK == CK_F16 ? 0x4C004C00u : 0x41804180u};
  asm("" : "+s"(c.mask), "+v"(c.base));
  return c;
}

// eight codes of one dword as 16 + q, in the pair order (0,4) (1,5) (2,6) (3,7)
template <int TK>
__device__ __forceinline__ u32x4 codes16(uint32_t w, const CodeBits& c) {
  constexpr int top = TK == CK_F16 ? 6 : 3;  // where the code's low bit goes
  u32x4 b;
  b[0] = ((w << top) & c.mask) | c.base;
  b[1] = ((TK == CK_F16 ? w << 2 : w >> 1) & c.mask) | c.base;
  b[2] = ((w >> (8 - top)) & c.mask) | c.base;
  b[3] = ((w >> (12 - top)) & c.mask) | c.base;
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

// ---------------------------------------------------------------------------
// A weight matrix as a wave sees it: CT tiles of 16 consecutive columns, each
// from a wave-uniform address, and one 32-bit offset per lane that serves all
// tiles (column l & 15 of a tile, block or elements of lane group h).
// Loads are plain: two units share a cache line of every column, and a
// non-temporal load gives the line's other half up (measured 5 to 20 % slower).
// ---------------------------------------------------------------------------
template <int WQ, int CT>
struct WTiles {
  const char* codes[CT];   // first column, k = 0 (16-bit weights or codes)
  const char* scales[CT];
  const char* zeros[CT];   // kZeros only
  uint32_t off;            // lane's byte offset into codes
  uint32_t col_groups;     // (l & 15) * groups per column
  int groups;              // per column
};

// tile c starts at column j[c] of a weight of row length k; cols: columns of a
// tile that exist (lanes past them read the last one, their sums are not stored)
template <int WQ, int CT>
__device__ __forceinline__ void w_tiles(WTiles<WQ, CT>& t, const WindowWeight& w, const int64_t (&j)[CT], int64_t k, int cols,
                                        int lane) {
  const int h = lane >> 4;
  const int col = min(lane & 15, cols - 1);
  if constexpr (WQ == kWFull) {
#pragma unroll
    for (int c = 0; c < CT; ++c) t.codes[c] = (const char*)w.codes + j[c] * k * 2;
    t.off = (uint32_t)col * (uint32_t)(k * 2) + 16 * h;
  } else {
    t.groups = (int)(k / group_len<WQ>());
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      t.codes[c] = (const char*)w.codes + j[c] * (k >> 1);
      t.scales[c] = (const char*)w.scales + j[c] * t.groups * 2;
      t.zeros[c] = (const char*)w.zeros + ((WQ & kZeros) != 0 ? j[c] * t.groups : 0);
    }
    t.off = (uint32_t)col * (uint32_t)(k >> 1) + 16 * h;
    t.col_groups = (uint32_t)(col * t.groups);
  }
}

// loaded, not yet decoded weights of one unit
template <int WQ, int CT>
struct WUnit {
  u32x4 v[CT][WQ == kWFull ? 2 : 1];
};

// Load unit u.  kPart: the last unit of a k that is no multiple of the unit
// (k is one of 32): blocks past k are not read.
template <int WQ, int CT, bool kPart>
__device__ __forceinline__ void load_w(WUnit<WQ, CT>& r, const WTiles<WQ, CT>& t, int u, int k, int h) {
  if constexpr (WQ == kWFull) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (!kPart || u * 64 + 32 * i < k) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
          r.v[c][i] = *(const u32x4*)(t.codes[c] + (int64_t)u * 128 + t.off + 64 * i);
      }
  } else {
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (kPart) r.v[c][0] = u32x4{0u, 0u, 0u, 0u};
      if (!kPart || u * 128 + 32 * h < k)
        r.v[c][0] = *(const u32x4*)(t.codes[c] + (int64_t)u * 64 + t.off);
    }
  }
}

// The scale (low half) and zero point (high half) of group g of the lane's
// column; g is clamped to the column's groups.
template <int WQ, int CT>
struct ScaleRaw {
  uint16_t s[CT];
  uint8_t z[CT];
};
template <int WQ, int CT>
__device__ __forceinline__ void load_scale(ScaleRaw<WQ, CT>& r, const WTiles<WQ, CT>& t, int g) {
  const uint32_t at = t.col_groups + (uint32_t)min(g, t.groups - 1);
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    r.s[c] = *(const uint16_t*)(t.scales[c] + 2 * at);
    r.z[c] = 8;
    if constexpr ((WQ & kZeros) != 0) r.z[c] = *(const uint8_t*)(t.zeros[c] + at);
  }
}

// what lane groups 0, 1, 2, 3 hold of `own`, in every lane
__device__ __forceinline__ u32x4 spread4(uint32_t own) {
  auto s = __builtin_amdgcn_permlane32_swap(own, own, false, false);
  auto lo = __builtin_amdgcn_permlane16_swap(s[0], s[0], false, false);
  auto hi = __builtin_amdgcn_permlane16_swap(s[1], s[1], false, false);
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// A's fragments of unit u from a row of 16-bit values.  `base` is the lane's
// row at element 8h (or, for groups of 128, 32h: there a step of the matrix
// core takes eight codes of each of the four blocks, so no exchange is needed).
template <int WQ>
constexpr int a_step() { return group_len<WQ>() == 128 ? 8 : 32; }   // elements from one fragment to the next
template <int WQ>
constexpr int a_group() { return group_len<WQ>() == 128 ? 32 : 8; }  // elements from one lane group to the next

template <int WQ, bool kPart>
__device__ __forceinline__ void load_a(u32x4 (&a)[unit_blocks<WQ>()], const uint16_t* base, int u, int k) {
#pragma unroll
  for (int i = 0; i < unit_blocks<WQ>(); ++i)
    if (!kPart || u * unit_len<WQ>() + 32 * i < k)
      a[i] = *(const u32x4*)(base + (int64_t)u * unit_len<WQ>() + a_step<WQ>() * i);
}

// tot[c] += A(unit) . W(unit) for CT column tiles; A is the sum of NP planes
// (kOrdered: their elements are in pair order already).  sz[c][g]: scale and
// zero point of the unit's group g.
template <int TK, int WQ, int CT, int NP, bool kOrdered, bool kPart>
__device__ __forceinline__ void mul_unit(const WUnit<WQ, CT>& w, const u32x4 (&sz)[CT],
                                         const u32x4 (&a)[NP][unit_blocks<WQ>()], f32x4 (&tot)[CT], int u, int k) {
  if constexpr (WQ == kWFull) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (kPart && u * 64 + 32 * i >= k) break;
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int c = 0; c < CT; ++c) tot[c] = mfma16<TK>(a[p][i], w.v[c][i], tot[c]);
    }
  } else {
    constexpr int NB = group_len<WQ>() / 32;  // blocks per group
    const CodeBits bits = code_bits<TK>();
    u32x4 q[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) q[c] = NB == 4 ? w.v[c][0] : exchange4(w.v[c][0]);
    constexpr uint32_t one = TK == CK_F16 ? 0x3C003C00u : 0x3F803F80u;
    const u32x4 ones = {one, one, one, one};
#pragma unroll
    for (int g = 0; g < 4 / NB; ++g) {
      if (kPart && u * 128 + 32 * g * NB >= k) break;
      f32x4 sa = {0.0f, 0.0f, 0.0f, 0.0f};
      f32x4 acc[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = g * NB; i < g * NB + NB; ++i) {
        u32x4 ap[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          ap[p] = kOrdered ? a[p][i] : pair_order(a[p][i]);
          sa = mfma16<TK>(ap[p], ones, sa);
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const uint32_t qi = q[c][i];
          const u32x4 b = codes16<TK>(qi, bits);
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
      // group by group, which takes fewer registers
      if constexpr (NB != 4) __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Scales of the two units u and u + 1.  A lane group holds one group's: of
// groups of 64 and 128 one load fetches both units' (and is issued a pair
// ahead), of groups of 32 each unit has a load of its own.
template <int WQ, int CT>
struct PairScales {
  ScaleRaw<WQ, CT> r[group_len<WQ>() == 32 ? 2 : 1];
};
// with the pair: both units' scales
template <int WQ, int CT>
__device__ __forceinline__ void load_pair_scales(PairScales<WQ, CT>& p, const WTiles<WQ, CT>& t, int u, int h) {
  if constexpr (group_len<WQ>() == 128) {
    load_scale(p.r[0], t, u + (h >> 1));
  } else if constexpr (group_len<WQ>() == 64) {
    load_scale(p.r[0], t, 2 * u + h);
  }
}
// with each unit: unit u as the first or second of its pair
template <int WQ, int CT>
__device__ __forceinline__ void load_unit_scales(PairScales<WQ, CT>& p, const WTiles<WQ, CT>& t, int u, int second, int h) {
  if constexpr (group_len<WQ>() == 32) load_scale(p.r[second], t, 4 * u + h);
}
// unit `second` (0 or 1) of the pair
template <int WQ, int CT>
__device__ __forceinline__ void unit_scales(u32x4 (&sz)[CT], const PairScales<WQ, CT>& p, int second) {
  if constexpr (WQ != kWFull) {
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const ScaleRaw<WQ, CT>& r = p.r[group_len<WQ>() == 32 ? second : 0];
      const uint32_t own = (uint32_t)r.s[c] | ((uint32_t)r.z[c] << 16);
      if constexpr (group_len<WQ>() == 128) {
        auto s = __builtin_amdgcn_permlane32_swap(own, own, false, false);
        sz[c][0] = s[second];
      } else {
        const u32x4 s = spread4(own);
        sz[c][0] = s[group_len<WQ>() == 64 ? 2 * second : 0];
        sz[c][1] = s[group_len<WQ>() == 64 ? 2 * second + 1 : 1];
        sz[c][2] = s[2];
        sz[c][3] = s[3];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// tot[c] += A . W over the units first .. first + n - 1 of k, and over the
// partial unit `part` (negative: none).  Two units are in flight: each is
// loaded again, two units on, as soon as it is used, so a wave always has
// about CT x 4 KiB of loads under way, and loads are never issued under a
// condition in the loop (a conditional load makes the compiler wait for more
// than it needs).
// ---------------------------------------------------------------------------
template <int TK, int WQ, int CT>
__device__ __forceinline__ void stream_units(f32x4 (&tot)[CT], const WTiles<WQ, CT>& t, const uint16_t* arow, int first,
                                             int n, int part, int k, int h) {
  constexpr int NB = unit_blocks<WQ>();
  if (n > 0) {
    WUnit<WQ, CT> w0, w1;
    u32x4 a0[1][NB], a1[1][NB], sz[CT];
    PairScales<WQ, CT> s, sn;
    int u = first;
    // unit v into the first or second of the two buffers
    auto load0 = [&](int v) __attribute__((always_inline)) {
      load_unit_scales(s, t, v, 0, h);
      load_w<WQ, CT, false>(w0, t, v, k, h);
      load_a<WQ, false>(a0[0], arow, v, k);
    };
    auto load1 = [&](int v) __attribute__((always_inline)) {
      load_unit_scales(s, t, v, 1, h);
      load_w<WQ, CT, false>(w1, t, v, k, h);
      load_a<WQ, false>(a1[0], arow, v, k);
    };
    load_pair_scales(s, t, u, h);
    load0(u);
    load1(n > 1 ? u + 1 : u);
    int left = n;
#pragma unroll 1
    while (left >= 4) {
      load_pair_scales(sn, t, u + 2, h);
      __builtin_amdgcn_sched_barrier(0);
      unit_scales(sz, s, 0);
      mul_unit<TK, WQ, CT, 1, false, false>(w0, sz, a0, tot, u, k);
      __builtin_amdgcn_sched_barrier(0);  // used up before it is loaded again: same registers, no copies
      load0(u + 2);
      __builtin_amdgcn_sched_barrier(0);
      unit_scales(sz, s, 1);
      mul_unit<TK, WQ, CT, 1, false, false>(w1, sz, a1, tot, u + 1, k);
      __builtin_amdgcn_sched_barrier(0);
      load1(u + 3);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (group_len<WQ>() != 32) s = sn;
      u += 2;
      left -= 2;
    }
    __builtin_amdgcn_sched_barrier(0);
    unit_scales(sz, s, 0);
    mul_unit<TK, WQ, CT, 1, false, false>(w0, sz, a0, tot, u, k);
    if (left == 3) {
      load_pair_scales(sn, t, u + 2, h);
      load0(u + 2);
    }
    if (left >= 2) {
      unit_scales(sz, s, 1);
      mul_unit<TK, WQ, CT, 1, false, false>(w1, sz, a1, tot, u + 1, k);
    }
    if (left == 3) {
      if constexpr (group_len<WQ>() == 32) {
        unit_scales(sz, s, 0);
      } else {
        unit_scales(sz, sn, 0);
      }
      mul_unit<TK, WQ, CT, 1, false, false>(w0, sz, a0, tot, u + 2, k);
    }
  }
  if (part >= 0) {
    WUnit<WQ, CT> w;
    u32x4 a[1][NB], sz[CT];
    PairScales<WQ, CT> s;
    load_pair_scales(s, t, part, h);
    load_unit_scales(s, t, part, 0, h);
    load_w<WQ, CT, true>(w, t, part, k, h);
    load_a<WQ, true>(a[0], arow, part, k);
    unit_scales(sz, s, 0);
    mul_unit<TK, WQ, CT, 1, false, true>(w, sz, a, tot, part, k);
  }
}

// how NW waves share k: wave w takes the full units first .. first + n - 1 and
// perhaps the partial one; depends on k alone
struct WaveShare {
  int first, n, part;
};
template <int WQ, int NW>
__device__ __forceinline__ WaveShare wave_share(int k, int wave) {
  const int full = k / unit_len<WQ>();
  const int all = (k + unit_len<WQ>() - 1) / unit_len<WQ>();
  const int per = (all + NW - 1) / NW;
  const int first = min(wave * per, full);
  const int last = min(wave * per + per, full);
  return {first, last - first, all > full && full / per == wave ? full : -1};
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
