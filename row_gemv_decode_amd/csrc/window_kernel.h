// window_kernel.h -- the matrix-core inner step of the decode window's 4-bit
// GEMV (w4.hip) and MoE layer (moe.hip), for gfx950 (MI355X).
//
// One wave multiplies 16 rows of A (the window's tokens) by tiles of 16 weight
// columns, k in units of 128, on v_mfma_f32_16x16x32_{f16,bf16}: lane l holds
// row (or column) l & 15 and, with h = l >> 4, the eight elements 8h .. 8h + 7
// of each block of 32; of the 16 x 16 result it holds column l & 15, rows
// 4h .. 4h + 3.  All 16 rows cost the same as one, and a row's sums do not
// depend on the other rows, so row i of any window equals the one-row call bit
// for bit.  A weight is read once for the whole window, by the wave that
// multiplies it.
//
// 4-bit weights (one scale, and optionally one zero point, per group of G
// elements along k; W = s * (q - z)):
//   * A wave load covers 16 columns x 64 bytes, the codes of one unit; lane
//     (column, h) needs the 16 bytes of block h.  A 4 x 4 exchange between
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
//     Both parts are some 5 times the difference for rows of mean 0, and more for
//     rows with a mean, which costs their sums' roundings no more than 1.5 times
//     the error of an fp32 product (the entry point states the bound).
//     Against subtracting the zero point from every code this takes one VALU
//     instruction per weight instead of two or more.
#pragma once

#include "device_common.h"
#include "wave_ops.h"
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
// Loads and the turn.  The cache combines the accesses of consecutive lanes
// only, so a load gives four consecutive lanes the 64 bytes of one row (a
// column of the weight, or a token): lane l fetches piece l & 3 of row l >> 2.
// The matrix core wants piece l >> 4 of row l & 15 in lane l.  Loading in that
// order makes every lane an access of its own, and the accesses, some 30 for each
// load, were what bounded the kernels (MoE, 16 of 256 experts: the up product
// took 175 us for 137).  So each 1 KiB passes through a slot of
// LDS that belongs to the wave: written as loaded, read as needed, no barrier.
// A row's four pieces are stored rotated by f(row), which keeps the reads (and
// the writes) free of bank conflicts.
// ---------------------------------------------------------------------------
struct Turn {
  u32x4* slots;    // the wave's slots, 64 entries each
  int put, get;    // the lane's entry to write, and to read

  __device__ __forceinline__ Turn(u32x4* wave_slots, int lane) : slots(wave_slots) {
    put = entry(lane >> 2, lane & 3);
    get = entry(lane & 15, lane >> 4);
  }
  static __device__ __forceinline__ int entry(int row, int piece) {
    return row * 4 + (piece ^ ((row >> 1) & 3) ^ (row >> 3));
  }
};

// barrier of a workgroup that shares LDS only: loads from memory stay in flight
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A weight matrix as a wave sees it: CT tiles of 16 consecutive columns, each
// from a wave-uniform address, and one 32-bit offset per lane that serves all
// tiles.  Weight loads are plain: two units share a cache line of every column,
// and a non-temporal load gives the line's other half up (measured 5 to 20 %
// slower).
template <int WQ, int CT>
struct WTiles {
  const char* codes[CT];  // first column, k = 0 (16-bit weights or codes)
  uint32_t off;           // lane's byte offset into codes
};

// tile c starts at column j[c] of a weight of row length k; cols: columns of a
// tile that exist (lanes past them read the last one, their sums are not stored)
template <int WQ, int CT>
__device__ __forceinline__ void w_tiles(WTiles<WQ, CT>& t, const WindowWeight& w, const int64_t (&j)[CT], int64_t k,
                                        int cols, int lane) {
  const uint32_t row = (uint32_t)(WQ == kWFull ? k * 2 : k >> 1);  // bytes of a column
#pragma unroll
  for (int c = 0; c < CT; ++c) t.codes[c] = (const char*)w.codes + j[c] * (int64_t)row;
  t.off = (uint32_t)min(lane >> 2, cols - 1) * row + 16 * (lane & 3);
}

// loaded, not yet turned and decoded weights of one unit
template <int WQ, int CT>
struct WUnit {
  static constexpr int N = WQ == kWFull ? 2 : 1;  // loads per tile
  u32x4 v[CT][N];
};

// Load unit u.  kPart: the last unit of a k that is no multiple of the unit
// (k is one of 32): blocks past k are not read.
template <int WQ, int CT, bool kPart>
__device__ __forceinline__ void load_w(WUnit<WQ, CT>& r, const WTiles<WQ, CT>& t, int u, int k, int lane) {
  if constexpr (WQ == kWFull) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (!kPart || u * 64 + 32 * i < k) {
#pragma unroll
        for (int c = 0; c < CT; ++c) r.v[c][i] = *(const u32x4*)(t.codes[c] + (int64_t)u * 128 + t.off + 64 * i);
      }
  } else {
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (kPart) r.v[c][0] = u32x4{0u, 0u, 0u, 0u};
      if (!kPart || u * 128 + 32 * (lane & 3) < k)
        r.v[c][0] = *(const u32x4*)(t.codes[c] + (int64_t)u * 64 + t.off);
    }
  }
}

// what lane groups 0, 1, 2, 3 hold of `own`, in every lane
__device__ __forceinline__ u32x4 spread4(uint32_t own) {
  auto s = __builtin_amdgcn_permlane32_swap(own, own, false, false);
  auto lo = __builtin_amdgcn_permlane16_swap(s[0], s[0], false, false);
  auto hi = __builtin_amdgcn_permlane16_swap(s[1], s[1], false, false);
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// A's blocks of unit u from a row of 16-bit values; `base` is the lane's row
// (l >> 2) at piece l & 3 of block 0
template <int WQ, bool kPart>
__device__ __forceinline__ void load_a(u32x4 (&a)[unit_blocks<WQ>()], const uint16_t* base, int u, int k) {
#pragma unroll
  for (int i = 0; i < unit_blocks<WQ>(); ++i)
    if (!kPart || u * unit_len<WQ>() + 32 * i < k) a[i] = *(const u32x4*)(base + (int64_t)u * unit_len<WQ>() + 32 * i);
}

// Turn a unit: afterwards w.v and a.v hold, in lane l, piece l >> 4 of row
// l & 15.  For groups of 128 A's fragment i is piece i of block l >> 4
// instead: there a step of the matrix core takes eight codes of each of the
// four blocks, so the codes need no exchange.
template <int WQ, int CT>
constexpr int turn_slots() { return CT * WUnit<WQ, CT>::N + unit_blocks<WQ>(); }

template <int WQ, int CT>
__device__ __forceinline__ void turn_unit(WUnit<WQ, CT>& w, u32x4 (&a)[unit_blocks<WQ>()], const Turn& t, int lane) {
  constexpr int NW = WUnit<WQ, CT>::N, NB = unit_blocks<WQ>();
  wave_lds_order();
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < NW; ++i) t.slots[(c * NW + i) * 64 + t.put] = w.v[c][i];
  u32x4* as = t.slots + CT * NW * 64;
#pragma unroll
  for (int i = 0; i < NB; ++i) as[i * 64 + t.put] = a[i];
  wave_lds_order();
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < NW; ++i) w.v[c][i] = t.slots[(c * NW + i) * 64 + t.get];
#pragma unroll
  for (int i = 0; i < NB; ++i)
    a[i] = group_len<WQ>() == 128 ? as[(lane >> 4) * 64 + Turn::entry(lane & 15, i)] : as[i * 64 + t.get];
}

// tot[c] += A(unit) . W(unit) for CT column tiles (kOrdered: A's elements are in
// pair order already).  sv[c][g], zv[c][g]: the unit's group g's scale and
// -(16 + zero point).
//
// The matrix core's sums are read (and added to tot by vector instructions) in the
// straight line of code that forms them, with no branch between: a read behind a
// branch or a loop's end needs a wait that a listing of an earlier form of these
// kernels did not have on every path.
template <int TK, int WQ, int CT, bool kOrdered, bool kPart>
__device__ __forceinline__ void mul_unit(const WUnit<WQ, CT>& w, const f32x4 (&sv)[CT], const f32x4 (&zv)[CT],
                                         const u32x4 (&a)[unit_blocks<WQ>()], f32x4 (&tot)[CT], int u, int k) {
  if constexpr (WQ == kWFull) {
    f32x4 acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < (kPart ? 1 : 2); ++i)  // (k is a multiple of 32: a partial unit is one block)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[c] = mfma16<TK>(a[i], w.v[c][i], acc[c]);
#pragma unroll
    for (int c = 0; c < CT; ++c) tot[c] += acc[c];
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
        const u32x4 ap = kOrdered ? a[i] : pair_order(a[i]);
        sa = mfma16<TK>(ap, ones, sa);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const uint32_t qi = q[c][i];
          acc[c] = mfma16<TK>(ap, codes16<TK>(qi, bits), acc[c]);
        }
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const float s = sv[c][g], z = zv[c][g];
#pragma unroll
        for (int e = 0; e < 4; ++e) tot[c][e] = __builtin_fmaf(s, __builtin_fmaf(z, sa[e], acc[c][e]), tot[c][e]);
      }
      // group by group, which takes fewer registers
      if constexpr (NB != 4) __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// ---------------------------------------------------------------------------
// A workgroup's scales and zero points, in LDS as the fp32 pairs (s, -(16 + z))
// that the product takes: column by column, `groups` of each, for at most
// kSpanGroups groups at a time.  The 16 columns of a tile lie together in memory,
// so the workgroup fetches them with full 16-byte loads; fetched by the lanes
// that use them, 2 and 1 bytes of 16 columns at a time, they cost the load path
// as much as a third of the codes (16 of 256 experts, groups of 128: 198 us for
// the up product against 165 without any scale).  Converted once here, a pair
// serves every unit without further instructions.
// ---------------------------------------------------------------------------
constexpr int kSpanGroups = 80;  // (four tiles' pairs and the slots of the turn: two workgroups per CU)
typedef float f32x2 __attribute__((ext_vector_type(2)));
template <int WQ, int CT>
struct ScaleLds {
  f32x2 v[CT][WQ == kWFull ? 1 : 16 * (kSpanGroups + 2)] __attribute__((aligned(16)));
};
// pairs from a column to the next: twice an odd number, so that the 16 columns'
// reads of 16 bytes meet no bank conflict
__device__ __forceinline__ int scale_stride(int n) {
  const int even = (n + 1) & ~1;
  return (even & 2) != 0 ? even : even + 2;
}

// Staging in two steps, so that other loads can be issued between them: `load`
// fetches, `store` writes to LDS.  g0, n: the span's groups; cols as in w_tiles.
template <int TK, int WQ, int CT, int THREADS>
struct ScaleStage {
  static_assert(2 * kSpanGroups <= THREADS, "one piece of 8 groups of a tile per thread");
  u32x4 s[CT];
  uint64_t z[CT];

  // pieces of 8 groups of a tile: of all columns in one run when the span is the
  // whole k, else of each column's part; anything odder goes one by one
  static __device__ __forceinline__ bool pieces(int n, int groups, int cols) {
    return cols == 16 && (n == groups || n % 8 == 0);
  }

  __device__ __forceinline__ void load(const WindowWeight& w, const int64_t (&j)[CT], int g0, int n, int groups, int cols) {
    if (!pieces(n, groups, cols)) return;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int t = (int)(threadIdx.x + 128 * c) % THREADS;  // the tiles' pieces start at different waves
      const int per = n / 8;  // pieces of a column's part
      const int64_t at = j[c] * groups + g0 + (n == groups ? 8 * t : t / per * groups + t % per * 8);
      typedef u32x4 any16 __attribute__((aligned(2)));
      typedef uint64_t any8 __attribute__((aligned(1)));
      if (t < 2 * n) {
        s[c] = *(const any16*)((const uint16_t*)w.scales + at);
        if constexpr ((WQ & kZeros) != 0) z[c] = *(const any8*)((const uint8_t*)w.zeros + at);
      }
    }
  }

  static __device__ __forceinline__ f32x2 pair(uint32_t s, uint32_t z) {
    return f32x2{half_f32<TK>((uint16_t)s), (WQ & kZeros) != 0 ? -16.0f - (float)z : -24.0f};
  }

  __device__ __forceinline__ void store(ScaleLds<WQ, CT>& lds, const WindowWeight& w, const int64_t (&j)[CT], int g0, int n,
                                        int groups, int cols) {
    const int stride = scale_stride(n);
    if (pieces(n, groups, cols)) {
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int t = (int)(threadIdx.x + 128 * c) % THREADS;
        if (t < 2 * n) {
          int col = 8 * t / n, g = 8 * t - col * n;
          f32x2 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t word = s[c][i / 2];
            v[i] = pair(word >> (16 * (i & 1)), (uint32_t)(z[c] >> (8 * i)) & 0xffu);
          }
          if (n % 8 == 0) {  // a piece is of one column
#pragma unroll
            for (int i = 0; i < 8; i += 2)
              *(f32x4*)&lds.v[c][col * stride + g + i] = f32x4{v[i][0], v[i][1], v[i + 1][0], v[i + 1][1]};
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              lds.v[c][col * stride + g] = v[i];
              if (++g == n) {
                g = 0;
                ++col;
              }
            }
          }
        }
      }
    } else {
#pragma unroll 1
      for (int c = 0; c < CT; ++c) {
        const uint16_t* sp = (const uint16_t*)w.scales + j[c] * groups + g0;
        const uint8_t* zp = (const uint8_t*)w.zeros + ((WQ & kZeros) != 0 ? j[c] * groups + g0 : 0);
#pragma unroll 4
        for (int i = threadIdx.x; i < cols * n; i += THREADS) {
          const int col = i / n, g = i - col * n;
          const int64_t at = (int64_t)col * groups + g;
          lds.v[c][col * stride + g] = pair(sp[at], (WQ & kZeros) != 0 ? zp[at] : 0u);
        }
      }
    }
  }
};

// the staged scales of the unit whose first pair in a column is at `at`
template <int WQ, int CT>
__device__ __forceinline__ void unit_scales(f32x4 (&sv)[CT], f32x4 (&zv)[CT], const ScaleLds<WQ, CT>& lds, int at) {
  if constexpr (WQ != kWFull) {
    constexpr int GU = 128 / group_len<WQ>();
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if constexpr (GU == 1) {
        const f32x2 v = lds.v[c][at];
        sv[c][0] = v[0];
        zv[c][0] = v[1];
      } else {
#pragma unroll
        for (int i = 0; i < GU; i += 2) {
          const f32x4 v = *(const f32x4*)&lds.v[c][at + i];
          sv[c][i] = v[0];
          zv[c][i] = v[1];
          sv[c][i + 1] = v[2];
          zv[c][i + 1] = v[3];
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// tot[c] = A . W over a whole k, by NW waves that each end with a part of the
// sum, to be added in the order of the waves.  k goes span by span (of at most
// kSpanGroups groups; 16-bit weights have one span), and in a span wave w takes
// a run of consecutive units; who sums what depends on k alone.  A wave has two
// units in flight: each is loaded again, two units on, as soon as it is used,
// and loads are never issued under a condition in the loop (a conditional load
// makes the compiler wait for more than it needs).
// ---------------------------------------------------------------------------
template <int TK, int WQ, int CT, int NW>
__device__ __forceinline__ void block_product(f32x4 (&tot)[CT], ScaleLds<WQ, CT>& lds, const Turn& turn,
                                              const WindowWeight& weight, const int64_t (&j)[CT], int cols,
                                              const uint16_t* arow, int k, int wave, int lane) {
  constexpr int NB = unit_blocks<WQ>();
  constexpr int UL = unit_len<WQ>();
  constexpr int GU = WQ == kWFull ? 0 : 128 / (WQ == kWFull ? 1 : group_len<WQ>());  // groups per unit
  WTiles<WQ, CT> t;
  w_tiles<WQ, CT>(t, weight, j, k, cols, lane);
  const int groups = WQ == kWFull ? 0 : k / (WQ == kWFull ? 1 : group_len<WQ>());
  int span = k;
  if constexpr (WQ != kWFull) {
    // as few spans as hold k, of about one length, each for all waves and (but
    // for the last) of whole pieces of 8 groups
    constexpr int most = kSpanGroups * group_len<WQ>() / UL;
    constexpr int step = NW * GU % 8 == 0 ? NW : 8 / GU;
    static_assert(most % step == 0 && step % NW == 0, "");
    const int units = (k + UL - 1) / UL, spans = (units + most - 1) / most;
    span = (((units + spans - 1) / spans + step - 1) / step * step) * UL;
  }
#pragma unroll 1
  for (int k0 = 0; k0 < k; k0 += span) {
    const int end = min(k, k0 + span);
    const int u0 = k0 / UL, full = end / UL;  // full units end here
    const int per = ((end + UL - 1) / UL - u0 + NW - 1) / NW;
    const int first = min(u0 + wave * per, full);
    const int n = min(u0 + wave * per + per, full) - first;
    const bool part = end % UL != 0 && (full - u0) / per == wave;
    const int g0 = u0 * GU, ng = min(span / UL * GU, groups - g0);  // the span's own groups
    const int row = min(lane & 15, cols - 1) * scale_stride(ng) - g0;

    WUnit<WQ, CT> w0, w1;
    u32x4 a0[NB], a1[NB];
    f32x4 sv[CT], zv[CT];
    auto load0 = [&](int u) __attribute__((always_inline)) {
      load_w<WQ, CT, false>(w0, t, u, k, lane);
      load_a<WQ, false>(a0, arow, u, k);
    };
    auto load1 = [&](int u) __attribute__((always_inline)) {
      load_w<WQ, CT, false>(w1, t, u, k, lane);
      load_a<WQ, false>(a1, arow, u, k);
    };
    const int second = n > 1 ? first + 1 : first;
    auto mul0 = [&](int u) __attribute__((always_inline)) {
      unit_scales(sv, zv, lds, row + u * GU);
      turn_unit<WQ, CT>(w0, a0, turn, lane);
      mul_unit<TK, WQ, CT, false, false>(w0, sv, zv, a0, tot, u, k);
    };
    auto mul1 = [&](int u) __attribute__((always_inline)) {
      unit_scales(sv, zv, lds, row + u * GU);
      turn_unit<WQ, CT>(w1, a1, turn, lane);
      mul_unit<TK, WQ, CT, false, false>(w1, sv, zv, a1, tot, u, k);
    };
    if constexpr (WQ != kWFull) {
      // the scales first, then the first units' codes, and the scales to LDS
      // while those are on their way
      ScaleStage<TK, WQ, CT, 64 * NW> st;
      st.load(weight, j, g0, ng, groups, cols);
      if (n > 0) {
        load_w<WQ, CT, false>(w0, t, first, k, lane);
        load_w<WQ, CT, false>(w1, t, second, k, lane);
      }
      if (n > 0) {
        load_a<WQ, false>(a0, arow, first, k);
        load_a<WQ, false>(a1, arow, second, k);
      }
      if (k0 > 0) lds_barrier();  // every wave is done with the span before
      st.store(lds, weight, j, g0, ng, groups, cols);
      lds_barrier();
    } else if (n > 0) {
      load0(first);
      load1(second);
    }
    if (n > 0) {
      int u = first;
      int left = n;
#pragma unroll 1
      while (left >= 4) {
        mul0(u);
        __builtin_amdgcn_sched_barrier(0);  // used up before it is loaded again: same registers, no copies
        load0(u + 2);
        __builtin_amdgcn_sched_barrier(0);
        mul1(u + 1);
        __builtin_amdgcn_sched_barrier(0);
        load1(u + 3);
        __builtin_amdgcn_sched_barrier(0);
        u += 2;
        left -= 2;
      }
      mul0(u);
      if (left == 3) load0(u + 2);
      if (left >= 2) mul1(u + 1);
      if (left == 3) mul0(u + 2);
    }
    if (part) {  // (groups past k are not staged: mul_unit does not use them)
      load_w<WQ, CT, true>(w0, t, full, k, lane);
      load_a<WQ, true>(a0, arow, full, k);
      unit_scales(sv, zv, lds, row + full * GU);
      turn_unit<WQ, CT>(w0, a0, turn, lane);
      mul_unit<TK, WQ, CT, false, true>(w0, sv, zv, a0, tot, full, k);
    }
  }
}

// The waves' sums: each writes its own into its slots of the turn (used up by
// then), and after a barrier any wave adds a tile's in the order of the waves.
template <int CT>
__device__ __forceinline__ void put_sums(u32x4* wave_slots, const f32x4 (&tot)[CT], int lane) {
  wave_lds_order();
#pragma unroll
  for (int c = 0; c < CT; ++c) ((f32x4*)wave_slots)[c * 64 + lane] = tot[c];
}
template <int NW, int N>
__device__ __forceinline__ f32x4 wave_sums(const u32x4 (&slots)[NW][N], int c, int lane) {
  f32x4 sum = ((const f32x4*)slots[0])[c * 64 + lane];
#pragma unroll
  for (int w = 1; w < NW; ++w) sum += ((const f32x4*)slots[w])[c * 64 + lane];
  return sum;
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
