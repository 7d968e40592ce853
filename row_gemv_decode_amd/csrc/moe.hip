// moe.hip -- a whole mixture-of-experts layer for a decode window's rows
// (m <= 16 tokens), for gfx950 (MI355X):
//
//   l_t   = x_t . Wr                                   (router logits, by the GEMV)
//   S_t   = the topk largest of l_t (equal values by lower expert first)
//   p_te  = exp(l_te) / sum over S_t (or over all experts) of exp(l_t.)
//   h_te  = silu(x_t . Wg_e) * (x_t . Wu_e)
//   out_t = sum over e in S_t of p_te (h_te . Wd_e)  +  sigmoid(x_t . wg) (h_t,shared . Wd_shared)
//
// HBM-bound on the distinct experts' weights, each read once per window (an
// expert's down weight once per 4 tokens that it serves).
//   moe_route_kernel  one workgroup, one wave per token: top-k, softmax and the
//                     list of distinct experts in ascending order with each
//                     one's tokens, whole and in parts of four (a second
//                     workgroup: the shared expert's gates)
//   moe_up_kernel     one workgroup per (distinct expert, 16 or 32 columns of
//                     h): gate and up columns side by side against all rows of
//                     x (a matrix-core tile holds 16 rows anyway, so tokens are
//                     not gathered), silu in the epilogue
//   moe_down_kernel   per distinct expert and part of its tokens, their output rows
//   moe_sum_kernel    adds each token's rows, times p
// h is kept as the sum of three 16-bit planes, multiplied in rows of the same
// matrix-core step, which hold the 24 bits of fp32.  (With two planes in bf16, 3 in
// 1000 bf16 outputs came out a step of the type away.)  The planes are bf16 where
// the weights can be, that is in bf16 layers and with 4-bit weights.  In f16 layers
// with 16-bit weights they are f16, which has few exponents: h is scaled by 2^-2,
// and each plane is the remainder of the one before times 2^11.  That is as good as
// fp32 for |h| from 2^-12 to 2^18; below, the first plane is subnormal, which the
// matrix core multiplies with as many fewer bits (inputs of 1e-3, h about 2^-20: a
// relative error of 3e-6).  p stays out of h for the same reason.  (Two planes of
// h p as they are: 3e-5 at inputs of 2^-4, 7e-3 at 2^-8, infinity past 65504.)  For
// 4-bit weights h is stored in the pair order that their decoding yields.
//
// Row invariance: which wave takes which part of k depends on the layer alone, a
// matrix-core row does not depend on the other rows, and a token's experts are
// added in the order of its own choice; so a token's output is the same bits in
// every window.
#include "skinny.h"
#include "wave_ops.h"
#include "window_kernel.h"

namespace skinny {

namespace {

constexpr int kMoeWaves = 4;
constexpr int kMoeDownTokens = 4;  // of a workgroup of the down product: 16 rows hold their planes

// Workgroup 0, one wave per token: each round of the top-k takes the largest
// remaining order key of the row (ties: the lowest column); lane i keeps the
// i-th winner.  The softmax sums in a fixed order: over the winners lane by
// lane, or over all logits.  Workgroup 1: the shared expert's gates.
// NC: logits per lane.
template <int TK, int NC>
__global__ __launch_bounds__(1024) void moe_route_kernel(MoeArgs a) {
  __shared__ uint32_t mask[64 * NC];  // tokens of each expert
  __shared__ int slot_of[64 * NC];      // its slot | its first part << 16
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int t = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int E = a.experts;

  if (blockIdx.x == 1) {
    const uint16_t* xr = (const uint16_t*)a.x + t * a.ldx;
    const uint16_t* wr = (const uint16_t*)a.shared_gate;
    float s = 0.0f;
#pragma unroll 4
    for (int c = lane * 8; c < a.d; c += 512) {
      const u32x4 xv = *(const u32x4*)(xr + c);
      const u32x4 wv = *(const u32x4*)(wr + c);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t xq = xv[q], wq = wv[q];
        s = __builtin_fmaf(half_f32<TK>((uint16_t)xq), half_f32<TK>((uint16_t)wq), s);
        s = __builtin_fmaf(half_f32<TK>((uint16_t)(xq >> 16)), half_f32<TK>((uint16_t)(wq >> 16)), s);
      }
    }
    s = wave_sum_f32(s);
    if (lane == 0) a.weights[t * (a.topk + 1) + a.topk] = 1.0f / (1.0f + expf(-s));
    return;
  }

  const float* row = a.logits + (int64_t)t * E;
  float x[NC];
#pragma unroll
  for (int u = 0; u < NC; ++u) x[u] = lane + 64 * u < E ? row[lane + 64 * u] : 0.0f;
  for (int e = tid; e < E; e += blockDim.x) mask[e] = 0;
  __syncthreads();

  // (a NaN may have the lowest key: it is moved up, so that no expert is taken twice)
  constexpr int kTaken = (int)0x80000000;
  int key[NC];
#pragma unroll
  for (int u = 0; u < NC; ++u) key[u] = lane + 64 * u < E ? max(order_key(x[u]), kTaken + 1) : kTaken;
  int top = 0, mine = 0, mine_e = 0;
  for (int i = 0; i < a.topk; ++i) {
    int best = key[0];
#pragma unroll
    for (int u = 1; u < NC; ++u) best = max(best, key[u]);
    const int kmax = wave_max_i32(best);
    int col = lane + 64 * (NC - 1);
#pragma unroll
    for (int u = NC - 2; u >= 0; --u) col = key[u] == kmax ? lane + 64 * u : col;
    const uint64_t b = __builtin_amdgcn_ballot_w64(best == kmax);
    int e;
    if ((b & (b - 1)) == 0) {  // uniform: one lane holds the maximum
      e = (int)__builtin_amdgcn_readlane((uint32_t)col, (uint32_t)__builtin_ctzll(b));
    } else {
      e = wave_min_i32(best == kmax ? col : 0x7fffffff);
    }
#pragma unroll
    for (int u = 0; u < NC; ++u) key[u] = lane + 64 * u == e ? kTaken : key[u];
    if (i == 0) top = kmax;
    mine = lane == i ? kmax : mine;
    mine_e = lane == i ? e : mine_e;
  }
  const float vtop = key_value(top);
  const float ex = lane < a.topk ? expf(key_value(mine) - vtop) : 0.0f;
  float total;
  if (a.renorm) {
    total = wave_sum_f32(ex);
  } else {
    total = 0.0f;
#pragma unroll
    for (int u = 0; u < NC; ++u) total += lane + 64 * u < E ? expf(x[u] - vtop) : 0.0f;
    total = wave_sum_f32(total);
  }
  const float p = ex / total;
  if (lane < a.topk) {
    atomicOr(&mask[mine_e], 1u << t);
    a.weights[t * (a.topk + 1) + lane] = p;
    if (a.topk_idx != nullptr) a.topk_idx[t * a.topk + lane] = mine_e;
    if (a.topk_weight != nullptr) a.topk_weight[t * a.topk + lane] = p;
  }
  __syncthreads();

  if (t == 0) {  // the distinct experts, ascending
    int n = 0, np = 0;
    uint32_t masks[NC];
#pragma unroll
    for (int u = 0; u < NC; ++u) masks[u] = lane + 64 * u < E ? mask[lane + 64 * u] : 0u;
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int e = lane + 64 * u;
      const uint32_t mk = masks[u];
      const uint64_t lower = (1ull << lane) - 1;
      const uint64_t b = __builtin_amdgcn_ballot_w64(mk != 0);
      const int slot = n + __builtin_popcountll(b & lower);
      const int parts = (__builtin_popcount(mk) + kMoeDownTokens - 1) / kMoeDownTokens;  // at most 4
      const uint64_t b1 = __builtin_amdgcn_ballot_w64((parts & 1) != 0);
      const uint64_t b2 = __builtin_amdgcn_ballot_w64((parts & 2) != 0);
      const uint64_t b4 = __builtin_amdgcn_ballot_w64((parts & 4) != 0);
      const int part = np + __builtin_popcountll(b1 & lower) + 2 * __builtin_popcountll(b2 & lower) +
                       4 * __builtin_popcountll(b4 & lower);
      if (mk != 0) {
        slot_of[e] = slot | (part << 16);
        a.slots[slot] = (uint32_t)e | (mk << 16);
        for (int q = 0, left = __builtin_popcount(mk); q < parts; ++q, left -= kMoeDownTokens)
          a.parts[4 * (part + q)] = (uint32_t)e | ((uint32_t)min(left, kMoeDownTokens) << 16);
      }
      n += __builtin_popcountll(b);
      np += __builtin_popcountll(b1) + 2 * __builtin_popcountll(b2) + 4 * __builtin_popcountll(b4);
    }
    for (int i = n + lane; i < a.max_slots; i += 64) a.slots[i] = 0;  // slots without a token
    for (int i = np + lane; i < a.max_parts; i += 64) a.parts[4 * i] = 0;
  }
  __syncthreads();
  if (lane < a.topk) {
    const int at = slot_of[mine_e];
    a.slot_rank[(at & 0xffff) * kGemvMaxM + t] = lane;  // (read for the tokens in the slot's mask only)
    const int place = __builtin_popcount(mask[mine_e] & ((1u << t) - 1));  // of the expert's tokens
    uint32_t* part = a.parts + 4 * ((at >> 16) + place / kMoeDownTokens);
    ((uint16_t*)(part + 1))[place % kMoeDownTokens] = (uint16_t)(t * a.topk + lane);
  }
}

// where column i of h lies in memory: for 4-bit weights each run of eight is
// kept in the pair order of codes16
template <int WQ>
__device__ __forceinline__ int h_place(int i) {
  if constexpr (WQ == kWFull) {
    return i;
  } else {
    const int e = i & 7;
    return (i & ~7) + (e < 4 ? 2 * e : 2 * e - 7);
  }
}

// Waves that share a column's sum in the down product: more than one where k has
// many units, or where one token's experts would leave most of the chip idle.  By
// the layer alone, so that every window adds in the same order.  Every wave has
// a unit.
__host__ __device__ __forceinline__ int down_waves(int units, int64_t d, int topk) {
  int n = 1;
  while (n < kMoeWaves && (units > 8 * n || topk * (d / 16) * n < 1024) &&
         (2 * n - 1) * ((units + 2 * n - 1) / (2 * n)) < units)
    n *= 2;
  return n;
}

// Column tiles of a wave in the down product (a column's arithmetic does not depend
// on them): one for 16-bit weights; for 4-bit ones two, or, where that leaves at
// least 3072 waves of work, four (not for groups of 32, whose waves then take too
// many registers).  Measured (us, 1 / 2 / 4 tiles; waves of 4): 16 bits, 1 of 256
// experts (d = 5120, inter = 896) 20.7 / 22.0 / 23.9, 16 of 64 (d = 2560) 55.3 / 55.6 /
// 59.2; groups of 128, 16 of 256 103 / 82 / 75 (12800), 16 of 8 (d = 4096, inter = 8192)
// 73 / 59 / 51 (3584), 1 of 8 15.4 / 14.7 / 18.6 (512); of 64, 3 of 256 28.7 / 26.0 / 28.5
// (2480); of 32, 5 of 512 (d = 2560, inter = 672) 28.4 / 26.1 / 25.1 (2000), 16 of 512 the
// whole layer - / 162 / 166 (6400)
int down_tiles(int group, int64_t d, int64_t waves_of_4) {
  return group == 0 ? 1 : group > 32 && d % 64 == 0 && waves_of_4 >= 3072 ? 4 : 2;
}

__device__ const u32x4 kZeroLine = {0u, 0u, 0u, 0u};

// The row that a lane of token tk reads: its own if the expert serves it, else
// one that is read anyway (whose sums are then not stored for tk)
__device__ __forceinline__ int served_row(uint32_t entry, int tk, int m) {
  const uint32_t mask = (entry >> 16) & ((1u << m) - 1);
  return ((mask >> tk) & 1u) != 0 ? tk : __builtin_ctz(mask);
}

// h's planes (see above): their type PK, and the scales
constexpr int kPlanes = 3;
template <int TK, int WQ>
constexpr int plane_kind() { return WQ == kWFull ? TK : CK_BF16; }
template <int PK>
constexpr float inner_scale() { return PK == CK_F16 ? 0.25f : 1.0f; }
template <int PK>
constexpr float plane_step() { return PK == CK_F16 ? 2048.0f : 1.0f; }

// Rows of h, kPlanes * inter long: token t's i-th expert's is row t * topk + i; the
// shared expert's rows, one per token, lie after them.  The rows of y likewise.
__device__ __forceinline__ int64_t shared_h(const MoeArgs& a) { return (int64_t)a.m * a.topk * kPlanes * a.inter; }

// GT tiles of 16 columns of h: columns of w13 are the gate's 0 .. inter - 1,
// then the up's
template <int TK, int WQ, int GT>
__global__ __launch_bounds__(64 * kMoeWaves, 2) void moe_up_kernel(MoeArgs a) {
  __shared__ ScaleLds<WQ, 2 * GT> lds;
  __shared__ u32x4 turn_s[kMoeWaves][turn_slots<WQ, 2 * GT>() * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 4;
  const int k = (int)a.d;
  const int tiles = (int)a.inter / (16 * GT);

  // the shared expert's workgroups come first: they are sure to have work
  const int shared_tiles = (int)a.shared_inter / (16 * GT);
  const bool shared = (int)blockIdx.x < shared_tiles;
  const int b = (int)blockIdx.x - shared_tiles;
  const int slot = shared ? 0 : b / tiles;
  const uint32_t entry = shared ? 0xffff0000u : a.slots[slot];  // every token goes to the shared expert
  if (entry < 0x10000u) return;  // no token: a slot past the window's experts
  const int tile = shared ? (int)blockIdx.x : b - slot * tiles;
  const int64_t inter = shared ? a.shared_inter : a.inter;
  const int64_t j0 = (int64_t)(entry & 0xffffu) * 2 * inter + 16 * GT * tile;
  int64_t j[2 * GT];
  f32x4 tot[2 * GT];
#pragma unroll
  for (int c = 0; c < GT; ++c) {
    j[c] = j0 + 16 * c;
    j[GT + c] = j0 + 16 * c + inter;
    tot[c] = tot[GT + c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const uint16_t* arow = (const uint16_t*)a.x + served_row(entry, lane >> 2, a.m) * a.ldx + 8 * (lane & 3);
  block_product<TK, WQ, 2 * GT, kMoeWaves>(tot, lds, Turn(turn_s[wave], lane), shared ? a.s13 : a.w13, j, 16, arow, k,
                                           wave, lane);
  put_sums(turn_s[wave], tot, lane);
  __syncthreads();
  if (wave < GT) {
    const f32x4 g = wave_sums(turn_s, wave, lane), up = wave_sums(turn_s, GT + wave, lane);
    constexpr int PK = plane_kind<TK, WQ>();
    uint16_t* hb = a.h + (shared ? shared_h(a) : 0) + 16 * (tile * GT + wave) + h_place<WQ>(lane & 15);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int tk = 4 * h + q;
      if (tk < a.m && ((entry >> (16 + tk)) & 1u) != 0) {
        float v = g[q] / (1.0f + expf(-g[q])) * up[q] * inner_scale<PK>();
        const int hrow = shared ? tk : tk * a.topk + a.slot_rank[slot * kGemvMaxM + tk];
        uint16_t* o = hb + (int64_t)hrow * kPlanes * inter;
#pragma unroll
        for (int i = 0; i < kPlanes; ++i) {
          const uint16_t bits = f32_half<PK>(v);
          o[i * inter] = bits;
          const float part = half_f32<PK>(bits);
          v = __builtin_isfinite(part) ? (v - part) * plane_step<PK>() : 0.0f;  // exact: the remainder of the rounding
        }
      }
    }
  }
}

// The scales and zero points of one unit of CT adjacent tiles of 16 columns:
// lane group h fetches tile h mod CT's, in one load for the scales (2, 4 or 8
// bytes of each column) and one for the zero points (half as many).
template <int WQ, int CT>
struct UnitScales {
  static constexpr int GU = 128 / group_len<WQ>();  // groups per unit
  uint32_t s[2], z;
  uint32_t shift;  // groups to drop at the low end

  // j: the first column, col: the lane's column from there, u: the unit,
  // groups: per column; rows: columns from j to the end of the weight (or 64,
  // if there are more): a load that would pass the end is moved back
  __device__ __forceinline__ void load(const WindowWeight& w, int64_t j, int col, int u, int groups, int rows) {
    const int at = col * groups + u * GU;
    const int from = min(at, rows * groups - GU);
    shift = (uint32_t)(at - from);
    const char* sp = (const char*)w.scales + j * groups * 2 + 2 * from;
    if constexpr (GU == 1) {
      s[0] = *(const uint16_t*)sp;
    } else if constexpr (GU == 2) {
      typedef uint32_t any __attribute__((aligned(2)));
      s[0] = *(const any*)sp;
    } else {
      typedef uint64_t any __attribute__((aligned(2)));
      const uint64_t q = *(const any*)sp;
      s[0] = (uint32_t)q;
      s[1] = (uint32_t)(q >> 32);
    }
    if constexpr ((WQ & kZeros) != 0) {
      const char* zp = (const char*)w.zeros + j * groups + from;
      if constexpr (GU == 1) {
        z = *(const uint8_t*)zp;
      } else if constexpr (GU == 2) {
        typedef uint16_t any __attribute__((aligned(1)));
        z = *(const any*)zp;
      } else {
        typedef uint32_t any __attribute__((aligned(1)));
        z = *(const any*)zp;
      }
    }
  }

  // the pairs that the product takes; a group past the unit's n has scale 0
  template <int TK>
  __device__ __forceinline__ void get(f32x4 (&sv)[CT], f32x4 (&zv)[CT], int n) const {
    uint32_t lo = s[0], hi = 0;
    if constexpr (GU == 4) {
      const uint64_t q = (((uint64_t)s[1] << 32) | s[0]) >> (16 * shift);
      lo = (uint32_t)q;
      hi = (uint32_t)(q >> 32);
    } else {
      lo >>= 16 * shift;
    }
    const u32x4 l = spread4(lo);
    u32x4 m = {0u, 0u, 0u, 0u}, zs = {0x08080808u, 0x08080808u, 0x08080808u, 0x08080808u};
    if constexpr (GU == 4) m = spread4(hi);
    if constexpr ((WQ & kZeros) != 0) zs = spread4(z >> (8 * shift));
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int g = 0; g < GU; ++g) {
        const uint32_t word = g < 2 ? (uint32_t)l[c] : (uint32_t)m[c], zw = zs[c];
        const float f = half_f32<TK>((uint16_t)((g & 1) != 0 ? word >> 16 : word));
        sv[c][g] = GU > 1 && g >= n ? 0.0f : f;
        zv[c][g] = -16.0f - (float)((zw >> (8 * g)) & 0xffu);
      }
  }
};
template <int CT>
struct UnitScales<kWFull, CT> {
  template <int TK>
  __device__ __forceinline__ void get(f32x4 (&)[CT], f32x4 (&)[CT], int) const {}
};

// The experts' outputs, as fp32 rows y for the tokens that each expert serves.
// A wave owns CT tiles of 16 columns (KS = 1), or KS waves share them, each with
// a run of the units of k.  Few experts serve many tokens, so the rows of the
// matrix-core tile hold the planes of h: 4 tokens, plane p in the rows from 4 p
// (the last plane twice), and one step multiplies all planes.  An expert that serves
// more tokens has further parts, which read its weight again.  The parts come as a
// list: as further workgroups of every slot, most of which had no token, they took
// 16 of 256 experts 20 us more.
// Bound by what a wave does per byte, not by memory alone: with the planes in
// turn, h for 16 tokens and the waves splitting k, 16 of 256 experts (d = 5120,
// inter = 896, 4 bits) took 130 to 170 us; so, 77 (3.8 TB/s).
template <int TK, int WQ, int CT>
__global__ __launch_bounds__(64 * kMoeWaves, 2) void moe_down_kernel(MoeArgs a) {
  constexpr int NB = unit_blocks<WQ>();
  constexpr int UL = unit_len<WQ>();
  constexpr int TT = kMoeDownTokens;
  constexpr int PK = plane_kind<TK, WQ>();
  constexpr int GU = WQ == kWFull ? 1 : 128 / (WQ == kWFull ? 1 : group_len<WQ>());
  __shared__ u32x4 turn_s[kMoeWaves][turn_slots<WQ, CT>() * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15;
  const int sets = (int)a.d / 16 / CT;  // (d is a multiple of 16 CT)

  // the workgroup's expert and sets of columns; the shared expert's come first
  const int KS0 = a.shared_inter > 0 ? down_waves((int)((a.shared_inter + UL - 1) / UL), a.d, a.topk) : 1;
  const int per0 = kMoeWaves / KS0;
  const int blocks0 = a.shared_inter > 0 ? (a.m + TT - 1) / TT * ((sets + per0 - 1) / per0) : 0;
  const bool shared = (int)blockIdx.x < blocks0;
  const int KS = shared ? KS0 : down_waves((int)((a.inter + UL - 1) / UL), a.d, a.topk);
  const int per = kMoeWaves / KS;  // sets of a workgroup
  const int blocks = (sets + per - 1) / per;
  // its part: the expert and its tokens' rows of h
  const int b = (int)blockIdx.x - (shared ? 0 : blocks0);
  const int part = b / blocks;
  uint32_t expert = 0;
  int tokens, hrows[TT];
  if (shared) {  // (every token goes to the shared expert)
    tokens = min(a.m - TT * part, TT);
#pragma unroll
    for (int i = 0; i < TT; ++i) hrows[i] = TT * part + i;
  } else {
    const u32x4 p = ((const u32x4*)a.parts)[part];
    const uint32_t head = p[0], r01 = p[1], r23 = p[2];
    expert = head & 0xffffu;
    tokens = (int)(head >> 16);
    if (tokens == 0) return;  // a part past the window's last
    hrows[0] = (int)(r01 & 0xffffu);
    hrows[1] = (int)(r01 >> 16);
    hrows[2] = (int)(r23 & 0xffffu);
    hrows[3] = (int)(r23 >> 16);
  }
  const int set = (b - part * blocks) * per + wave / KS;
  const int k = (int)(shared ? a.shared_inter : a.inter);
  const int units = (k + UL - 1) / UL;
  const int run = (units + KS - 1) / KS;  // every wave has a unit
  const int first = wave % KS * run, n = min(run, units - first);

  // lane group l >> 2 reads row l >> 2: a plane of a token, or of the first one
  int hrow = hrows[0];
#pragma unroll
  for (int i = 1; i < TT; ++i) hrow = (lane >> 2) % TT == i && i < tokens ? hrows[i] : hrow;
  const int plane = min((lane >> 2) / TT, kPlanes - 1);

  const WindowWeight& W = shared ? a.s2 : a.w2;
  const int64_t e0 = (int64_t)expert * a.d;  // the expert's first column
  const uint32_t cbytes = (uint32_t)(WQ == kWFull ? k * 2 : k >> 1);
  const uint32_t coff = (uint32_t)(lane >> 2) * cbytes + 16 * (lane & 3);
  const uint16_t* hbase = a.h + (shared ? shared_h(a) : 0);
  const uint32_t hoff = (uint32_t)((hrow * kPlanes + plane) * k + 8 * (lane & 3));
  const int groups = k / (WQ == kWFull ? 1 : group_len<WQ>());
  const int col = 16 * ((lane >> 4) % CT) + row;

  struct Item {
    WUnit<WQ, CT> w;
    UnitScales<WQ, CT> s;
    u32x4 a[NB];
  };
  const int64_t j = e0 + (int64_t)min(set, sets - 1) * (16 * CT);  // (a wave past the last set repeats it)
  const char* cset = (const char*)W.codes + j * cbytes;
  // A k that is no multiple of the unit: blocks past k read zeros for h and the
  // unit's first block for the weight, so every item is multiplied whole, with
  // no branch between the matrix-core steps.
  auto load = [&](Item& q, int u) __attribute__((always_inline)) {
    const int rest = k - u * UL;
    if constexpr (WQ == kWFull) {
      const char* cu = cset + (int64_t)u * 128;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int off = 32 * i >= rest ? 0 : 64 * i;
#pragma unroll
        for (int c = 0; c < CT; ++c) q.w.v[c][i] = *(const u32x4*)(cu + (coff + (uint32_t)(c * 16) * cbytes) + off);
      }
    } else {
      const char* cu = cset + (int64_t)u * 64;
      const uint32_t off = coff - (group_len<WQ>() != 128 && 32 * (lane & 3) >= rest ? 16u * (lane & 3) : 0u);
#pragma unroll
      for (int c = 0; c < CT; ++c) q.w.v[c][0] = *(const u32x4*)(cu + (off + (uint32_t)(c * 16) * cbytes));
      const int64_t rows = shared ? a.d - j : a.experts * a.d - j;
      q.s.load(W, j, col, u, groups, (int)min(rows, (int64_t)64));
    }
    const uint16_t* hu = hbase + (int64_t)u * UL;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint16_t* at = hu + hoff + 32 * i;
      if (group_len<WQ>() != 128 && 32 * i >= rest) at = (const uint16_t*)&kZeroLine;
      q.a[i] = *(const u32x4*)at;
    }
  };

  const Turn turn(turn_s[wave], lane);
  f32x4 tot[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) tot[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto mul = [&](Item& q, int u) __attribute__((always_inline)) {
    f32x4 sv[CT], zv[CT];
    q.s.template get<TK>(sv, zv, groups - u * GU);
    turn_unit<WQ, CT>(q.w, q.a, turn, lane);
    mul_unit<PK, WQ, CT, true, false>(q.w, sv, zv, q.a, tot, 0, 0);
    __builtin_amdgcn_sched_barrier(0);  // used up before it is loaded again: same registers, no copies
  };
  {
    Item q0, q1;
    int u = first, left = n;
    load(q0, u);
    load(q1, n > 1 ? u + 1 : u);
#pragma unroll 1
    while (left >= 4) {
      mul(q0, u);
      load(q0, u + 2);
      __builtin_amdgcn_sched_barrier(0);
      mul(q1, u + 1);
      load(q1, u + 3);
      __builtin_amdgcn_sched_barrier(0);
      u += 2;
      left -= 2;
    }
    mul(q0, u);
    if (left == 3) load(q0, u + 2);
    if (left >= 2) mul(q1, u + 1);
    if (left == 3) mul(q0, u + 2);
  }

  if (KS > 1) {
    f32x4* red = (f32x4*)turn_s[wave];
    wave_lds_order();
#pragma unroll
    for (int c = 0; c < CT; ++c) red[c * 64 + lane] = tot[c];
    __syncthreads();
    if (wave % KS == 0) {
      for (int w = 1; w < KS; ++w)
#pragma unroll
        for (int c = 0; c < CT; ++c) tot[c] += ((const f32x4*)turn_s[wave + w])[c * 64 + lane];
    }
  }
  // the planes' sums, lane group h plane h's, to one
  constexpr float down = 1.0f / plane_step<PK>();
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float v = tot[c][q];
      auto s32 = __builtin_amdgcn_permlane32_swap(ubits(v), ubits(v), false, false);
      auto lo = __builtin_amdgcn_permlane16_swap(s32[0], s32[0], false, false);  // planes 0 and 1
      auto hi = __builtin_amdgcn_permlane16_swap(s32[1], s32[1], false, false);  // plane 2
      const float rest = __builtin_fmaf(down, fbits(hi[0]), fbits(lo[1]));
      tot[c][q] = __builtin_fmaf(down, rest, fbits(lo[0])) * (1.0f / inner_scale<PK>());
    }
  if (wave % KS == 0 && set < sets && lane < 16) {
    float* y = a.y + (shared ? (int64_t)a.m * a.topk * a.d : 0) + (int64_t)set * (16 * CT) + row;
#pragma unroll
    for (int q = 0; q < TT; ++q)
      if (q < tokens) {
#pragma unroll
        for (int c = 0; c < CT; ++c) y[(int64_t)hrows[q] * a.d + 16 * c] = tot[c][q];
      }
  }
}

// out[t] = the sum of token t's experts' rows, largest logit first, then the
// shared expert's, each times its weight; a thread adds four columns.  Twelve rows are fetched before
// the first is added (loads past the last row repeat it), so the kernel waits
// for memory once for up to twelve (1 of 64 experts, top 4, as a plain sum: 2.4 us,
// and 2.7 row by row; 2.7 with the weights.  Of the 4.6 us of 5 of 512 most is
// reading rows that other XCDs wrote).
__global__ __launch_bounds__(64) void moe_sum_kernel(MoeArgs a) {
  constexpr int R = 12;
  const int64_t j = 4 * (int64_t)(blockIdx.x * 64 + threadIdx.x);
  const int t = blockIdx.y;
  if (j >= a.d) return;
  const float* y = a.y + (int64_t)t * a.topk * a.d + j;
  const float* ys = a.y + (int64_t)(a.m * a.topk + t) * a.d + j;  // the shared expert's
  const float* w = a.weights + t * (a.topk + 1);
  const int n = a.topk + (a.shared_inter > 0 ? 1 : 0);
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += R) {
    f32x4 v[R];
    float p[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int at = min(i0 + i, n - 1);
      v[i] = *(const f32x4*)(at < a.topk ? y + (int64_t)at * a.d : ys);
      p[i] = w[at];
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = i0 + i < n ? __builtin_fmaf(p[i], v[i][e], sum[e]) : sum[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) store_kind(a.out, t * a.ldo + j + e, sum[e], a.out_kind);
}

typedef void (*moe_fn)(MoeArgs);

template <int TK>
moe_fn pick_route(int experts) {
  return experts <= 64    ? moe_route_kernel<TK, 1>
         : experts <= 128 ? moe_route_kernel<TK, 2>
         : experts <= 256 ? moe_route_kernel<TK, 4>
         : experts <= 512 ? moe_route_kernel<TK, 8>
                          : moe_route_kernel<TK, 16>;
}

template <int TK, int WQ>
moe_fn pick_up(bool wide) { return wide ? moe_up_kernel<TK, WQ, 2> : moe_up_kernel<TK, WQ, 1>; }

template <int TK, int WQ>
moe_fn pick_down(int tiles) {
  if constexpr (WQ == kWFull) {
    return moe_down_kernel<TK, WQ, 1>;
  } else {
    if constexpr (group_len<WQ>() > 32)
      if (tiles == 4) return moe_down_kernel<TK, WQ, 4>;
    return moe_down_kernel<TK, WQ, 2>;
  }
}

// the up kernel (tiles 0), or the down kernel of that many column tiles
template <int TK>
moe_fn pick_weight(int group, bool zeros, int tiles, bool wide) {
#define SKINNY_MOE_PICK(wq) return tiles == 0 ? pick_up<TK, wq>(wide) : pick_down<TK, wq>(tiles)
  switch (group + (zeros ? kZeros : 0)) {
    case 0: SKINNY_MOE_PICK(kWFull);
    case 32: SKINNY_MOE_PICK(32);
    case 64: SKINNY_MOE_PICK(64);
    case 128: SKINNY_MOE_PICK(128);
    case 32 + kZeros: SKINNY_MOE_PICK(32 + kZeros);
    case 64 + kZeros: SKINNY_MOE_PICK(64 + kZeros);
    default: SKINNY_MOE_PICK(128 + kZeros);
  }
#undef SKINNY_MOE_PICK
}

moe_fn pick(int kind, int group, bool zeros, int tiles, bool wide) {
  return kind == CK_F16 ? pick_weight<CK_F16>(group, zeros, tiles, wide) : pick_weight<CK_BF16>(group, zeros, tiles, wide);
}

}  // namespace

int moe_planes() { return kPlanes; }

namespace {

// workgroups of a layer's launches, and how many slots and parts they cover
struct MoeGrid {
  int64_t slots, parts, up, down;
  int down_tiles;
  bool wide;
};

MoeGrid moe_grid(const MoeArgs& a, int group) {
  MoeGrid g;
  const int64_t pairs = (int64_t)a.m * a.topk;
  g.slots = pairs < a.experts ? pairs : a.experts;
  // An expert of n tokens has (n + 3) / 4 parts: one for n <= 4, (n + 3 slots) / 4 in all at most
  static_assert(kMoeDownTokens == 4, "");
  g.parts = a.m <= 4 ? g.slots : (pairs + 3 * g.slots) / 4;
  // Two column tiles of h per workgroup where that still leaves many workgroups:
  // the loads of x serve twice the columns (a column's arithmetic does not depend
  // on it).  Measured (us, one / two tiles; sets of 32 columns): 4480 (16 of 256
  // experts) 154 / 146, 2048 (16 of 8, inter = 8192) 78 / 74, 1050 (5 of 512) 36 / 40,
  // 280 (1 of 256 bf16) 42 / 49
  g.wide = g.slots * (a.inter / 32) >= 2048;
  const int64_t tile = g.wide ? 32 : 16;
  g.up = g.slots * (a.inter / tile) + a.shared_inter / tile;
  // the down product: as in its kernel
  const int unit = group == 0 ? unit_len<kWFull>() : unit_len<128>();
  const int64_t shared_parts = a.shared_inter > 0 ? (a.m + kMoeDownTokens - 1) / kMoeDownTokens : 0;
  auto waves = [&](int64_t inter) { return down_waves((int)((inter + unit - 1) / unit), a.d, a.topk); };
  const int64_t ks = waves(a.inter), ks0 = shared_parts > 0 ? waves(a.shared_inter) : 1;
  g.down_tiles = down_tiles(group, a.d, (g.parts * ks + shared_parts * ks0) * (a.d / 64));
  const int64_t sets = a.d / 16 / g.down_tiles;
  auto blocks = [&](int64_t k) { return (sets + kMoeWaves / k - 1) / (kMoeWaves / k); };
  g.down = g.parts * blocks(ks) + shared_parts * blocks(ks0);
  return g;
}

}  // namespace

bool moe_fits(const MoeArgs& args, int group) {
  const MoeGrid g = moe_grid(args, group);
  return (g.up > g.down ? g.up : g.down) * (64 * kMoeWaves) <= kMaxLaunchThreads;
}

hipError_t launch_moe(const MoeArgs& args, int kind, int group, hipStream_t stream) {
  MoeArgs a = args;
  if (a.m < 1 || a.m > kGemvMaxM || a.experts < 1 || a.experts > kMoeMaxExperts || a.topk < 1 ||
      a.topk > SKINNY_TOPK_MAX || a.topk > a.experts || a.d % 32 != 0 || a.inter % 32 != 0 || a.shared_inter % 32 != 0 ||
      (group != 0 && group != 32 && group != 64 && group != 128) ||
      (group != 0 && (a.d % group != 0 || a.inter % group != 0 || a.shared_inter % group != 0)) ||
      (kind != CK_F16 && kind != CK_BF16))
    return hipErrorInvalidValue;
  const MoeGrid g = moe_grid(a, group);
  if (g.slots > a.max_slots || a.max_slots > kGemvMaxM * SKINNY_TOPK_MAX || !moe_fits(a, group)) return hipErrorInvalidValue;
  a.max_parts = (int32_t)g.parts;
  const bool zeros = a.w13.zeros != nullptr;
  const bool f16 = kind == CK_F16;
  hipLaunchKernelGGL(f16 ? pick_route<CK_F16>(a.experts) : pick_route<CK_BF16>(a.experts),
                     dim3(a.shared_inter > 0 ? 2 : 1), dim3(64 * a.m), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(pick(kind, group, zeros, 0, g.wide), dim3((unsigned)g.up), dim3(64 * kMoeWaves), 0, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(pick(kind, group, zeros, g.down_tiles, false), dim3((unsigned)g.down), dim3(64 * kMoeWaves), 0, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_sum_kernel, dim3((unsigned)((a.d + 255) / 256), (unsigned)a.m), dim3(64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace skinny
