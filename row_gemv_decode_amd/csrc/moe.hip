// moe.hip -- a whole mixture-of-experts layer for a decode window's rows
// (m <= 16 tokens), for gfx950 (MI355X):
//
//   l_t   = x_t . Wr                                   (router logits, by the GEMV)
//   S_t   = the topk largest of l_t (equal values by lower expert first)
//   p_te  = exp(l_te) / sum over S_t (or over all experts) of exp(l_t.)
//   h_te  = silu(x_t . Wg_e) * (x_t . Wu_e) * p_te
//   out_t = sum over e in S_t of h_te . Wd_e  +  (sigmoid(x_t . wg) * h_t,shared) . Wd_shared
//
// HBM-bound on the distinct experts' weights, each read once per window.
//   moe_route_kernel  one workgroup, one wave per token: top-k, softmax and the
//                     list of distinct experts in ascending order with each
//                     one's tokens (a second workgroup: the shared expert's
//                     gates)
//   moe_up_kernel     one workgroup per (distinct expert, 16 or 32 columns of
//                     h): gate and up columns side by side against all rows of
//                     x (a matrix-core tile holds 16 rows anyway, so tokens are
//                     not gathered), p and silu in the epilogue
//   moe_down_kernel   one workgroup per 32 columns of the layer's output and
//                     share of the experts' k: a row that an expert does not
//                     serve is a row of zeros, so the matrix core adds the
//                     experts of every token by itself, and the combine costs
//                     nothing; the last workgroup of a column range to finish
//                     adds the shares in order
// h is kept as the sum of planes in the weights' type, multiplied one after
// another (the matrix cores have time for it while the weights stream): two,
// 16 (bf16) or 22 (f16) bits, under a 16-bit output, where one plane would add
// as much error as the output's own rounding; three (bf16, 24 bits) under an
// fp32 output.  For 4-bit weights h is stored in the pair order that their
// decoding yields.
//
// Row invariance: which wave takes which part of k depends on the expert and
// the part alone, each wave adds its experts in ascending order, and what the
// other tokens' experts add to a row is an exact zero; so a token's output is
// the same bits in every window.
#include "skinny.h"
#include "wave_ops.h"
#include "window_kernel.h"

namespace skinny {

namespace {

constexpr int kMoeWaves = 4;

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

// Workgroup 0, one wave per token: each round of the top-k takes the largest
// remaining order key of the row (ties: the lowest column); lane i keeps the
// i-th winner.  The softmax sums in a fixed order: over the winners lane by
// lane, or over all logits.  Workgroup 1: the shared expert's gates.
// NC: logits per lane.
template <int TK, int NC>
__global__ __launch_bounds__(1024) void moe_route_kernel(MoeArgs a) {
  __shared__ uint32_t mask[64 * NC];  // tokens of each expert
  __shared__ int slot_of[64 * NC];
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
    if (lane == 0) a.gates[t] = 1.0f / (1.0f + expf(-s));
    return;
  }

  const float* row = a.logits + (int64_t)t * E;
  float x[NC];
#pragma unroll
  for (int u = 0; u < NC; ++u) x[u] = lane + 64 * u < E ? row[lane + 64 * u] : 0.0f;
  for (int e = tid; e < E; e += blockDim.x) mask[e] = 0;
  __syncthreads();

  int key[NC];
#pragma unroll
  for (int u = 0; u < NC; ++u) key[u] = lane + 64 * u < E ? order_key(x[u]) : (int)0x80000000;
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
    e = min(e, E - 1);  // (a NaN logit may leave no key above the lowest: keep the index in range)
#pragma unroll
    for (int u = 0; u < NC; ++u) key[u] = lane + 64 * u == e ? (int)0x80000000 : key[u];
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
    if (a.topk_idx != nullptr) a.topk_idx[t * a.topk + lane] = mine_e;
    if (a.topk_weight != nullptr) a.topk_weight[t * a.topk + lane] = p;
  }
  __syncthreads();

  if (t == 0) {  // the distinct experts, ascending
    int n = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const uint32_t mk = e < E ? mask[e] : 0u;
      const uint64_t b = __builtin_amdgcn_ballot_w64(mk != 0);
      const int slot = n + __builtin_popcountll(b & ((1ull << lane) - 1));
      if (mk != 0) {
        slot_of[e] = slot;
        a.slots[slot] = (uint32_t)e | (mk << 16);
      }
      n += __builtin_popcountll(b);
    }
    for (int i = n + lane; i < a.max_slots; i += 64) a.slots[i] = 0;  // slots without a token
    if (lane == 0) *a.nslots = n;
  }
  __syncthreads();
  // (a weight is read for the tokens in the slot's mask only)
  if (lane < a.topk) a.slot_w[slot_of[mine_e] * kGemvMaxM + t] = p;
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

// GT tiles of 16 columns of h: columns of w13 are the gate's 0 .. inter - 1,
// then the up's
template <int TK, int WQ, int NP, int GT>
__global__ __launch_bounds__(64 * kMoeWaves, 2) void moe_up_kernel(MoeArgs a) {
  __shared__ f32x4 red[kMoeWaves][2 * GT][64];
  __shared__ ScaleLds<WQ, 2 * GT> lds;
  __shared__ u32x4 turn_s[kMoeWaves][turn_slots<WQ, 2 * GT, 1>() * 64];
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
  const int row = min(lane >> 2, a.m - 1);
  const uint16_t* arow = (const uint16_t*)a.x + row * a.ldx + 8 * (lane & 3);
  block_product<TK, WQ, 2 * GT, kMoeWaves>(tot, lds, Turn(turn_s[wave], lane), shared ? a.s13 : a.w13, j, 16, arow, k,
                                           wave, lane);
#pragma unroll
  for (int c = 0; c < 2 * GT; ++c) red[wave][c][lane] = tot[c];
  __syncthreads();
  if (wave < GT) {
    f32x4 g = red[0][wave][lane], up = red[0][GT + wave][lane];
#pragma unroll
    for (int w = 1; w < kMoeWaves; ++w) {
      g += red[w][wave][lane];
      up += red[w][GT + wave][lane];
    }
    const float* weight = shared ? a.gates : a.slot_w + slot * kGemvMaxM;
    uint16_t* hb = a.h + (shared ? a.max_slots : slot) * (int64_t)(kGemvMaxM * NP) * a.inter;
    hb += 16 * (tile * GT + wave) + h_place<WQ>(lane & 15);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int tk = 4 * h + q;
      if (tk < a.m && ((entry >> (16 + tk)) & 1u) != 0) {
        float v = g[q] / (1.0f + expf(-g[q])) * up[q] * weight[tk];
        uint16_t* o = hb + (int64_t)tk * NP * inter;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const uint16_t bits = f32_half<TK>(v);
          o[i * inter] = bits;
          const float part = half_f32<TK>(bits);
          v = __builtin_isfinite(part) ? v - part : 0.0f;  // exact: the remainder of the rounding
        }
      }
    }
  }
}

// The items (expert, unit of its k) that wave `id` of `step` takes, expert by
// expert in the list's order: run r of RUN consecutive units of expert e goes
// to wave (e * runs + r) mod step.  RUN units of a column fill a cache line
// (two units of codes, one of 16-bit weights): a line is read by one wave
// (units of a line in two workgroups, on two XCDs, were read twice from memory).
// step is a power of two; the shared expert, last in the list, counts as
// expert 0 with runs of its own.
template <int RUN>
struct DownItems {
  const uint32_t* list;  // nslots entries, then the shared expert's, if any
  int slots;             // entries in all
  int shared_slot;       // its place, or one past the list
  int units, shared_units, id, step;
  int s, u;              // the current item
  uint32_t entry;

  __device__ __forceinline__ int units_of(int slot) const { return slot == shared_slot ? shared_units : units; }
  // the wave's first unit in a slot (perhaps past its last)
  __device__ __forceinline__ int first_of(int slot, uint32_t en) const {
    const int runs = (units + RUN - 1) / RUN;
    return ((slot == shared_slot ? id : id - (int)(en & 0xffffu) * runs) & (step - 1)) * RUN;
  }
  __device__ __forceinline__ int count(int lane) const {
    int n = 0;
    for (int q = lane; q < slots; q += 64) {
      const int f = first_of(q, list[q]), un = units_of(q);
      const int whole = f < un ? (un - f) / (step * RUN) : 0;  // rounds that hold a whole run
      n += f < un ? whole * RUN + min(RUN, un - f - whole * step * RUN) : 0;
    }
    return (int)wave_sum_f32((float)n);  // (exact: far below 2^24)
  }
  __device__ __forceinline__ void begin() {
    s = -1;
    u = RUN - 1;
    entry = 0;
    next();
  }
  // to the next item; past the last one it stays there
  __device__ __forceinline__ void next() {
    int ns = s, nu = u + 1;
    uint32_t ne = entry;
    if (nu % RUN == 0) nu += (step - 1) * RUN;
    while (ns < 0 || nu >= units_of(ns)) {
      if (ns + 1 >= slots) return;
      ++ns;
      ne = (uint32_t)__builtin_amdgcn_readfirstlane((int)list[ns]);
      nu = first_of(ns, ne);
    }
    s = ns;
    u = nu;
    entry = ne;
  }
};

// The scales and zero points of one unit of two adjacent tiles of 16 columns:
// even lane groups fetch the first tile's, odd ones the second's, in one load
// for the scales (2, 4 or 8 bytes of each column) and one for the zero points
// (half as many).
template <int WQ>
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

  // per tile and group: scale in the low half, zero point in the high half
  __device__ __forceinline__ void get(u32x4 (&sz)[2]) const {
    uint32_t lo = s[0], hi = 0, zz = 0;
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
    if constexpr ((WQ & kZeros) != 0) {
      zz = z >> (8 * shift);
      zs = spread4(zz);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int g = 0; g < GU; ++g) {
        const uint32_t word = g < 2 ? (uint32_t)l[c] : (uint32_t)m[c];
        const uint32_t sc = (g & 1) != 0 ? word >> 16 : word & 0xffffu;
        const uint32_t zw = zs[c];
        sz[c][g] = sc | (((zw >> (8 * g)) & 0xffu) << 16);
      }
  }
};
template <>
struct UnitScales<kWFull> {
  __device__ __forceinline__ void get(u32x4 (&)[2]) const {}
};

template <int TK, int WQ, int NP>
__global__ __launch_bounds__(64 * kMoeWaves, 2) void moe_down_kernel(MoeArgs a) {
  constexpr int CT = 2;
  constexpr int NB = unit_blocks<WQ>();
  constexpr int UL = unit_len<WQ>();
  __shared__ f32x4 red[kMoeWaves][CT][64];
  __shared__ u32x4 turn_s[kMoeWaves][turn_slots<WQ, CT, NP>() * 64];
  __shared__ uint32_t list[kGemvMaxM * SKINNY_TOPK_MAX + 1];
  __shared__ int last_s;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 4;
  const int row = lane & 15;
  // Workgroups go to the eight XCDs in turn: the shares of one column range are
  // eight apart, so they find each other's cache lines (a column's scales and
  // its ends of code lines) in one L2.
  int split, tile;
  {
    const int S = a.down_splits, b = blockIdx.x, tiles = (int)(gridDim.x / (unsigned)S);
    const int whole = tiles / 8 * 8 * S;  // workgroups of whole sets of eight ranges
    if (b < whole) {
      split = b / 8 % S;
      tile = b / (8 * S) * 8 + b % 8;
    } else {
      split = (b - whole) % S;
      tile = whole / S + (b - whole) / S;
    }
  }
  const int64_t j0 = (int64_t)tile * (16 * CT);

  int nslots = *a.nslots;
  for (int i = threadIdx.x; i < a.max_slots; i += 64 * kMoeWaves) list[i] = a.slots[i];
  nslots = __builtin_amdgcn_readfirstlane(nslots);
  __syncthreads();
  if (threadIdx.x == 0 && a.shared_inter > 0) list[nslots] = 0xffff0000u;
  __syncthreads();

  DownItems<(WQ == kWFull ? 1 : 2)> it;
  it.list = list;
  it.slots = nslots + (a.shared_inter > 0 ? 1 : 0);
  it.shared_slot = nslots;
  it.units = (int)((a.inter + UL - 1) / UL);
  it.shared_units = (int)((a.shared_inter + UL - 1) / UL);
  it.id = wave + kMoeWaves * split;
  it.step = kMoeWaves * a.down_splits;
  const int n = __builtin_amdgcn_readfirstlane(it.count(lane));

  f32x4 tot[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) tot[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  struct Item {
    WUnit<WQ, CT> w;
    UnitScales<WQ> s;
    u32x4 a[NP][NB];
  };
  // Load the current item.  A row that the expert does not serve reads zeros,
  // and so do all rows in blocks past the expert's k, where the weight reads
  // the unit's first block instead: every item is then multiplied whole, with
  // no branch between the matrix-core steps.
  auto load = [&](Item& q) __attribute__((always_inline)) {
    const bool shared = it.s == it.shared_slot;
    const int k = (int)(shared ? a.shared_inter : a.inter);
    const WindowWeight& W = shared ? a.s2 : a.w2;
    const int64_t jb = (shared ? 0 : (int64_t)(it.entry & 0xffffu) * a.d) + j0;
    int64_t j[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) j[c] = jb + 16 * c;
    WTiles<WQ, CT> t;
    w_tiles<WQ, CT>(t, W, j, k, 16, lane);
    const bool part = it.u * UL + UL > k;
    const int tk = lane >> 2, piece = lane & 3;  // this lane's token (or column) and piece of each block
    const bool served = tk < a.m && ((it.entry >> (16 + tk)) & 1u) != 0;
    const uint16_t* hr = a.h + (shared ? a.max_slots : it.s) * (int64_t)(kGemvMaxM * NP) * a.inter +
                         (int64_t)tk * NP * k + it.u * UL + 8 * piece;
    if constexpr (WQ == kWFull) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = part && it.u * UL + 32 * i >= k ? 0 : 64 * i;
#pragma unroll
        for (int c = 0; c < CT; ++c) q.w.v[c][i] = *(const u32x4*)(t.codes[c] + (int64_t)it.u * 128 + t.off + at);
      }
    } else {
      const int at = part && it.u * UL + 32 * piece >= k ? -16 * piece : 0;
#pragma unroll
      for (int c = 0; c < CT; ++c) q.w.v[c][0] = *(const u32x4*)(t.codes[c] + (int64_t)it.u * 64 + t.off + at);
      const int64_t rows = shared ? a.d - j0 : (a.experts - (int64_t)(it.entry & 0xffffu)) * a.d - j0;
      q.s.load(W, jb, 16 * (h & 1) + row, it.u, k / group_len<WQ>(), (int)min(rows, (int64_t)64));
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const uint16_t* hp = served ? hr + (int64_t)p * k : a.zero_page;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const uint16_t* hi = part && it.u * UL + 32 * i >= k ? a.zero_page : hp + 32 * i;
        q.a[p][i] = *(const u32x4*)hi;
      }
    }
  };
  const Turn turn(turn_s[wave], lane);
  auto mul = [&](Item& q) __attribute__((always_inline)) {
    u32x4 sz[CT];
    q.s.get(sz);
    turn_unit<WQ, CT, NP>(q.w, q.a, turn, lane);
    mul_unit<TK, WQ, CT, NP, true, false>(q.w, sz, q.a, tot, 0, 0);
  };

  if (n > 0) {
    Item i0, i1;
    it.begin();
    load(i0);
    it.next();  // (past the last item: the last again)
    load(i1);
    int left = n;
#pragma unroll 1
    while (left >= 4) {
      mul(i0);
      __builtin_amdgcn_sched_barrier(0);
      it.next();
      load(i0);
      __builtin_amdgcn_sched_barrier(0);
      mul(i1);
      __builtin_amdgcn_sched_barrier(0);
      it.next();
      load(i1);
      __builtin_amdgcn_sched_barrier(0);
      left -= 2;
    }
    mul(i0);
    if (left == 3) {
      it.next();
      load(i0);
    }
    if (left >= 2) mul(i1);
    if (left == 3) mul(i0);
  }

#pragma unroll
  for (int c = 0; c < CT; ++c) red[wave][c][lane] = tot[c];
  __syncthreads();
  const int64_t jc = j0 + 16 * wave + row;  // waves 0 and 1: this thread's column
  const bool mine = wave < CT;
  if (mine) {
    f32x4 sum = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kMoeWaves; ++w) sum += red[w][wave][lane];
    if (a.down_splits == 1) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (4 * h + q < a.m) store_kind(a.out, (4 * h + q) * a.ldo + jc, sum[q], a.out_kind);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (4 * h + q < a.m) st_dev(a.partial + ((int64_t)split * kGemvMaxM + 4 * h + q) * a.d + jc, sum[q]);
      wait_mem();  // this share has reached the device-coherent level
    }
  }
  if (a.down_splits > 1) {
    __syncthreads();  // every wave's share has
    if (threadIdx.x == 0) last_s = atomicAdd(&a.counters[tile], 1u) == (uint32_t)(a.down_splits - 1);
    __syncthreads();
    if (last_s && mine) {
      // every share is there: add them in order
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (4 * h + q < a.m) {
          const float* p = a.partial + (int64_t)(4 * h + q) * a.d + jc;
          float v[kMoeMaxSplits];
#pragma unroll
          for (int i = 0; i < kMoeMaxSplits; ++i)
            v[i] = ld_dev(p + (int64_t)(i < a.down_splits ? i : 0) * kGemvMaxM * a.d);
          float sum = v[0];
#pragma unroll
          for (int i = 1; i < kMoeMaxSplits; ++i) sum = i < a.down_splits ? sum + v[i] : sum;
          store_kind(a.out, (4 * h + q) * a.ldo + jc, sum, a.out_kind);
        }
      }
    }
    if (last_s && threadIdx.x == 0) a.counters[tile] = 0u;  // ready for the next call
  }
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

template <int TK, int WQ, int NP>
moe_fn pick_stage(bool up, bool wide) {
  return !up ? moe_down_kernel<TK, WQ, NP> : wide ? moe_up_kernel<TK, WQ, NP, 2> : moe_up_kernel<TK, WQ, NP, 1>;
}

template <int TK, int NP>
moe_fn pick_weight(int group, bool zeros, bool up, bool wide) {
  switch (group + (zeros ? kZeros : 0)) {
    case 0: return pick_stage<TK, kWFull, NP>(up, wide);
    case 32: return pick_stage<TK, 32, NP>(up, wide);
    case 64: return pick_stage<TK, 64, NP>(up, wide);
    case 128: return pick_stage<TK, 128, NP>(up, wide);
    case 32 + kZeros: return pick_stage<TK, 32 + kZeros, NP>(up, wide);
    case 64 + kZeros: return pick_stage<TK, 64 + kZeros, NP>(up, wide);
    default: return pick_stage<TK, 128 + kZeros, NP>(up, wide);
  }
}

moe_fn pick(int kind, int np, int group, bool zeros, bool up, bool wide) {
  return kind == CK_F16 ? pick_weight<CK_F16, 2>(group, zeros, up, wide)
         : np == 2      ? pick_weight<CK_BF16, 2>(group, zeros, up, wide)
                        : pick_weight<CK_BF16, 3>(group, zeros, up, wide);
}

}  // namespace

int moe_planes(int kind, int out_kind) { return kind == CK_BF16 && out_kind == CK_F32 ? 3 : 2; }

// Shares of the down product's k, a power of two: enough workgroups for about
// ten waves per CU of 256, but not more waves than one token's experts have
// units.  By the layer alone, which also fixes every row's order of additions.
int moe_down_splits(int64_t d, int64_t inter, int64_t shared_inter, int topk, int group) {
  const int64_t unit = group == 0 ? 64 : 128;
  const int64_t units = topk * ((inter + unit - 1) / unit) + (shared_inter + unit - 1) / unit;
  int s = 1;
  while (s < kMoeMaxSplits && d / 32 * s < 640 && s * kMoeWaves < units) s *= 2;
  return s;
}

hipError_t launch_moe(const MoeArgs& a, int kind, int group, hipStream_t stream) {
  if (a.m < 1 || a.m > kGemvMaxM || a.experts < 1 || a.experts > kMoeMaxExperts || a.topk < 1 ||
      a.topk > SKINNY_TOPK_MAX || a.topk > a.experts || a.d % 32 != 0 || a.inter % 32 != 0 || a.shared_inter % 32 != 0 ||
      (group != 0 && group != 32 && group != 64 && group != 128) ||
      (group != 0 && (a.d % group != 0 || a.inter % group != 0 || a.shared_inter % group != 0)) ||
      (kind != CK_F16 && kind != CK_BF16) || a.down_splits != moe_down_splits(a.d, a.inter, a.shared_inter, a.topk, group))
    return hipErrorInvalidValue;
  const int64_t slots = (int64_t)a.m * a.topk < a.experts ? (int64_t)a.m * a.topk : a.experts;
  if (slots > a.max_slots || a.max_slots > kGemvMaxM * SKINNY_TOPK_MAX) return hipErrorInvalidValue;
  // two column tiles of h per workgroup where that still leaves many
  // workgroups: the loads of x serve twice the columns (a column's arithmetic
  // does not depend on it)
  const bool wide = slots * (a.inter / 32) >= 2048;
  const int64_t tile = wide ? 32 : 16;
  const int64_t up_blocks = slots * (a.inter / tile) + a.shared_inter / tile;
  const int64_t down_blocks = a.d / 32 * a.down_splits;
  if (up_blocks > 0x7fffffff) return hipErrorInvalidValue;
  const int np = moe_planes(kind, a.out_kind);
  const bool zeros = a.w13.zeros != nullptr;
  const bool f16 = kind == CK_F16;
  hipLaunchKernelGGL(f16 ? pick_route<CK_F16>(a.experts) : pick_route<CK_BF16>(a.experts),
                     dim3(a.shared_inter > 0 ? 2 : 1), dim3(64 * a.m), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(pick(kind, np, group, zeros, true, wide), dim3((unsigned)up_blocks), dim3(64 * kMoeWaves), 0,
                     stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(pick(kind, np, group, zeros, false, false), dim3((unsigned)down_blocks), dim3(64 * kMoeWaves), 0,
                     stream, a);
  return hipGetLastError();
}

}  // namespace skinny
