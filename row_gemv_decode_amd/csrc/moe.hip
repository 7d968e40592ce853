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
//   moe_route_kernel  one workgroup, one wave per token: top-k, softmax, the
//                     shared expert's gate, and the list of distinct experts
//                     in ascending order with each one's tokens
//   moe_up_kernel     one workgroup per (distinct expert, 16 columns of h):
//                     gate and up columns side by side against all rows of x
//                     (a matrix-core tile holds 16 rows anyway, so tokens are
//                     not gathered), p and silu in the epilogue
//   moe_down_kernel   one workgroup per 16 columns of the layer's output, over
//                     all distinct experts: a row that an expert does not
//                     serve is a row of zeros, so the matrix core adds the
//                     experts of every token by itself, and the combine costs
//                     nothing
// h is kept exactly enough to lose nothing against fp32: as the sum of two
// f16 (22 bits) or three bf16 (24 bits) planes, multiplied one after another;
// the matrix cores have time for it while the weights stream.
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

constexpr int kMoeWaves = 8;
constexpr int kRouteCols = kMoeMaxExperts / 64;  // logits per lane

template <int TK>
constexpr int planes() { return TK == CK_F16 ? 2 : 3; }

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

// One workgroup of m waves.  Each round of a wave's top-k takes the largest
// remaining order key of the row (ties: the lowest column); lane i keeps the
// i-th winner.  The softmax sums in a fixed order: over the winners lane by
// lane, or over all logits.
template <int TK>
__global__ __launch_bounds__(1024) void moe_route_kernel(MoeArgs a) {
  __shared__ uint32_t mask[kMoeMaxExperts];     // tokens of each expert
  __shared__ int slot_of[kMoeMaxExperts];
  __shared__ int win_e[kGemvMaxM][SKINNY_TOPK_MAX];
  __shared__ float win_p[kGemvMaxM][SKINNY_TOPK_MAX];
  __shared__ float gate[kGemvMaxM];
  __shared__ int nslots_s;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int t = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int E = a.experts;
  for (int e = tid; e < E; e += blockDim.x) mask[e] = 0;
  __syncthreads();

  {
    const float* row = a.logits + (int64_t)t * E;
    float x[kRouteCols];
    int key[kRouteCols];
#pragma unroll
    for (int u = 0; u < kRouteCols; ++u) x[u] = lane + 64 * u < E ? row[lane + 64 * u] : 0.0f;
#pragma unroll
    for (int u = 0; u < kRouteCols; ++u) key[u] = lane + 64 * u < E ? order_key(x[u]) : (int)0x80000000;
    float top = 0.0f, mine = 0.0f;
    int mine_e = 0;
    for (int i = 0; i < a.topk; ++i) {
      int best = key[0];
#pragma unroll
      for (int u = 1; u < kRouteCols; ++u) best = max(best, key[u]);
      const int kmax = wave_max_i32(best);
      int col = 0x7fffffff;
#pragma unroll
      for (int u = kRouteCols - 1; u >= 0; --u) col = key[u] == kmax ? lane + 64 * u : col;
      // (a NaN logit may leave no column below E: keep the index in range)
      const int e = min(wave_min_i32(col), E - 1);
#pragma unroll
      for (int u = 0; u < kRouteCols; ++u) key[u] = lane + 64 * u == e ? (int)0x80000000 : key[u];
      const float v = row[e];
      if (i == 0) top = v;
      mine = lane == i ? v : mine;
      mine_e = lane == i ? e : mine_e;
    }
    const float ex = lane < a.topk ? expf(mine - top) : 0.0f;
    float total = 0.0f;
    if (a.renorm) {
      total = wave_sum_f32(ex);
    } else {
#pragma unroll
      for (int u = 0; u < kRouteCols; ++u) total += lane + 64 * u < E ? expf(x[u] - top) : 0.0f;
      total = wave_sum_f32(total);
    }
    const float p = ex / total;
    if (lane < a.topk) {
      win_e[t][lane] = mine_e;
      win_p[t][lane] = p;
      atomicOr(&mask[mine_e], 1u << t);
      if (a.topk_idx != nullptr) a.topk_idx[t * a.topk + lane] = mine_e;
      if (a.topk_weight != nullptr) a.topk_weight[t * a.topk + lane] = p;
    }
  }
  if (a.shared_inter > 0) {
    const uint16_t* xr = (const uint16_t*)a.x + t * a.ldx;
    const uint16_t* wr = (const uint16_t*)a.shared_gate;
    float s = 0.0f;
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
    if (lane == 0) gate[t] = 1.0f / (1.0f + expf(-s));
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
    if (lane == 0) {
      nslots_s = n;
      *a.nslots = n;
    }
  }
  __syncthreads();
  const int n = nslots_s;
  for (int i = tid; i < (n + 1) * kGemvMaxM; i += blockDim.x) {
    // the shared expert's weights come last
    const int row = i & (kGemvMaxM - 1);
    a.slot_w[i] = (i >= n * kGemvMaxM && a.shared_inter > 0 && row < a.m) ? gate[row] : 0.0f;
  }
  __syncthreads();  // (orders this workgroup's global writes too: the next ones overwrite some)
  if (lane < a.topk) a.slot_w[slot_of[win_e[t][lane]] * kGemvMaxM + t] = win_p[t][lane];
}

// columns of w13: gate columns 0 .. inter - 1, up columns inter .. 2 inter - 1
template <int TK, int WQ>
__global__ __launch_bounds__(64 * kMoeWaves) void moe_up_kernel(MoeArgs a) {
  constexpr int UB = WQ == kWFull ? 2 : 3;
  constexpr int NP = planes<TK>();
  __shared__ f32x4 red[kMoeWaves][2][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 4;
  const int k = (int)a.d;
  const int nslots = *a.nslots;
  const int tiles = (int)a.inter / 16;

  // the shared expert's workgroups come first: they are sure to have work
  const int shared_tiles = (int)a.shared_inter / 16;
  const bool shared = (int)blockIdx.x < shared_tiles;
  const int b = (int)blockIdx.x - shared_tiles;
  const int slot = shared ? nslots : b / tiles;
  if (!shared && slot >= nslots) return;
  const int tile = shared ? (int)blockIdx.x : b - slot * tiles;
  const int64_t inter = shared ? a.shared_inter : a.inter;
  const uint32_t entry = shared ? 0xffff0000u : a.slots[slot];  // every token goes to the shared expert
  const int64_t e = (int64_t)(entry & 0xffffu);
  const WindowWeight& W = shared ? a.s13 : a.w13;

  const int row = (lane & 15) < a.m ? (lane & 15) : a.m - 1;
  const uint16_t* arow = (const uint16_t*)a.x + row * a.ldx + 8 * h;
  WCol<WQ> col[2];
  const int64_t j = e * 2 * inter + 16 * tile + (lane & 15);
  col[0] = w_col<WQ>(W.codes, W.scales, W.zeros, j, a.d, h);
  col[1] = w_col<WQ>(W.codes, W.scales, W.zeros, j + inter, a.d, h);
  f32x4 tot[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};

  const int units = k / kUnit;
  for (int u = wave; u < units; u += kMoeWaves * UB) {
    WRaw<WQ> w[UB][2];
    u32x4 x[UB][1][4];
#pragma unroll
    for (int q = 0; q < UB; ++q) {
      if (u + q * kMoeWaves < units) {  // wave-uniform
        load_unit<WQ, false>(w[q][0], col[0], u + q * kMoeWaves, k, h);
        load_unit<WQ, false>(w[q][1], col[1], u + q * kMoeWaves, k, h);
        load_a_unit<false>(x[q][0], arow, u + q * kMoeWaves, k);
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // every load above is issued before the first product
#pragma unroll
    for (int q = 0; q < UB; ++q)
      if (u + q * kMoeWaves < units) mul_unit<TK, WQ, 2, 1, false>(w[q], x[q], tot, u + q * kMoeWaves, k);
  }
  if (k % kUnit != 0 && wave == units % kMoeWaves) {
    WRaw<WQ> w[2];
    u32x4 x[1][4];
    load_unit<WQ, true>(w[0], col[0], units, k, h);
    load_unit<WQ, true>(w[1], col[1], units, k, h);
    load_a_unit<true>(x[0], arow, units, k);
    mul_unit<TK, WQ, 2, 1, true>(w, x, tot, units, k);
  }
  red[wave][0][lane] = tot[0];
  red[wave][1][lane] = tot[1];
  __syncthreads();
  if (wave == 0) {
    f32x4 g = red[0][0][lane], up = red[0][1][lane];
#pragma unroll
    for (int w = 1; w < kMoeWaves; ++w) {
      g += red[w][0][lane];
      up += red[w][1][lane];
    }
    uint16_t* hb = a.h + (shared ? (int64_t)a.max_slots * kGemvMaxM * NP * a.inter : (int64_t)slot * kGemvMaxM * NP * inter);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = 4 * h + q;
      if (t < a.m && ((entry >> (16 + t)) & 1u) != 0) {
        const float p = a.slot_w[slot * kGemvMaxM + t];
        float v = g[q] / (1.0f + expf(-g[q])) * up[q] * p;
        uint16_t* o = hb + (int64_t)t * NP * inter + 16 * tile + (lane & 15);
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

// One expert's share of one wave: units u, u + kMoeWaves, ... of its k = inter
template <int TK, int WQ>
__device__ __forceinline__ void down_expert(const WCol<WQ>& col, const uint16_t* hrow, bool served, int64_t inter, int u0,
                                            int h, f32x4 (&tot)[1]) {
  constexpr int NP = planes<TK>();
  const int k = (int)inter;
  for (int u = u0; u * kUnit < k; u += kMoeWaves) {
    const bool part = u * kUnit + kUnit > k;
    WRaw<WQ> w[1];
    u32x4 x[NP][4];
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[p][i] = u32x4{0u, 0u, 0u, 0u};
    if (!part) {
      load_unit<WQ, false>(w[0], col, u, k, h);
      if (served) {
#pragma unroll
        for (int p = 0; p < NP; ++p) load_a_unit<false>(x[p], hrow + p * inter, u, k);
      }
      mul_unit<TK, WQ, 1, NP, false>(w, x, tot, u, k);
    } else {
      load_unit<WQ, true>(w[0], col, u, k, h);
      if (served) {
#pragma unroll
        for (int p = 0; p < NP; ++p) load_a_unit<true>(x[p], hrow + p * inter, u, k);
      }
      mul_unit<TK, WQ, 1, NP, true>(w, x, tot, u, k);
    }
  }
}

template <int TK, int WQ>
__global__ __launch_bounds__(64 * kMoeWaves) void moe_down_kernel(MoeArgs a) {
  constexpr int NP = planes<TK>();
  __shared__ f32x4 red[kMoeWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 4;
  const int row = lane & 15;
  const int64_t j = (int64_t)blockIdx.x * 16 + (lane & 15);
  const int nslots = *a.nslots;
  const int units = (int)((a.inter + kUnit - 1) / kUnit);
  f32x4 tot[1] = {{0.0f, 0.0f, 0.0f, 0.0f}};
  for (int s = 0; s < nslots; ++s) {
    const uint32_t entry = __builtin_amdgcn_readfirstlane(a.slots[s]);
    const int e = (int)(entry & 0xffffu);
    // wave (e * units + u) mod kMoeWaves takes unit u of expert e
    const int u0 = (wave - e * units) & (kMoeWaves - 1);
    const WCol<WQ> col = w_col<WQ>(a.w2.codes, a.w2.scales, a.w2.zeros, (int64_t)e * a.d + j, a.inter, h);
    const uint16_t* hrow = a.h + ((int64_t)s * kGemvMaxM + row) * NP * a.inter + 8 * h;
    down_expert<TK, WQ>(col, hrow, ((entry >> (16 + row)) & 1u) != 0, a.inter, u0, h, tot);
  }
  if (a.shared_inter > 0) {
    const WCol<WQ> col = w_col<WQ>(a.s2.codes, a.s2.scales, a.s2.zeros, j, a.shared_inter, h);
    const uint16_t* hrow =
        a.h + (int64_t)a.max_slots * kGemvMaxM * NP * a.inter + (int64_t)row * NP * a.shared_inter + 8 * h;
    down_expert<TK, WQ>(col, hrow, row < a.m, a.shared_inter, wave, h, tot);
  }
  red[wave][lane] = tot[0];
  __syncthreads();
  if (wave == 0) {
    f32x4 sum = red[0][lane];
#pragma unroll
    for (int w = 1; w < kMoeWaves; ++w) sum += red[w][lane];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (4 * h + q < a.m) store_kind(a.out, (4 * h + q) * a.ldo + j, sum[q], a.out_kind);
  }
}

typedef void (*moe_fn)(MoeArgs);

template <int TK>
moe_fn pick_up(int group) {
  return group == 0    ? moe_up_kernel<TK, kWFull>
         : group == 32 ? moe_up_kernel<TK, 32>
         : group == 64 ? moe_up_kernel<TK, 64>
                       : moe_up_kernel<TK, 128>;
}

template <int TK>
moe_fn pick_down(int group) {
  return group == 0    ? moe_down_kernel<TK, kWFull>
         : group == 32 ? moe_down_kernel<TK, 32>
         : group == 64 ? moe_down_kernel<TK, 64>
                       : moe_down_kernel<TK, 128>;
}

}  // namespace

int moe_planes(int kind) { return kind == CK_F16 ? planes<CK_F16>() : planes<CK_BF16>(); }

hipError_t launch_moe(const MoeArgs& a, int kind, int group, hipStream_t stream) {
  if (a.m < 1 || a.m > kGemvMaxM || a.experts < 1 || a.experts > kMoeMaxExperts || a.topk < 1 ||
      a.topk > SKINNY_TOPK_MAX || a.topk > a.experts || a.d % 32 != 0 || a.inter % 32 != 0 || a.shared_inter % 32 != 0 ||
      (group != 0 && group != 32 && group != 64 && group != 128) ||
      (group != 0 && (a.d % group != 0 || a.inter % group != 0 || a.shared_inter % group != 0)) ||
      (kind != CK_F16 && kind != CK_BF16))
    return hipErrorInvalidValue;
  const int64_t slots = (int64_t)a.m * a.topk < a.experts ? (int64_t)a.m * a.topk : a.experts;
  const int64_t up_blocks = slots * (a.inter / 16) + a.shared_inter / 16;
  if (slots > a.max_slots || up_blocks > 0x7fffffff) return hipErrorInvalidValue;
  const bool f16 = kind == CK_F16;
  hipLaunchKernelGGL(f16 ? moe_route_kernel<CK_F16> : moe_route_kernel<CK_BF16>, dim3(1), dim3(64 * a.m), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(f16 ? pick_up<CK_F16>(group) : pick_up<CK_BF16>(group), dim3((unsigned)up_blocks),
                     dim3(64 * kMoeWaves), 0, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(f16 ? pick_down<CK_F16>(group) : pick_down<CK_BF16>(group), dim3((unsigned)(a.d / 16)),
                     dim3(64 * kMoeWaves), 0, stream, a);
  return hipGetLastError();
}

}  // namespace skinny
