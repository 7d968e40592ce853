// logprobs.hip -- log probabilities of given tokens from rows of logits, with
// the distribution's entropy, the token's rank and the top alternatives, for
// gfx950 (MI355X).
//
// For a row x of V logits and a token t, with M = max x, d_j = x_j - M,
// S = sum exp(d_j) and U = sum exp(d_j) d_j:
//   log p_t = d_t - ln S          entropy = ln S - U / S
//   rank    = 1 + #{j : x_j > x_t, or x_j = x_t and j < t}
// and the topk largest x_j (equal values by lower index first) with their log
// probabilities.  One pass over the logits: HBM-bound for long inputs.
//
// A workgroup of four waves owns a row (or, when there are few rows, one of a
// row's segments).  Every thread keeps a running (M, S, U) of its own and
// rescales it when its maximum grows; nothing crosses lanes until the end of
// the row.  Exponentials are base 2: S and U of exp2(d log2 e).
//
// Top-k: every wave keeps the best entries it has seen in a list over its
// lanes, lane i the i-th best, and the topk-th of them is a bar.  An entry is a
// 64-bit key: the logit's order key above, the complement of its index below,
// so one comparison ranks by value and then by lower index.  A chunk without a
// lane whose maximum reaches the bar costs one comparison.  When many lanes
// reach it (the first chunk, or logits in rising order) the topk-th largest of
// the 64 lane maxima, found bit by bit with ballots, is a better bar: at least
// topk entries are at or above it.  The entries that qualify are gathered in
// LDS; when 64 have come together they are sorted over the lanes by a bitonic
// network and merged with the list.  At the row's end the waves' entries are
// joined (see the kernel).
//
// Segments of one row leave their (M, S, U), rank count and list in the
// workspace; the last workgroup of the row to arrive joins them, in the order
// of the segments.
#include "skinny.h"
#include "wave_ops.h"
#include "window.h"

namespace skinny {

namespace {

constexpr int kNone = 0x7fffff00;  // index of an entry that holds no logit (V stays below it)
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int XK>
constexpr int vec_elems() { return XK == CK_F32 ? 4 : 8; }  // in 16 bytes

template <int XK>
__device__ __forceinline__ float to_f32(const void* p, int64_t i) {
  if constexpr (XK == CK_F32) {
    return ((const float*)p)[i];
  } else if constexpr (XK == CK_F16) {
    return (float)((const _Float16*)p)[i];
  } else {
    return f32_from_bits((uint32_t)((const uint16_t*)p)[i] << 16);
  }
}

template <int XK>
__device__ __forceinline__ void unpack(u32x4 v, float* x) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t w = v[q];
    if constexpr (XK == CK_F32) {
      x[q] = f32_from_bits(w);
    } else if constexpr (XK == CK_F16) {
      const h2_t hh = as_h2(w);
      x[2 * q] = (float)hh[0];
      x[2 * q + 1] = (float)hh[1];
    } else {
      x[2 * q] = f32_from_bits(w << 16);
      x[2 * q + 1] = f32_from_bits(w & 0xffff0000u);
    }
  }
}

typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_align4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_align2 __attribute__((ext_vector_type(4), aligned(2)));

// 16 bytes from an address that is a multiple of the element's size
template <int ES>
__device__ __forceinline__ u32x4 load16(const char* p) {
  if constexpr (ES == 4) {
    return __builtin_nontemporal_load((const u32x4_align4*)p);
  } else {
    return __builtin_nontemporal_load((const u32x4_align2*)p);
  }
}

__device__ __forceinline__ float exp2_hw(float t) { return __builtin_amdgcn_exp2f(t); }

// (M, S, U) with U in base-2 units: U = sum 2^t t, t = (x - M) log2 e
struct Soft {
  float m, s, u;
};

// the state's exponents moved to a maximum `to` >= m; a state without weight
// (m = kLowest, s = 0) stays one
__device__ __forceinline__ void rebase(Soft& a, float to) {
  const float t = fmaxf((a.m - to) * kLog2e, -16384.0f);
  const float f = exp2_hw(t);
  a.u = f * __builtin_fmaf(t, a.s, a.u);
  a.s *= f;
  a.m = to;
}

__device__ __forceinline__ Soft wave_join(Soft a) {
  rebase(a, wave_max_f32(a.m));
  a.s = wave_sum_f32(a.s);
  a.u = wave_sum_f32(a.u);
  return a;
}

// --- entries and lists -------------------------------------------------------
__device__ __forceinline__ uint64_t entry_of(float v, int i) {
  return ((uint64_t)((uint32_t)order_key(v) ^ 0x80000000u) << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float entry_value(uint64_t e) { return key_value((int)((uint32_t)(e >> 32) ^ 0x80000000u)); }
__device__ __forceinline__ int entry_index(uint64_t e) { return (int)~(uint32_t)e; }

constexpr uint32_t kKeyNegInf = 0x007fffffu;  // upper half of -inf's entry
constexpr uint32_t kKeyLowest = 0x00800000u;  // of kLowest's
constexpr uint64_t kNoEntry = ((uint64_t)kKeyNegInf << 32) | (uint32_t)~kNone;

__device__ __forceinline__ uint64_t join64(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }

// a DPP move that reads a lane for every lane: no old value is needed, which
// saves the move that would set it
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_all(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

// the value of lane ^ J
template <int J>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v, int lane) {
  if constexpr (J == 1) {
    return dpp_all<kDppXor1>(v);
  } else if constexpr (J == 2) {
    return dpp_all<kDppXor2>(v);
  } else if constexpr (J == 4) {  // 7 ^ 3
    return dpp_all<0x1B>(dpp_all<kDppRowHalfMirror>(v));
  } else if constexpr (J == 8) {  // a rotation by 8 in the row of 16
    return dpp_all<0x128>(v);
  } else if constexpr (J == 16) {
    auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (lane & 16) != 0 ? r[0] : r[1];
  } else {
    auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (lane & 32) != 0 ? r[0] : r[1];
  }
}

// lanes that keep the larger of a pair at stride J of a network of blocks of K
constexpr uint64_t keep_larger(int K, int J) {
  uint64_t m = 0;
  for (int l = 0; l < 64; ++l)
    if (((l & J) == 0) == ((l & K) == 0)) m |= 1ull << l;
  return m;
}
template <int K, int J>
__device__ __forceinline__ uint64_t exchange(uint64_t v, int lane) {
  const uint64_t o = join64(lane_xor<J>((uint32_t)v, lane), lane_xor<J>((uint32_t)(v >> 32), lane));
  const uint64_t larger = __builtin_amdgcn_ballot_w64(v > o);
  return __builtin_amdgcn_inverse_ballot_w64(~(larger ^ keep_larger(K, J))) ? v : o;
}
template <int K, int J>
__device__ __forceinline__ uint64_t exchanges(uint64_t v, int lane) {
  v = exchange<K, J>(v, lane);
  if constexpr (J > 1) v = exchanges<K, J / 2>(v, lane);
  return v;
}
// descending over the lanes
__device__ __forceinline__ uint64_t lane_sort(uint64_t v, int lane) {
  v = exchanges<2, 1>(v, lane);
  v = exchanges<4, 2>(v, lane);
  v = exchanges<8, 4>(v, lane);
  v = exchanges<16, 8>(v, lane);
  v = exchanges<32, 16>(v, lane);
  return exchanges<64, 32>(v, lane);
}
// the value of lane 63 - lane
__device__ __forceinline__ uint32_t lane_reverse(uint32_t v, int lane) {
  return lane_xor<32>(lane_xor<16>(dpp_all<kDppRowMirror>(v), lane), lane);
}

// A wave's list: lane i holds the i-th best entry; `bar` is the topk-th, and no
// logit below bar_value can be among the topk best any more (wave-uniform).
struct List {
  uint64_t e;
  uint64_t bar;
  float bar_value;
};

__device__ __forceinline__ void list_bar(List& l, int topk) {
  l.bar = join64(__builtin_amdgcn_readlane((uint32_t)l.e, topk - 1),
                 __builtin_amdgcn_readlane((uint32_t)(l.e >> 32), topk - 1));
  l.bar_value = fmaxf(l.bar_value, entry_value(l.bar));
}

__device__ __forceinline__ void list_clear(List& l) {
  l.e = l.bar = kNoEntry;
  l.bar_value = -__builtin_inff();
}

// add 64 entries that descend over the lanes
__device__ __forceinline__ void list_merge_sorted(List& l, uint64_t e, int topk, int lane) {
  const uint64_t r = join64(lane_reverse((uint32_t)e, lane), lane_reverse((uint32_t)(e >> 32), lane));
  l.e = exchanges<64, 32>(l.e > r ? l.e : r, lane);  // the 64 best of both, a bitonic sequence
  list_bar(l, topk);
}

// entries waiting to be added: n in a wave's part of LDS
constexpr int kPending = 64 + 4 * 64;
constexpr int kPoolTopk = 10;
constexpr int kPendingEnd = 64 + 64;  // at a row's end: 64 from the steps, then one logit per lane
struct Pending {
  uint64_t* e;
  int n;
};

__device__ __forceinline__ void list_flush(List& l, Pending& p, int topk, int lane) {
  wave_lds_order();
#pragma unroll 1
  for (int i = 0; i < p.n; i += 64)
    list_merge_sorted(l, lane_sort(i + lane < p.n ? p.e[i + lane] : kNoEntry, lane), topk, lane);
  p.n = 0;
  wave_lds_order();
}

// A bar from the lanes' values: at least topk of them are at or above it.  The
// topk-th largest order key, found bit by bit in its upper 16 bits (the lower
// ones would only save a few candidates).
__device__ __forceinline__ float bar_of_lanes(float v, int topk) {
  const uint32_t key = (uint32_t)order_key(v) ^ 0x80000000u;
  uint32_t t = 0;
#pragma unroll
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t c = t | (1u << bit);
    t = __builtin_popcountll(__builtin_amdgcn_ballot_w64(key >= c)) >= topk ? c : t;
  }
  t = t <= kKeyLowest ? kKeyNegInf : t;  // a running maximum starts at kLowest: no logit stands for that
  return key_value((int)(t ^ 0x80000000u));
}

// N logits per lane into the running state, the list and the rank count.
// idx[q]: index of x[q * per], or kNone where a lane has none (x = -inf there).
// where: -1 all indices lie before the token, 1 after it, 0 neither.
template <int N, int PER>
__device__ __forceinline__ void take(const float (&x)[N], const int (&idx)[N / PER], Soft& a, List& l, Pending& pend,
                                     int& above, float xt, int tok, int where, int topk, int lane) {
  float top = x[0];
#pragma unroll
  for (int e = 1; e < N; ++e) top = fmaxf(top, x[e]);
  rebase(a, fmaxf(a.m, top));
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float t = (x[e] - a.m) * kLog2e;
    const float p = exp2_hw(t);  // 0 for -inf, NaN for NaN and (M = inf) infinity
    a.s += p;
    a.u = __builtin_fmaf(p, fmaxf(t, -16384.0f), a.u);  // 0 for -inf
  }
  if (where < 0) {
#pragma unroll
    for (int e = 0; e < N; ++e) above += __builtin_popcountll(__builtin_amdgcn_ballot_w64(x[e] >= xt));
  } else if (where > 0) {
#pragma unroll
    for (int e = 0; e < N; ++e) above += __builtin_popcountll(__builtin_amdgcn_ballot_w64(x[e] > xt));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      above += __builtin_popcountll(
          __builtin_amdgcn_ballot_w64(x[e] > xt || (x[e] == xt && idx[e / PER] + e % PER < tok)));
  }
  if (topk > 0) {
    const uint64_t b = __builtin_amdgcn_ballot_w64(top >= l.bar_value);
    if (b != 0) {
      // Every lane's maximum so far, where it reaches the lanes' bar, has been
      // gathered or is gathered below, and so have topk entries at least: the
      // bar can replace a lower one before they reach the list.
      if (__builtin_popcountll(b) > 8) l.bar_value = fmaxf(l.bar_value, bar_of_lanes(a.m, topk));
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (__builtin_amdgcn_ballot_w64(x[e] >= l.bar_value) != 0) {  // uniform
          const uint64_t en = entry_of(x[e], idx[e / PER] + e % PER);
          const bool in = x[e] >= l.bar_value && en > l.bar;  // (false for NaN)
          const uint64_t q = __builtin_amdgcn_ballot_w64(in);
          if (in) pend.e[pend.n + __builtin_popcountll(q & ((1ull << lane) - 1))] = en;
          pend.n += __builtin_popcountll(q);
        }
        if (e % 4 == 3 && pend.n > 64) list_flush(l, pend, topk, lane);  // (room for four more times 64)
      }
    }
  }
}

template <int XK, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void logprobs_kernel(LogprobArgs g) {
  constexpr int kThreads = 64 * kWaves;
  constexpr int VE = vec_elems<XK>();
  constexpr int NV = 16 / VE;  // 16 logits per thread and step
  constexpr int ES = XK == CK_F32 ? 4 : 2;
  __shared__ Soft soft_s[kWaves];
  __shared__ int above_s[kWaves];
  __shared__ uint64_t pending_s[kWaves][kPending];
  constexpr int kPool = kWaves * (SKINNY_TOPK_MAX + kPendingEnd);
  __shared__ uint64_t pool_s[kPool] __attribute__((aligned(16)));  // entries of all waves
  __shared__ int place_s[kPool];
  __shared__ uint64_t best_s[SKINNY_TOPK_MAX];
  __shared__ uint32_t bar_s[kLogprobMaxSegments];  // (segments or waves)
  __shared__ int pool_n;
  __shared__ int last_s;
  static_assert(kPool >= kLogprobMaxSegments * kPoolTopk && kLogprobMaxSegments >= kWaves,
                "the pool holds the waves' entries, or the segments'");
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int topk = g.topk;
  const uint32_t row_index = blockIdx.x / (uint32_t)g.segments;
  const int64_t r = row_index;
  const int seg = (int)(blockIdx.x - row_index * (uint32_t)g.segments);
  const char* row = (const char*)g.logits + r * g.ld * ES;

  // this segment: first .. first + len - 1, in vectors of 16 bytes and, after
  // them, single logits.  A row may start at any element; its vectors are then
  // loaded unaligned (global loads take any alignment here), so which thread
  // adds which logits, hence every bit of the result, does not depend on it.
  const int first = seg * g.seg_len;
  const int len = min(g.seg_len, (int)g.vocab - first);
  const int nvec = len / VE;
  const char* vec = row + (int64_t)first * ES;

  Soft a = {kLowest, 0.0f, 0.0f};
  List l;
  list_clear(l);
  Pending pend = {pending_s[wave], 0};
  int above = 0;

  u32x4 raw[NV];  // the first loads are on their way before anything waits
#pragma unroll
  for (int q = 0; q < NV; ++q)
    if (q * kThreads + tid < nvec) raw[q] = load16<ES>(vec + (int64_t)(q * kThreads + tid) * 16);
  // the token and its logit; a token outside the row has none
  const int64_t token = g.tokens64 ? ((const int64_t*)g.tokens)[r] : (int64_t)((const int32_t*)g.tokens)[r];
  const bool known = token >= 0 && token < g.vocab;
  const int tok = known ? (int)token : 0;
  const float xt = to_f32<XK>(row, tok);

  for (int c = 0; c < nvec; c += NV * kThreads) {
    float x[NV * VE];
    int idx[NV];
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int v = c + q * kThreads + tid;
      unpack<XK>(raw[q], &x[q * VE]);
      idx[q] = first + v * VE;
    }
    const bool full = c + NV * kThreads <= nvec;  // uniform: only the last step is not
    if (!full) {
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const bool out = c + q * kThreads + tid >= nvec;
        idx[q] = out ? kNone : idx[q];
#pragma unroll
        for (int e = 0; e < VE; ++e) x[q * VE + e] = out ? -__builtin_inff() : x[q * VE + e];
      }
    }
#pragma unroll
    for (int q = 0; q < NV; ++q) {  // the next step's logits are on their way during this one's work
      const int v = c + (NV + q) * kThreads + tid;
      if (v < nvec) raw[q] = load16<ES>(vec + (int64_t)v * 16);
    }
    const int i0 = first + c * VE, i1 = i0 + NV * kThreads * VE;
    const int where = !full ? 0 : i1 <= tok ? -1 : i0 > tok ? 1 : 0;
    take<NV * VE, VE>(x, idx, a, l, pend, above, xt, tok, where, topk, lane);
  }
  if (wave == 0 && len % VE != 0) {  // the last logits
    const int i = lane < len % VE ? first + nvec * VE + lane : kNone;
    float x[1] = {-__builtin_inff()};
    if (i != kNone) x[0] = to_f32<XK>(row, i);
    const int idx[1] = {i};
    take<1, 1>(x, idx, a, l, pend, above, xt, tok, 0, topk, lane);
  }

  // The topk best of what the waves (later: the segments) hold, in two ways.  Up
  // to kPoolTopk: the entries that reach the highest of their bars go into a pool,
  // in any order, and an entry's place is the number of larger ones.  Beyond: each
  // wave sorts its entries, and sorted lists are merged in turn.  Measured (us,
  // pool / merged): 512 x 50021 f16, top 1 20.2 / 22.2, top 10 24.7 / 25.3; 1 x 50021
  // f16, top 1 8.4 / 10.3, top 10 10.0 / 10.8, top 20 13.7 / 11.1; 16 x 131071 bf16, top
  // 20, 18.4 / 14.4.
  const bool merged = topk > kPoolTopk;
  auto pool_clear = [&]() __attribute__((always_inline)) {
    if (tid < topk) best_s[tid] = kNoEntry;
    if (tid == 0) pool_n = 0;
  };
  auto pool_put = [&](uint64_t e, bool in) __attribute__((always_inline)) {
    const uint64_t q = __builtin_amdgcn_ballot_w64(in);
    if (q == 0) return;
    int at = 0;
    if (lane == 0) at = atomicAdd(&pool_n, __builtin_popcountll(q));
    at = __builtin_amdgcn_readfirstlane(at) + __builtin_popcountll(q & ((1ull << lane) - 1));
    if (in) {
      pool_s[at] = e;
      place_s[at] = 0;
    }
  };
  // (every wave counts the larger ones of its share of the pool, for all entries)
  auto pool_rank = [&]() __attribute__((always_inline)) {
    const int n = pool_n, per = ((n + kWaves - 1) / kWaves + 1) & ~1;
    const int k0 = min(wave * per, n), k1 = min(k0 + per, n);
    for (int i = lane; i < n; i += 64) {
      const uint64_t e = pool_s[i];
      int larger = 0;
      int k = k0;
#pragma unroll 4
      for (; k + 2 <= k1; k += 2) {
        const u64x2 v = *(const u64x2*)&pool_s[k];
        larger += (v[0] > e ? 1 : 0) + (v[1] > e ? 1 : 0);
      }
      if (k < k1) larger += pool_s[k] > e ? 1 : 0;
      if (larger != 0) atomicAdd(&place_s[i], larger);
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads)
      if (place_s[i] < topk) best_s[place_s[i]] = pool_s[i];
    __syncthreads();
  };
  auto highest_bar = [&](int n) __attribute__((always_inline)) {
    uint32_t bar = kKeyNegInf;
#pragma unroll
    for (int q = 0; q < kLogprobMaxSegments; ++q) bar = q < n ? max(bar, bar_s[q]) : bar;
    return bar;
  };

  // the lists of waves 1 .. kWaves - 1, which lie in the pool's place, into wave 0's
  auto merge_put = [&]() __attribute__((always_inline)) {
    if (wave > 0 && lane < topk) pool_s[wave * SKINNY_TOPK_MAX + lane] = l.e;
  };
  auto merge_waves = [&]() __attribute__((always_inline)) {
    if (wave == 0) {
#pragma unroll
      for (int q = 1; q < kWaves; ++q)
        list_merge_sorted(l, lane < topk ? pool_s[q * SKINNY_TOPK_MAX + lane] : kNoEntry, topk, lane);
    }
  };

  if (merged) {
    if (pend.n > 0) list_flush(l, pend, topk, lane);
    merge_put();
  }
  pool_clear();
  a = wave_join(a);
  if (lane == 0) {
    soft_s[wave] = a;
    above_s[wave] = above;
    bar_s[wave] = (uint32_t)order_key(l.bar_value) ^ 0x80000000u;
  }
  wave_lds_order();
  __syncthreads();
  if (merged) {
    merge_waves();
  } else if (topk > 0) {
    const uint32_t bar = highest_bar(kWaves);
    pool_put(l.e, lane < topk && l.e > kNoEntry && (uint32_t)(l.e >> 32) >= bar);
    for (int i = 0; i < pend.n; i += 64) {
      const uint64_t e = i + lane < pend.n ? pend.e[i + lane] : 0;
      pool_put(e, (uint32_t)(e >> 32) >= bar);
    }
    __syncthreads();
    pool_rank();
  }
  if (wave == 0) {
    Soft b = {kLowest, 0.0f, 0.0f};
    int n = 0;
    if (lane < kWaves) {
      b = soft_s[lane];
      n = above_s[lane];
    }
    a = wave_join(b);
    above = 0;
#pragma unroll
    for (int q = 0; q < kWaves; ++q) above += (int)__builtin_amdgcn_readlane((uint32_t)n, q);
    if (!merged && lane < topk) l.e = best_s[lane];
  }

  if (g.segments > 1) {
    const int stride = 4 + 2 * topk;
    float* part = g.partial + ((int64_t)r * g.segments) * stride;
    if (wave == 0) {
      float* mine = part + (int64_t)seg * stride;
      if (lane == 0) {
        st_dev(mine, a.m);
        st_dev(mine + 1, a.s);
        st_dev(mine + 2, a.u);
        st_dev(mine + 3, fbits((uint32_t)above));
      }
      if (lane < topk) {
        st_dev(mine + 4 + lane, fbits((uint32_t)l.e));
        st_dev(mine + 4 + topk + lane, fbits((uint32_t)(l.e >> 32)));
      }
      wait_mem();  // this segment has reached the device-coherent level
      if (lane == 0) last_s = atomicAdd(&g.counters[r], 1u) == (uint32_t)(g.segments - 1);
    }
    __syncthreads();
    if (!last_s) return;
    // the last workgroup of the row: every segment is there
    a = Soft{kLowest, 0.0f, 0.0f};
    above = 0;
    if (tid < g.segments) {  // one segment per thread of wave 0
      const float* p = part + (int64_t)tid * stride;
      a = Soft{ld_dev(p), ld_dev(p + 1), ld_dev(p + 2)};
      above = (int)ubits(ld_dev(p + 3));
    }
    if (merged) {
      // wave w takes segments w, w + kWaves, ...: each list descends over its lanes
      constexpr int R = kLogprobMaxSegments / kWaves;
      uint32_t lo[R], hi[R];
#pragma unroll
      for (int q = 0; q < R; ++q) {  // every load before the first merge
        const int sg = q * kWaves + wave;
        const float* p = part + (int64_t)(sg < g.segments ? sg : 0) * stride + 4 + (lane < topk ? lane : 0);
        lo[q] = ubits(ld_dev(p));
        hi[q] = ubits(ld_dev(p + topk));
      }
      list_clear(l);
#pragma unroll
      for (int q = 0; q < R; ++q)
        if (q * kWaves + wave < g.segments) list_merge_sorted(l, lane < topk ? join64(lo[q], hi[q]) : kNoEntry, topk, lane);
      merge_put();
      __syncthreads();
      merge_waves();
    } else if (topk > 0) {
      // one entry per thread, segment by segment
      constexpr int R = (kLogprobMaxSegments * kPoolTopk + kThreads - 1) / kThreads;
      uint64_t e[R];
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int i = q * kThreads + tid, sg = i / topk, at = i - sg * topk;
        e[q] = 0;
        if (sg < g.segments) {
          const float* p = part + (int64_t)sg * stride + 4 + at;
          e[q] = join64(ubits(ld_dev(p)), ubits(ld_dev(p + topk)));
          if (at == topk - 1) bar_s[sg] = (uint32_t)(e[q] >> 32);
        }
      }
      pool_clear();
      __syncthreads();
      const uint32_t bar = highest_bar(g.segments);
#pragma unroll
      for (int q = 0; q < R; ++q) pool_put(e[q], e[q] > kNoEntry && (uint32_t)(e[q] >> 32) >= bar);
      __syncthreads();
      pool_rank();
      if (lane < topk) l.e = best_s[lane];
    }
    if (wave == 0) {
      a = wave_join(a);
      // the sum over lanes (counts fit: below 2^31 in all)
      above += dpp_mov_i<kDppXor1>(above);
      above += dpp_mov_i<kDppXor2>(above);
      above += dpp_mov_i<kDppRowHalfMirror>(above);
      above += dpp_mov_i<kDppRowMirror>(above);
      above = (int)(__builtin_amdgcn_readlane((uint32_t)above, 0) + __builtin_amdgcn_readlane((uint32_t)above, 16) +
                    __builtin_amdgcn_readlane((uint32_t)above, 32) + __builtin_amdgcn_readlane((uint32_t)above, 48));
    }
    if (tid == 0) g.counters[r] = 0u;  // ready for the next call
  }

  if (wave == 0) {
    // a row whose logits are all -inf has no distribution: log probabilities
    // of -inf and an entropy of 0
    const float nan = __builtin_nanf(""), ninf = -__builtin_inff();
    const bool none = a.s == 0.0f;
    const float ln_s = logf(a.s);
    if (lane == 0) {
      g.logprob[r] = !known ? nan : none ? ninf : (xt - a.m) - ln_s;
      g.entropy[r] = none ? 0.0f : ln_s - kLn2 * (a.u / a.s);
      g.rank[r] = known ? 1 + above : 0;
    }
    if (lane < topk) {
      const int i = entry_index(l.e);
      g.top_ids[r * topk + lane] = i == kNone ? -1 : i;
      g.top_logprobs[r * topk + lane] = none ? ninf : (entry_value(l.e) - a.m) - ln_s;
    }
  }
}

}  // namespace

hipError_t launch_logprobs(const LogprobArgs& a, int x_kind, hipStream_t stream) {
  if (a.m < 1 || a.vocab < 1 || a.vocab > (1 << 30) || a.topk < 0 || a.topk > SKINNY_TOPK_MAX || a.topk > a.vocab ||
      a.segments < 1 || a.segments > kLogprobMaxSegments || a.seg_len < 1 ||
      (int64_t)a.segments * a.seg_len < a.vocab || (int64_t)(a.segments - 1) * a.seg_len >= a.vocab ||
      a.m * a.segments > 0x7fffffff)
    return hipErrorInvalidValue;
  if (a.waves != 4 && a.waves != 8) return hipErrorInvalidValue;
  constexpr int64_t most = kMaxLaunchThreads / (64 * 8);  // rows of a launch
  if (a.m > most) {
    if (a.segments != 1) return hipErrorInvalidValue;
    LogprobArgs part = a;
    for (int64_t r = 0; r < a.m; r += most) {
      part.m = a.m - r < most ? a.m - r : most;
      part.logits = (const char*)a.logits + r * a.ld * (x_kind == CK_F32 ? 4 : 2);
      part.tokens = (const char*)a.tokens + r * (a.tokens64 ? 8 : 4);
      part.logprob = a.logprob + r;
      part.entropy = a.entropy + r;
      part.rank = a.rank + r;
      if (a.topk > 0) {
        part.top_ids = a.top_ids + r * a.topk;
        part.top_logprobs = a.top_logprobs + r * a.topk;
      }
      const hipError_t e = launch_logprobs(part, x_kind, stream);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const bool eight = a.waves == 8;
  const auto fn = x_kind == CK_F32   ? (eight ? logprobs_kernel<CK_F32, 8> : logprobs_kernel<CK_F32, 4>)
                  : x_kind == CK_F16 ? (eight ? logprobs_kernel<CK_F16, 8> : logprobs_kernel<CK_F16, 4>)
                                     : (eight ? logprobs_kernel<CK_BF16, 8> : logprobs_kernel<CK_BF16, 4>);
  hipLaunchKernelGGL(fn, dim3((unsigned)(a.m * a.segments)), dim3(64 * a.waves), 0, stream, a);
  return hipGetLastError();
}

}  // namespace skinny
