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
// Top-k: every wave keeps the best candidates it has seen in a list over its
// lanes, lane i the i-th best, and the topk-th of them is a bar.  A chunk
// without a lane whose maximum reaches the bar costs one comparison.  Entries
// above it are inserted one by one: a ballot finds the place, a DPP shift
// makes room.  When many lanes reach the bar at once (the first chunk, or
// logits in rising order) the topk-th largest of the 64 lane maxima, found bit
// by bit with ballots, is a better bar: at least topk entries are above it.
//
// Segments of one row leave their (M, S, U), rank count and list in the
// workspace; the last workgroup of the row to arrive joins them, in the order
// of the segments.
#include "skinny.h"
#include "wave_ops.h"
#include "window.h"

namespace skinny {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
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

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_mov<kDppXor1>(v);
  v += dpp_mov<kDppXor2>(v);
  v += dpp_mov<kDppRowHalfMirror>(v);
  v += dpp_mov<kDppRowMirror>(v);
  auto r16 = __builtin_amdgcn_permlane16_swap(ubits(v), ubits(v), false, false);
  v = fbits(r16[0]) + fbits(r16[1]);
  auto r32 = __builtin_amdgcn_permlane32_swap(ubits(v), ubits(v), false, false);
  return fbits(r32[0]) + fbits(r32[1]);
}

__device__ __forceinline__ Soft wave_join(Soft a) {
  rebase(a, wave_max_f32(a.m));
  a.s = wave_sum(a.s);
  a.u = wave_sum(a.u);
  return a;
}

// A wave's list: lane i holds the i-th best entry; (bar, bar_i) is its topk-th.
struct List {
  float v;
  int i;
  float bar;
  int bar_i;
};

__device__ __forceinline__ void list_clear(List& l) {
  l.v = -__builtin_inff();
  l.i = kNone;
  l.bar = l.v;
  l.bar_i = kNone;
}

__device__ __forceinline__ bool over_bar(const List& l, float v, int i) {
  return v > l.bar || (v == l.bar && i < l.bar_i);
}

// insert the wave-uniform entry (v, i); it is over the bar
__device__ __forceinline__ void list_insert(List& l, float v, int i, int topk, int lane) {
  const uint64_t ahead = __builtin_amdgcn_ballot_w64(l.v > v || (l.v == v && l.i < i));
  const int pos = __builtin_popcountll(ahead);
  const float up_v = dpp_mov<0x138>(l.v);  // wave_shr:1, lane i takes lane i - 1's
  const int up_i = dpp_mov_i<0x138>(l.i);
  l.v = lane < pos ? l.v : lane == pos ? v : up_v;
  l.i = lane < pos ? l.i : lane == pos ? i : up_i;
  l.bar = fbits(__builtin_amdgcn_readlane(ubits(l.v), topk - 1));
  l.bar_i = (int)__builtin_amdgcn_readlane((uint32_t)l.i, topk - 1);
}

// insert every lane's entry (v, i) that is over the bar and at least `least`
__device__ __forceinline__ void list_add(List& l, float v, int i, float least, int topk, int lane) {
  uint64_t b = __builtin_amdgcn_ballot_w64(v >= least && over_bar(l, v, i));
  while (b != 0) {
    const int from = __builtin_ctzll(b);
    list_insert(l, fbits(__builtin_amdgcn_readlane(ubits(v), from)),
                (int)__builtin_amdgcn_readlane((uint32_t)i, from), topk, lane);
    b = (b & (b - 1)) & __builtin_amdgcn_ballot_w64(over_bar(l, v, i));
  }
}

// the topk-th largest of the lanes' values: its order key, bit by bit
__device__ __forceinline__ float kth_of_lanes(float v, int topk) {
  const uint32_t key = (uint32_t)order_key(v) ^ 0x80000000u;
  uint32_t t = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t c = t | (1u << bit);
    t = __builtin_popcountll(__builtin_amdgcn_ballot_w64(key >= c)) >= topk ? c : t;
  }
  const int k = (int)(t ^ 0x80000000u);
  return fbits((uint32_t)k ^ ((uint32_t)(k >> 31) & 0x7fffffffu));
}

// N logits per lane into the running state, the list and the rank count.
// idx[q]: index of x[q * per], or kNone where a lane has none (x = -inf there).
// where: -1 all indices lie before the token, 1 after it, 0 neither.
template <int N, int PER>
__device__ __forceinline__ void take(const float (&x)[N], const int (&idx)[N / PER], Soft& a, List& l, int& above,
                                     float xt, int tok, int where, int topk, int lane) {
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
    const uint64_t b = __builtin_amdgcn_ballot_w64(top >= l.bar);
    if (b != 0) {
      const float least = __builtin_popcountll(b) > 8 ? kth_of_lanes(top, topk) : l.bar;
#pragma unroll
      for (int e = 0; e < N; ++e) list_add(l, x[e], idx[e / PER] + e % PER, least, topk, lane);
    }
  }
}

template <int XK>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobArgs g) {
  constexpr int VE = vec_elems<XK>();
  constexpr int NV = 16 / VE;  // 16 logits per thread and step
  constexpr int ES = XK == CK_F32 ? 4 : 2;
  __shared__ Soft soft_s[kWaves];
  __shared__ int above_s[kWaves];
  __shared__ float list_v[kWaves][SKINNY_TOPK_MAX];
  __shared__ int list_i[kWaves][SKINNY_TOPK_MAX];
  __shared__ int last_s;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int topk = g.topk;
  const int64_t r = (int64_t)blockIdx.x / g.segments;
  const int seg = (int)((int64_t)blockIdx.x - r * g.segments);
  const char* row = (const char*)g.logits + r * g.ld * ES;

  // the token and its logit; a token outside the row has none
  const int64_t token = g.tokens64 ? ((const int64_t*)g.tokens)[r] : (int64_t)((const int32_t*)g.tokens)[r];
  const bool known = token >= 0 && token < g.vocab;
  const int tok = known ? (int)token : 0;
  const float xt = to_f32<XK>(row, tok);

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
  int above = 0;

  u32x4 raw[NV];
#pragma unroll
  for (int q = 0; q < NV; ++q)
    if (q * kThreads + tid < nvec) raw[q] = load16<ES>(vec + (int64_t)(q * kThreads + tid) * 16);
  for (int c = 0; c < nvec; c += NV * kThreads) {
    float x[NV * VE];
    int idx[NV];
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int v = c + q * kThreads + tid;
      unpack<XK>(raw[q], &x[q * VE]);
      idx[q] = first + v * VE;
      if (v >= nvec) {
        idx[q] = kNone;
#pragma unroll
        for (int e = 0; e < VE; ++e) x[q * VE + e] = -__builtin_inff();
      }
    }
#pragma unroll
    for (int q = 0; q < NV; ++q) {  // the next step's logits are on their way during this one's work
      const int v = c + (NV + q) * kThreads + tid;
      if (v < nvec) raw[q] = load16<ES>(vec + (int64_t)v * 16);
    }
    const bool full = c + NV * kThreads <= nvec;
    const int i0 = first + c * VE, i1 = i0 + NV * kThreads * VE;
    const int where = !full ? 0 : i1 <= tok ? -1 : i0 > tok ? 1 : 0;
    take<NV * VE, VE>(x, idx, a, l, above, xt, tok, where, topk, lane);
  }
  if (wave == 0 && len % VE != 0) {  // the last logits
    const int i = lane < len % VE ? first + nvec * VE + lane : kNone;
    float x[1] = {-__builtin_inff()};
    if (i != kNone) x[0] = to_f32<XK>(row, i);
    const int idx[1] = {i};
    take<1, 1>(x, idx, a, l, above, xt, tok, 0, topk, lane);
  }

  // join the waves in wave 0
  auto join_waves = [&]() __attribute__((always_inline)) {
    a = wave_join(a);
    if (lane == 0) {
      soft_s[wave] = a;
      above_s[wave] = above;
    }
    if (wave > 0 && lane < topk) {
      list_v[wave][lane] = l.v;
      list_i[wave][lane] = l.i;
    }
    __syncthreads();
    if (wave == 0) {
      Soft b = {kLowest, 0.0f, 0.0f};
      int n = 0;
      if (lane < kWaves) {
        b = soft_s[lane];
        n = above_s[lane];
      }
      a = wave_join(b);
      above = n;
      above += __builtin_amdgcn_readlane((uint32_t)n, 1) + __builtin_amdgcn_readlane((uint32_t)n, 2) +
               __builtin_amdgcn_readlane((uint32_t)n, 3);
      above = (int)__builtin_amdgcn_readfirstlane((uint32_t)above);
      if (topk > 0) {
#pragma unroll
        for (int q = 1; q < kWaves; ++q) {
          const float v = lane < topk ? list_v[q][lane] : -__builtin_inff();
          const int i = lane < topk ? list_i[q][lane] : kNone;
          list_add(l, v, i, l.bar, topk, lane);
        }
      }
    }
  };
  join_waves();

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
        st_dev(mine + 4 + lane, l.v);
        st_dev(mine + 4 + topk + lane, fbits((uint32_t)l.i));
      }
      wait_mem();  // this segment has reached the device-coherent level
      if (lane == 0) last_s = atomicAdd(&g.counters[r], 1u) == (uint32_t)(g.segments - 1);
    }
    __syncthreads();
    if (!last_s) return;
    // the last workgroup of the row: every segment is there
    a = Soft{kLowest, 0.0f, 0.0f};
    above = 0;
    list_clear(l);
    const int at = tid;  // one segment per thread (kMaxSegments <= 64: wave 0)
    if (at < g.segments) {
      const float* p = part + (int64_t)at * stride;
      a = Soft{ld_dev(p), ld_dev(p + 1), ld_dev(p + 2)};
      above = (int)ubits(ld_dev(p + 3));
    }
    // the sum over lanes (counts fit: below 2^31 in all)
    above += dpp_mov_i<kDppXor1>(above);
    above += dpp_mov_i<kDppXor2>(above);
    above += dpp_mov_i<kDppRowHalfMirror>(above);
    above += dpp_mov_i<kDppRowMirror>(above);
    above = (int)(__builtin_amdgcn_readlane((uint32_t)above, 0) + __builtin_amdgcn_readlane((uint32_t)above, 16) +
                  __builtin_amdgcn_readlane((uint32_t)above, 32) + __builtin_amdgcn_readlane((uint32_t)above, 48));
    if (topk > 0) {
      // kMaxSegments * SKINNY_TOPK_MAX entries over kThreads threads
      constexpr int R = kLogprobMaxSegments * SKINNY_TOPK_MAX / kThreads;
      const int n = g.segments * topk;
      float v[R];
      int i[R];
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int e = q * kThreads + tid;
        v[q] = -__builtin_inff();
        i[q] = kNone;
        if (e < n) {
          const int s = e / topk;
          const float* p = part + (int64_t)s * stride + 4 + (e - s * topk);
          v[q] = ld_dev(p);
          i[q] = (int)ubits(ld_dev(p + topk));
        }
      }
#pragma unroll
      for (int q = 0; q < R; ++q) list_add(l, v[q], i[q], l.bar, topk, lane);
    }
    __syncthreads();  // last_s and the waves' slots were read
    join_waves();
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
      g.top_ids[r * topk + lane] = l.i == kNone ? -1 : l.i;
      g.top_logprobs[r * topk + lane] = none ? ninf : (l.v - a.m) - ln_s;
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
  const auto fn = x_kind == CK_F32   ? logprobs_kernel<CK_F32>
                  : x_kind == CK_F16 ? logprobs_kernel<CK_F16>
                                     : logprobs_kernel<CK_BF16>;
  hipLaunchKernelGGL(fn, dim3((unsigned)(a.m * a.segments)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace skinny
