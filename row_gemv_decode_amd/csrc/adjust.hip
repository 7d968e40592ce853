// adjust.hip -- penalties for repeated tokens, biases and grammar masks on rows
// of logits, for gfx950 (MI355X).
//
//   x_j = s_j ? (x_j > 0 ? x_j / theta : x_j theta) : x_j     s_j: j occurs in the row's tokens
//   x_j = x_j - (frequency c_j + presence [c_j > 0])          c_j: times j was generated
//   x_j = x_j + bias_j;   x_j = -inf where the mask does not allow j
//
// A workgroup owns a segment of a row.  It counts the row's tokens that fall into
// the segment in a table in LDS (an entry per token of the vocabulary: times
// generated, whether in the prompt, whether biased), then streams the segment
// from input to output with each vector's entries and mask bits at hand; in place it
// touches only the vectors that change.  Counts are integers, so the order of the
// atomics changes nothing.  Biased tokens are few: the stream leaves their logits as
// they are, and where a segment has any, one thread each computes them afterwards,
// adding a token's biases in the order of the list, whose first 1024 entries wait in LDS
// (read from memory again for each token that is listed twice, 64 x 50000 with 300 biases
// took 90 us for 17).  Rules without a history or without biases have kernels of their
// own, which are shorter (64 x 32000 with 4096 ids 7.9 -> 7.5).
// HBM-bound for many rows: the logits are read and written once; a row's tokens
// are read once per segment, from L2.  For few rows the chain of memory latencies
// counts: what the first steps need is all in flight before the table is cleared.
// Measured: 512 x 100003 fp32 with 1024 ids, 32 biases and a mask each 81 us (5.1 TB/s),
// 16 x 131071 bf16 to fp32 with 4096 ids 7.8, 1 x 32000 fp32 3.9, 256 masks of 50021
// f16 logits in place 8.7.
#include <math.h>

#include <type_traits>

#include "requests.h"
#include "vector_io.h"
#include "window_kernel.h"

namespace skinny {

namespace {

constexpr int kSegmentMax = 16384;      // tokens of a segment with a table (half as many where
                                        // 32-bit entries and a list of biases share 64 KiB)
constexpr int kShortSegmentMax = 4096;  // and where a row's tokens are few
constexpr int kFewTokens = 4096;
constexpr int kThreadsMax = 512;
constexpr int kBiasesHeld = 1024;  // a row's first biases are kept in LDS
constexpr int kBiasStep = 16;
constexpr int biases_held(int biases) {
  return ((biases < kBiasesHeld ? biases : kBiasesHeld) + kBiasStep - 1) / kBiasStep * kBiasStep;
}
// table entries: 16 bits, or 32 for histories that could count further than 14 bits
constexpr uint32_t kInPrompt = 1, kBiased = 2, kOnce = 4;

template <int CW>
struct Entry {  // entry `off` of the table: word and shift
  int word, shift;
  __device__ __forceinline__ explicit Entry(int off)
      : word(CW == 16 ? off >> 1 : off), shift(CW == 16 ? (off & 1) * 16 : 0) {}
  static constexpr uint32_t kMask = CW == 16 ? 0xffffu : 0xffffffffu;
  __device__ __forceinline__ uint32_t of(uint32_t w) const { return (w >> shift) & kMask; }
};

__device__ __forceinline__ bool allowed_at(const uint8_t* mask, int64_t j) {
  return mask == nullptr || ((mask[j >> 3] >> (j & 7)) & 1) != 0;
}

struct Penalties {
  float theta, frequency, presence;
};

// the penalised logit; products and sums are rounded one by one, as written
__device__ __forceinline__ float penalised(float x, uint32_t entry, const Penalties& p) {
#pragma clang fp contract(off)
  const uint32_t count = entry / kOnce;
  if ((entry & ~kBiased) != 0) x = x > 0.0f ? x / p.theta : x * p.theta;
  if (count != 0) {
    const float t = p.frequency * (float)count;
    x = x - (t + p.presence);
  }
  return x;
}

// 16 bytes of a list of `room` token ids, from position i on (any past the list): four
// ids of 32 bits, two of 64
__device__ __forceinline__ u32x4 load_tokens(const void* list, int64_t at, int i, int room, int tokens64) {
  u32x4 w = {0, 0, 0, 0};
  if (tokens64 != 0) {
    const uint32_t* p = (const uint32_t*)list + 2 * (at + i);
    if (i + 2 <= room) {
      w = *(const u32x4_align4*)p;
    } else if (i < room) {
      w[0] = p[0], w[1] = p[1];
    }
  } else {
    const uint32_t* p = (const uint32_t*)list + at + i;
    if (i + 4 <= room) {
      w = *(const u32x4_align4*)p;
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (i + e < room) w[e] = p[e];
    }
  }
  return w;
}
// id e's place in a segment that starts at token `first`; not below its length (which
// is at most 2^30) where the id lies elsewhere
__device__ __forceinline__ uint32_t token_off(const u32x4& w, int e, int tokens64, int first) {
  const uint32_t low32 = w[e], low64 = w[2 * (e & 1)], high64 = w[2 * (e & 1) + 1];
  return tokens64 == 0 ? low32 - (uint32_t)first : e < 2 && high64 == 0 ? low64 - (uint32_t)first : ~0u;
}

__device__ __forceinline__ int64_t token_at(const void* list, int64_t i, int tokens64) {
  return tokens64 != 0 ? ((const int64_t*)list)[i] : (int64_t)((const int32_t*)list)[i];
}

// values per vector of the stream: 16 bytes of the wider type
template <int XK, int OK>
constexpr int stream_elems() { return XK == CK_F32 || OK == CK_F32 ? 4 : 8; }

// TABLE: 0 (mask only), or an entry's bits; HISTORY, BIASES: which of the two there are
template <int XK, int OK, bool IN_PLACE, int TABLE, bool HISTORY, bool BIASES>
__global__ __launch_bounds__(kThreadsMax) void adjust_kernel(AdjustArgs g) {
  extern __shared__ uint32_t table_s[] __attribute__((aligned(16)));  // the table, then the first biases
  __shared__ int biased_s, twice_s;
  constexpr int CW = TABLE == 0 ? 16 : TABLE;
  using At = Entry<CW>;
  const int tid = threadIdx.x, threads = blockDim.x;
  // (a row's segments on one XCD, so that its tokens are read into one L2: 64 x 32000 with
  // 4096 ids 8.8 -> 7.8 us; masks alone take 3 % longer so)
  const uint32_t index = TABLE != 0 ? xcd_place(blockIdx.x, gridDim.x) : blockIdx.x;
  const uint32_t row_index = index / (uint32_t)g.segments;
  const int64_t r = row_index;
  const int first = (int)(index - row_index * (uint32_t)g.segments) * g.seg_len;  // a multiple of 32
  const int len = min(g.seg_len, g.vocab - first);
  const char* x_row = (const char*)g.logits + (r * g.ld + first) * kind_size<XK>();
  char* o_row = (char*)g.out + (r * g.ldo + first) * kind_size<OK>();
  const uint8_t* mask = nullptr;
  if (g.mask != nullptr) {
    const int which = g.mask_rows != nullptr ? g.mask_rows[r] : (int)r;
    if (which >= 0 && which < g.masks) mask = (const uint8_t*)(g.mask + which * g.ldm) + (first >> 3);
  }

  // what the first steps of both loops need is in flight before either begins
  constexpr int H = 2;  // history loads of a thread in flight
  const int per = g.tokens64 != 0 ? 2 : 4;  // ids of a load
  u32x4 ids[H];
  int held = 0, prompt = 0;
  Penalties pen = {1.0f, 0.0f, 0.0f};
  const int64_t bias_row = r * g.biases;
  // a listed id's place in the segment, -1 for every id that does not lie in it (compared
  // before anything is subtracted or cut: a list may be filled up with any id)
  auto bias_off = [&](int i) -> int {
    const int64_t id = token_at(g.bias_ids, bias_row + i, g.tokens64);
    return id >= first && id < (int64_t)first + len ? (int)(id - first) : -1;
  };
  int my_bias = -1;
  float my_value = 0.0f;
  if constexpr (HISTORY) {
#pragma unroll
    for (int u = 0; u < H; ++u)
      if (u * threads * per < g.history_len)
        ids[u] = load_tokens(g.history, r * g.ldh, (u * threads + tid) * per, g.history_len, g.tokens64);
    held = g.lengths != nullptr ? max(0, min(g.lengths[r], g.history_len)) : g.history_len;
    prompt = g.prompt_lengths != nullptr ? max(0, min(g.prompt_lengths[r], held)) : 0;
    if (g.repetition != nullptr) pen.theta = g.repetition[r];
    if (g.frequency != nullptr) pen.frequency = g.frequency[r];
    if (g.presence != nullptr) pen.presence = g.presence[r];
  }
  if constexpr (BIASES) {
    if (tid < g.biases) {
      my_bias = bias_off(tid);
      my_value = g.bias_values[bias_row + tid];
    }
  }
  constexpr int VE = stream_elems<XK, OK>();
  constexpr int U = 4;  // vectors of a thread in flight
  constexpr uint32_t kAll = (1u << VE) - 1;
  const int vectors = len / VE;
  auto mask_bits = [&](int v) -> uint32_t {  // bits of vector v's tokens
    if (mask == nullptr) return kAll;
    return VE == 8 ? mask[v] : (uint32_t)mask[v >> 1] >> (4 * (v & 1)) & kAll;
  };
  // A step is U vectors of each thread.  The last one has fewer and skips those that
  // no thread has; the others run straight through (with a branch at each vector 512
  // rows of 100003 took 92.8 us for 85.3).
  Raw<XK, VE> raw[U];
  uint32_t bits[U];
  auto whole = [&](int v0) { return v0 - tid + U * threads <= vectors; };
  auto load_step = [&](auto full, int v0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!full.value && v0 - tid + u * threads >= vectors) break;
      const int v = min(v0 + u * threads, vectors - 1);
      bits[u] = mask_bits(v);
      if (!IN_PLACE) raw[u] = load_raw<XK, VE>(x_row, (int64_t)v * VE);
    }
  };
  auto load_vectors = [&](int v0) {
    if (whole(v0)) {
      load_step(std::true_type{}, v0);
    } else {
      load_step(std::false_type{}, v0);
    }
  };
  if (vectors > 0) load_vectors(tid);

  // the first biases in LDS: places in the segment and values, up to a multiple of a step
  const int held_biases = biases_held(g.biases), biases = max(g.biases, held_biases);
  int* bias_off_s = (int*)(table_s + g.seg_len * CW / 32);
  float* bias_s = (float*)(bias_off_s + held_biases);
  if constexpr (TABLE != 0) {
    for (int i = tid; i < g.seg_len * CW / 32; i += threads) table_s[i] = 0;
    if (BIASES && tid == 0) biased_s = twice_s = 0;
    lds_barrier();
    for (int i0 = 0; HISTORY && i0 < held; i0 += H * threads * per) {
      if (i0 > 0) {
#pragma unroll
        for (int u = 0; u < H; ++u)
          ids[u] = load_tokens(g.history, r * g.ldh, i0 + (u * threads + tid) * per, held, g.tokens64);
      }
#pragma unroll
      for (int u = 0; u < H; ++u) {
        if (i0 + u * threads * per >= held) break;
        const int i = i0 + (u * threads + tid) * per;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t off = token_off(ids[u], e, g.tokens64, first);
          if (i + e < held && off < (uint32_t)len) {  // (a 64-bit load's ids 2 and 3 lie nowhere)
            const At at((int)off);
            if (i + e < prompt) {
              atomicOr(&table_s[at.word], kInPrompt << at.shift);
            } else {
              atomicAdd(&table_s[at.word], kOnce << at.shift);
            }
          }
        }
      }
    }
    for (int i = tid; BIASES && i < biases; i += threads) {
      const int off = i == tid ? my_bias : i < g.biases ? bias_off(i) : -1;
      if (i < held_biases) {
        bias_off_s[i] = off;
        bias_s[i] = i == tid ? my_value : i < g.biases ? g.bias_values[bias_row + i] : 0.0f;
      }
      if (off >= 0) {
        const At at(off);
        biased_s = 1;
        if ((at.of(atomicOr(&table_s[at.word], kBiased << at.shift)) & kBiased) != 0) twice_s = 1;
      }
    }
    lds_barrier();
  }

  // the entries of vector v, and whether any of them is not 0
  auto entries = [&](int v, uint32_t(&e)[VE]) -> bool {
    constexpr int W = VE * CW / 32;
    uint32_t w[W], some = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) some |= w[i] = table_s[v * W + i];
#pragma unroll
    for (int i = 0; i < VE; ++i) e[i] = CW == 16 ? (w[i / 2] >> (16 * (i & 1))) & 0xffffu : w[i];
    return some != 0;
  };
  auto adjusted = [&](float x, uint32_t entry) { return BIASES && (entry & kBiased) != 0 ? x : penalised(x, entry, pen); };
  auto stream_step = [&](auto full, int v0) {
    uint32_t e[U][VE];
    bool some[U];  // whether a vector has entries
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!full.value && v0 - tid + u * threads >= vectors) break;
      const int v = v0 + u * threads;
      some[u] = HISTORY && entries(min(v, vectors - 1), e[u]);
      if (IN_PLACE) {
        if (v >= vectors) some[u] = false, bits[u] = kAll;
        if (bits[u] != 0 && some[u]) raw[u] = load_raw<XK, VE>(x_row, (int64_t)v * VE);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!full.value && v0 - tid + u * threads >= vectors) break;
      const int v = v0 + u * threads;
      float x[VE];
      unpack_raw<XK, VE>(raw[u], x);
      if (HISTORY && some[u]) {
#pragma unroll
        for (int i = 0; i < VE; ++i) x[i] = adjusted(x[i], e[u][i]);
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) x[i] = (bits[u] >> i & 1) != 0 ? x[i] : -INFINITY;
      if (IN_PLACE ? bits[u] == 0 : full.value || v < vectors) {
        store_vec<OK, VE>(o_row, (int64_t)v * VE, x);
      } else if (IN_PLACE && (bits[u] != kAll || some[u])) {
        // one by one: without reading what stays (256 masks of 50021 in f16 took 10.5 us
        // with whole vectors read and written again, 9.0 so; 512 of 50000 in fp32 47 and 35)
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if ((bits[u] >> i & 1) == 0 || (HISTORY && e[u][i] != 0)) store_out<OK>(o_row, (int64_t)v * VE + i, x[i]);
      }
    }
  };
  for (int v0 = tid; v0 - tid < vectors; v0 += U * threads) {
    if (v0 != tid) load_vectors(v0);
    if (whole(v0)) {
      stream_step(std::true_type{}, v0);
    } else {
      stream_step(std::false_type{}, v0);
    }
  }
  for (int j = vectors * VE + tid; j < len; j += threads) {
    const At at(j);
    const uint32_t entry = HISTORY ? at.of(table_s[at.word]) : 0;
    if (!allowed_at(mask, j)) {
      store_out<OK>(o_row, j, -INFINITY);
    } else if (!IN_PLACE || entry != 0) {
      store_out<OK>(o_row, j, adjusted(value_at<XK>(x_row, j), entry));
    }
  }

  if constexpr (BIASES) {
    if (biased_s == 0) return;  // (the same in every thread)
    wait_mem();                 // the stream's stores come before the biased tokens'
    __syncthreads();
    const bool twice = twice_s != 0;
    for (int i = tid; i < g.biases; i += threads) {
      const int off = i < held_biases ? bias_off_s[i] : bias_off(i);
      if (off < 0) continue;
      const At at(off);
      // the first to take the flag away writes the token's logit
      const uint32_t entry = at.of(atomicAnd(&table_s[at.word], ~(kBiased << at.shift)));
      if ((entry & kBiased) == 0) continue;
      float b = 0.0f;
      if (!twice) {
        b = i < held_biases ? bias_s[i] : g.bias_values[bias_row + i];
      } else {
        for (int k0 = 0; k0 < held_biases; k0 += kBiasStep) {
          u32x4 offs[kBiasStep / 4];
          f32x4 values[kBiasStep / 4];
#pragma unroll
          for (int q = 0; q < kBiasStep / 4; ++q) {
            offs[q] = *(const u32x4*)(bias_off_s + k0 + 4 * q);
            values[q] = *(const f32x4*)(bias_s + k0 + 4 * q);
          }
#pragma unroll
          for (int k = 0; k < kBiasStep; ++k) b += offs[k / 4][k % 4] == (uint32_t)off ? values[k / 4][k % 4] : 0.0f;
        }
#pragma unroll 1
        for (int k = held_biases; k < g.biases; ++k)
          if (bias_off(k) == off) b += g.bias_values[bias_row + k];
      }
      const float x = penalised(value_at<XK>(x_row, off), entry, pen) + b;
      store_out<OK>(o_row, off, allowed_at(mask, off) ? x : -INFINITY);
    }
  }
}

template <int XK, int OK, bool IN_PLACE>
hipError_t launch_kinds(AdjustArgs a, hipStream_t stream) {
  const bool rules = a.history != nullptr || a.biases > 0;
  const int bits = a.history_len < 1 << 14 ? 16 : 32;
  // Segments: as many as give four workgroups per CU, of at least 1024 tokens, and short
  // where a row has few tokens; each reads all of them, so where they are many it is as
  // long as the table stays small beside the workgroups that share a CU's LDS.  Measured (us):
  //   four / eight workgroups per CU  16 x 131071 bf16, 4096 ids  8.8 / 12.1, 64 x 32000 6.6 / 8.6
  //   at least 1024 / 2048 / 4096     1 x 32000 fp32  3.9 / 4.5 / 5.6
  //   at most 2048 / 4096 / 8192 / 16384   512 x 100003 fp32, 1024 ids  77.8 / 80.4 / 80.6 / 86.4,
  //                                   4096 ids  92.1 / 82.8 / 83.2 / 88.1, 14000 ids  180 / 121 / 94.7 / 92.7
  //                                   512 x 50021 bf16, 1024 ids  45.5 / 35.6 / 40.5 / 38.4, 8192 ids
  //                                   96.8 / 62.5 / 48.1 / 45.3
  //                                   masks alone, 512 x 50000 fp32 in place  27.7 / 26.1 / 27.2 / 34.4,
  //                                   bf16 to fp32  35.9 / 35.0 / 35.0 / 40.7
  // and 512 threads for segments or histories past 4096 (512 x 100003 in segments of 14304
  // 85.3, with 256 92.9; 1 x 131071 with 8192 ids 4.9 and 6.5).
  int64_t want = (1024 + a.m - 1) / a.m;
  int64_t seg = (a.vocab + want - 1) / want;
  if (seg < 1024) seg = 1024;
  const int64_t longest = a.history_len <= kFewTokens   ? kShortSegmentMax
                          : bits == 16 || a.biases == 0 ? kSegmentMax : kSegmentMax / 2;
  if (seg > longest) seg = longest;
  if (seg > a.vocab) seg = a.vocab;
  a.seg_len = (int32_t)((seg + 31) / 32 * 32);
  a.segments = (a.vocab + a.seg_len - 1) / a.seg_len;
  const int threads = a.seg_len > kShortSegmentMax || a.history_len > kFewTokens ? kThreadsMax : 256;
  const size_t lds = rules ? (size_t)a.seg_len * bits / 8 + biases_held(a.biases) * 8 : 0;
  const auto fn = !rules                ? adjust_kernel<XK, OK, IN_PLACE, 0, false, false>
                  : a.history == nullptr ? adjust_kernel<XK, OK, IN_PLACE, 16, false, true>
                  : a.biases == 0        ? (bits == 16 ? adjust_kernel<XK, OK, IN_PLACE, 16, true, false>
                                                       : adjust_kernel<XK, OK, IN_PLACE, 32, true, false>)
                  : bits == 16           ? adjust_kernel<XK, OK, IN_PLACE, 16, true, true>
                                         : adjust_kernel<XK, OK, IN_PLACE, 32, true, true>;
  const int64_t most = kMaxLaunchThreads / 2 / threads / a.segments;  // rows of a launch
  if (most < 1) return hipErrorInvalidValue;
  for (int64_t r = 0; r < a.m; r += most) {
    AdjustArgs part = a;
    part.m = a.m - r < most ? a.m - r : most;
    part.logits = (const char*)a.logits + r * a.ld * kind_size<XK>();
    part.out = (char*)a.out + r * a.ldo * kind_size<OK>();
    const int64_t token = a.tokens64 != 0 ? 8 : 4;
    if (a.history != nullptr) part.history = (const char*)a.history + r * a.ldh * token;
    if (a.lengths != nullptr) part.lengths = a.lengths + r;
    if (a.prompt_lengths != nullptr) part.prompt_lengths = a.prompt_lengths + r;
    if (a.repetition != nullptr) part.repetition = a.repetition + r;
    if (a.frequency != nullptr) part.frequency = a.frequency + r;
    if (a.presence != nullptr) part.presence = a.presence + r;
    if (a.biases > 0) {
      part.bias_ids = (const char*)a.bias_ids + r * a.biases * token;
      part.bias_values = a.bias_values + r * a.biases;
    }
    if (a.mask_rows != nullptr) {
      part.mask_rows = a.mask_rows + r;
    } else if (a.mask != nullptr) {
      part.mask = a.mask + r * a.ldm;
      part.masks = (int32_t)(a.masks - r);
    }
    hipLaunchKernelGGL(fn, dim3((unsigned)(part.m * a.segments)), dim3(threads), lds, stream, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_adjust(const AdjustArgs& a, int x_kind, int out_kind, hipStream_t stream) {
  if (a.m < 1 || a.vocab < 1 || (out_kind != CK_F32 && out_kind != x_kind)) return hipErrorInvalidValue;
  const bool in_place = a.out == a.logits;
  if (x_kind == CK_F32)
    return in_place ? launch_kinds<CK_F32, CK_F32, true>(a, stream) : launch_kinds<CK_F32, CK_F32, false>(a, stream);
  if (x_kind == CK_F16)
    return in_place              ? launch_kinds<CK_F16, CK_F16, true>(a, stream)
           : out_kind == CK_F32  ? launch_kinds<CK_F16, CK_F32, false>(a, stream)
                                 : launch_kinds<CK_F16, CK_F16, false>(a, stream);
  return in_place             ? launch_kinds<CK_BF16, CK_BF16, true>(a, stream)
         : out_kind == CK_F32 ? launch_kinds<CK_BF16, CK_F32, false>(a, stream)
                              : launch_kinds<CK_BF16, CK_BF16, false>(a, stream);
}

}  // namespace skinny
