// adjust.hip -- penalties for repeated tokens, biases and grammar masks on rows
// of logits, for gfx950 (MI355X).
//
//   x_j = s_j ? (x_j > 0 ? x_j / theta : x_j theta) : x_j     s_j: j occurs in the row's tokens
//   x_j = x_j - (frequency c_j + presence [c_j > 0])          c_j: times j was generated
//   x_j = x_j + bias_j;   x_j = -inf where the mask does not allow j
//
// Few of a row's logits are penalised or biased, so the work is a stream and a
// few corrections.  A workgroup owns a segment of a row:
//   * it counts the row's tokens that fall into the segment in a table in LDS
//     (one entry per token of the vocabulary: times generated, whether in the
//     prompt, whether biased) and lists those that occur, each once, by the
//     first count of its entry;
//   * it copies the segment, converted to the output's type, with -inf where the
//     mask says so (in place: it writes only what the mask takes away);
//   * it then computes each listed token's logit from the input and the
//     table and overwrites the copy.
// The stream needs no table, and the corrections cost a gather of a few logits.
// Counts are integers and each logit has one writer after the stream, so the
// order of the atomics changes nothing.  HBM-bound for many rows: the logits
// are read and written once; a row's tokens are read once per segment, from L2.
#include <math.h>

#include "requests.h"
#include "vector_io.h"

namespace skinny {

namespace {

constexpr int kThreads = 256;
constexpr int kSegmentMax = 16384;  // tokens of a segment with a table
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

// four token ids from position i of a list of `room` on (-1 past it)
__device__ __forceinline__ void load_tokens4(const void* list, int64_t at, int i, int room, int tokens64, int64_t (&t)[4]) {
  if (i + 4 <= room) {
    if (tokens64 != 0) {
      const Raw<CK_F32, 8> w = load_raw<CK_F32, 8>(list, 2 * (at + i));
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = (int64_t)((uint64_t)w.w[2 * e + 1] << 32 | w.w[2 * e]);
    } else {
      const Raw<CK_F32, 4> w = load_raw<CK_F32, 4>(list, at + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = (int32_t)w.w[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      t[e] = i + e >= room ? -1 : tokens64 != 0 ? ((const int64_t*)list)[at + i + e] : (int64_t)((const int32_t*)list)[at + i + e];
  }
}

__device__ __forceinline__ int64_t token_at(const void* list, int64_t i, int tokens64) {
  return tokens64 != 0 ? ((const int64_t*)list)[i] : (int64_t)((const int32_t*)list)[i];
}

// values per vector of the stream: 16 bytes of the wider type
template <int XK, int OK>
constexpr int stream_elems() { return XK == CK_F32 || OK == CK_F32 ? 4 : 8; }

// TABLE: 0 (mask only), or an entry's bits
template <int XK, int OK, bool IN_PLACE, int TABLE>
__global__ __launch_bounds__(kThreads) void adjust_kernel(AdjustArgs g) {
  extern __shared__ uint32_t table_s[];
  __shared__ int listed_s, twice_s;
  constexpr int CW = TABLE == 0 ? 16 : TABLE;
  using At = Entry<CW>;
  const int tid = threadIdx.x;
  const uint32_t row_index = blockIdx.x / (uint32_t)g.segments;
  const int64_t r = row_index;
  const int first = (int)(blockIdx.x - row_index * (uint32_t)g.segments) * g.seg_len;  // a multiple of 32
  const int len = min(g.seg_len, g.vocab - first);
  const char* x_row = (const char*)g.logits + (r * g.ld + first) * kind_size<XK>();
  char* o_row = (char*)g.out + (r * g.ldo + first) * kind_size<OK>();
  const uint8_t* mask = nullptr;
  if (g.mask != nullptr) {
    const int which = g.mask_rows != nullptr ? g.mask_rows[r] : (int)r;
    if (which >= 0 && which < g.masks) mask = (const uint8_t*)(g.mask + which * g.ldm) + (first >> 3);
  }
  uint16_t* list_s = (uint16_t*)(table_s + (g.seg_len * CW / 32));

  if constexpr (TABLE != 0) {
    for (int i = tid; i < g.seg_len * CW / 32; i += kThreads) table_s[i] = 0;
    if (tid == 0) listed_s = twice_s = 0;
    __syncthreads();
    if (g.history != nullptr) {
      const int held = g.lengths != nullptr ? max(0, min(g.lengths[r], g.history_len)) : g.history_len;
      const int prompt = g.prompt_lengths != nullptr ? max(0, min(g.prompt_lengths[r], held)) : 0;
      for (int i = tid * 4; i < held; i += kThreads * 4) {
        int64_t t[4];
        load_tokens4(g.history, r * g.ldh, i, g.history_len, g.tokens64, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t off = t[e] - first;
          if (i + e < held && off >= 0 && off < len) {
            const At at((int)off);
            const uint32_t old = i + e < prompt ? atomicOr(&table_s[at.word], kInPrompt << at.shift)
                                                : atomicAdd(&table_s[at.word], kOnce << at.shift);
            if (at.of(old) == 0) list_s[atomicAdd(&listed_s, 1)] = (uint16_t)off;
          }
        }
      }
    }
  }

  // the stream
  constexpr int VE = stream_elems<XK, OK>();
  const int vectors = len / VE;
  auto mask_bits = [&](int v) -> uint32_t {  // bits of vector v's tokens
    if (mask == nullptr) return 0xffu;
    return VE == 8 ? mask[v] : (uint32_t)mask[v >> 1] >> (4 * (v & 1)) & 15u;
  };
  constexpr uint32_t kAll = (1u << VE) - 1;
  if constexpr (IN_PLACE) {
    if (mask != nullptr) {
      for (int v = tid; v < vectors; v += kThreads) {
        const uint32_t b = mask_bits(v) & kAll;
        if (b == kAll) continue;
        float x[VE];
        if (b != 0) unpack_raw<XK, VE>(load_raw<XK, VE>(x_row, (int64_t)v * VE), x);
#pragma unroll
        for (int e = 0; e < VE; ++e) x[e] = (b >> e & 1) != 0 ? x[e] : -INFINITY;
        store_vec<OK, VE>(o_row, (int64_t)v * VE, x);
      }
      for (int j = vectors * VE + tid; j < len; j += kThreads)
        if (!allowed_at(mask, j)) store_out<OK>(o_row, j, -INFINITY);
    }
  } else {
    constexpr int U = 4;  // vectors of a thread in flight
    for (int v0 = tid; v0 < vectors; v0 += U * kThreads) {
      Raw<XK, VE> raw[U];
      uint32_t bits[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = min(v0 + u * kThreads, vectors - 1);
        raw[u] = load_raw<XK, VE>(x_row, (int64_t)v * VE);
        bits[u] = mask_bits(v);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[VE];
        unpack_raw<XK, VE>(raw[u], x);
#pragma unroll
        for (int e = 0; e < VE; ++e) x[e] = (bits[u] >> e & 1) != 0 ? x[e] : -INFINITY;
        if (v0 + u * kThreads < vectors) store_vec<OK, VE>(o_row, (int64_t)(v0 + u * kThreads) * VE, x);
      }
    }
    for (int j = vectors * VE + tid; j < len; j += kThreads)
      store_out<OK>(o_row, j, allowed_at(mask, j) ? value_at<XK>(x_row, j) : -INFINITY);
  }

  if constexpr (TABLE != 0) {
    // the biased tokens' flags; which are listed twice matters later
    const int64_t bias_row = r * g.biases;
    if (g.biases > 0) {
      for (int i = tid; i < g.biases; i += kThreads) {
        const int64_t off = token_at(g.bias_ids, bias_row + i, g.tokens64) - first;
        if (off >= 0 && off < len) {
          const At at((int)off);
          if ((at.of(atomicOr(&table_s[at.word], kBiased << at.shift)) & kBiased) != 0) twice_s = 1;
        }
      }
    }
    wait_mem();  // the stream's stores come before the corrections
    __syncthreads();
    Penalties p;
    p.theta = g.repetition != nullptr ? g.repetition[r] : 1.0f;
    p.frequency = g.frequency != nullptr ? g.frequency[r] : 0.0f;
    p.presence = g.presence != nullptr ? g.presence[r] : 0.0f;
    const int listed = listed_s;
    for (int i = tid; i < listed; i += kThreads) {
      const int off = list_s[i];
      const At at(off);
      const uint32_t entry = at.of(table_s[at.word]);
      if ((entry & kBiased) != 0) continue;
      const float x = penalised(value_at<XK>(x_row, off), entry, p);
      store_out<OK>(o_row, off, allowed_at(mask, off) ? x : -INFINITY);
    }
    if (g.biases > 0) {
      __syncthreads();
      const bool twice = twice_s != 0;
      for (int i = tid; i < g.biases; i += kThreads) {
        const int64_t token = token_at(g.bias_ids, bias_row + i, g.tokens64), o = token - first;
        if (o < 0 || o >= len) continue;
        const int off = (int)o;
        const At at(off);
        // the first to take the flag away writes the token's logit
        const uint32_t entry = at.of(atomicAnd(&table_s[at.word], ~(kBiased << at.shift)));
        if ((entry & kBiased) == 0) continue;
        float b = g.bias_values[bias_row + i];
        if (twice) {
          b = 0.0f;
          for (int k = 0; k < g.biases; ++k)
            if (token_at(g.bias_ids, bias_row + k, g.tokens64) == token) b += g.bias_values[bias_row + k];
        }
        const float x = penalised(value_at<XK>(x_row, off), entry, p) + b;
        store_out<OK>(o_row, off, allowed_at(mask, off) ? x : -INFINITY);
      }
    }
  }
}

template <int XK, int OK, bool IN_PLACE>
hipError_t launch_kinds(AdjustArgs a, hipStream_t stream) {
  const bool rules = a.history != nullptr || a.biases > 0;
  const int bits = a.history_len < 1 << 14 ? 16 : 32;
  // segments: as many as give eight workgroups per CU, of at least 2048 tokens
  int64_t want = (2048 + a.m - 1) / a.m;
  int64_t seg = (a.vocab + want - 1) / want;
  if (seg < 2048) seg = 2048;
  if (seg > kSegmentMax) seg = kSegmentMax;
  if (seg > a.vocab) seg = a.vocab;
  a.seg_len = (int32_t)((seg + 31) / 32 * 32);
  a.segments = (a.vocab + a.seg_len - 1) / a.seg_len;
  a.list_len = a.history == nullptr ? 0 : a.history_len < a.seg_len ? a.history_len : a.seg_len;
  const size_t lds = rules ? (size_t)a.seg_len * bits / 8 + (size_t)(a.list_len + 1) / 2 * 4 : 0;
  const auto fn = !rules ? adjust_kernel<XK, OK, IN_PLACE, 0>
                  : bits == 16 ? adjust_kernel<XK, OK, IN_PLACE, 16> : adjust_kernel<XK, OK, IN_PLACE, 32>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024 - 256);
    if (e != hipSuccess) return e;
  }
  const int64_t most = kMaxLaunchThreads / 2 / kThreads / a.segments;  // rows of a launch
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
    hipLaunchKernelGGL(fn, dim3((unsigned)(part.m * a.segments)), dim3(kThreads), lds, stream, part);
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
