// abi_window.cpp -- the C ABI of the decode window's further operators
// declared in include/skinny_window.h (4-bit grouped GEMV, the MoE layer, token
// log probabilities): argument validation, all on the host and before any HIP
// call, and dispatch to the kernels in w4.hip, moe.hip and logprobs.hip.
#include <hip/hip_runtime_api.h>

#include <new>

#include "abi_checks.h"
#include "skinny_window.h"
#include "window.h"

using namespace skinny;

namespace {

bool group_ok(int32_t group) { return group == 32 || group == 64 || group == 128; }

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

// Workgroups per row of the log probabilities: as many as give four workgroups of
// four waves per CU of 256, but at most 16 (which cuts a window's rows alike at
// every m), each of at least 4096 logits.  From 256 rows on a row is one
// workgroup's, of eight waves up to 1023 rows and four from there on, but for long
// rows that leave the CUs unevenly filled: fewer than 512 of at least 98304 logits
// are cut in three, of four waves each.  Measured (us): at most 16 / 32 segments,
// 16 x 131071 bf16, top 20, 15.1 / 17.9, 1 x 151000 bf16 11.3 / 13.0; segments of at
// least 4096 / 8192, 1 x 32000 fp32 9.3 / 10.7, 4 x 50000 10.6 / 11.9.  Top 5, one
// workgroup of four waves / one of eight / two, three, four of four:
//   256 x 50021 f16     25.2 / 18.1 / 21.0, 19.4, 19.3
//   256 x 100003 fp32   39.0 / 28.4 / 31.1, 27.7, 28.3
//   300 x 100003 bf16   40.5 / 33.9 / 33.4, 29.4, 28.0
//   300 x 100003 fp32   41.8 / 35.9 / 34.6, 32.7, 34.0
//   400 x 151936 bf16   54.2 / 44.8 / 47.2, 42.0, 44.7
//   512 x 100003 bf16   41.5 / 35.7 / 38.0, 36.4, 41.9
//   512 x 151936 fp32   57.4 / 55.3 / 58.1, 63.4, 64.1
//   1023 x 151936 bf16  74.4 / 74.5 / 83.0, 81.4, 85.2   (2048 x 32000 bf16  45 / 54)
struct RowSegments {
  int64_t count, len;
  int waves;
};
RowSegments row_segments(int64_t m, int64_t vocab) {
  const bool thirds = m >= 256 && m < 512 && vocab >= 98304;
  int64_t want = m < 256 ? (1024 + m - 1) / m : thirds ? 3 : 1;
  if (want > kLogprobMaxSegments) want = kLogprobMaxSegments;
  const int64_t most = (vocab + 4095) / 4096;
  if (want > most) want = most;
  const int64_t len = ((vocab + want - 1) / want + 7) / 8 * 8;
  return {(vocab + len - 1) / len, len, m >= 256 && m < 1024 && !thirds ? 8 : 4};
}
// workspace: the rows' arrival counters, then the segments' partial results.
// The counters' region has one fixed size, so that one workspace serves runs
// of several sizes: no run's partial results touch another's counters.
constexpr int64_t kRowCounterBytes = SKINNY_WINDOW_COUNTER_BYTES;
int64_t logprob_bytes(int64_t m, int64_t vocab, int32_t topk) {
  const RowSegments s = row_segments(m, vocab);
  return s.count == 1 ? 0 : kRowCounterBytes + round256(m * s.count * (4 + 2 * (int64_t)topk) * 4);
}
bool logprob_sizes_ok(int64_t m, int64_t vocab, int32_t topk) {
  constexpr int64_t kMax = 1LL << 30;
  return m >= 1 && m <= kMax && vocab >= 1 && vocab <= kMax && m <= (1LL << 50) / vocab && topk >= 0 &&
         topk <= SKINNY_TOPK_MAX && topk <= vocab;
}

}  // namespace

static_assert(SKINNY_MOE_MAX_EXPERTS == kMoeMaxExperts, "expert limit");
// (the router's GEMV counts arrivals per range of columns, so at most one per expert)
static_assert(SKINNY_MOE_MAX_EXPERTS * 4 <= SKINNY_WINDOW_COUNTER_BYTES, "the router's counters");

struct skinny_moe_plan {
  skinny_moe_desc d;      // normalised copy (ldx / ldo filled in)
  skinny_plan* router;    // the logits' GEMV
  int64_t max_slots;      // distinct experts a window can reach
  // workspace regions, in bytes from its start
  int64_t router_ws;      // the router plan's own workspace comes first (its counters start at zero)
  int64_t logits, slots, slot_rank, parts, weights, h, y, bytes;
};

extern "C" {

skinny_status skinny_w4_mm_run(int64_t m, int64_t n, int64_t k, int32_t group, const void* A, int64_t lda,
                               int32_t a_dtype, const skinny_w4* W, void* C, int64_t ldc, int32_t c_dtype,
                               void* stream) {
  if (A == nullptr || W == nullptr || C == nullptr || W->codes == nullptr || W->scales == nullptr)
    return SKINNY_ERR_INVALID_ARG;
  if (!half_type(a_dtype) || !float_type(c_dtype) || !group_ok(group)) return SKINNY_ERR_UNSUPPORTED;
  if (m < 1 || m > SKINNY_GEMV_MAX_M || n < 1 || n > kMaxDim || k < 1 || k > kW4MaxK) return SKINNY_ERR_INVALID_ARG;
  if (lda == 0) lda = k;
  if (ldc == 0) ldc = n;
  if (lda > (1LL << 40) || ldc > (1LL << 40)) return SKINNY_ERR_INVALID_ARG;
  if (k % group != 0 || lda < k || ldc < n) return SKINNY_ERR_SHAPE;
  if (lda % 8 != 0 || !aligned(A, 16) || !aligned(W->codes, 16) || !aligned(W->scales, 2) ||
      !aligned(C, (uintptr_t)size_of(c_dtype)))
    return SKINNY_ERR_ALIGNMENT;
  const int64_t cb = span(m, ldc, n, size_of(c_dtype));
  if (overlap(C, cb, A, span(m, lda, k, 2)) || overlap(C, cb, W->codes, n * (k / 2)) ||
      overlap(C, cb, W->scales, n * (k / group) * 2) || overlap(C, cb, W->zeros, n * (k / group)))
    return SKINNY_ERR_INVALID_ARG;
  W4Args g;
  g.A = A;
  g.lda = lda;
  g.w = WindowWeight{W->codes, W->scales, W->zeros};
  g.n = n;
  g.k = k;
  g.C = C;
  g.ldc = ldc;
  g.m = (int32_t)m;
  g.c_kind = kind_of(c_dtype);
  return hip_status(launch_w4_mm(g, kind_of(a_dtype), group, (hipStream_t)stream));
}

skinny_status skinny_moe_plan_create(const skinny_moe_desc* desc, skinny_moe_plan** out_plan) {
  if (desc == nullptr || out_plan == nullptr || desc->struct_size < sizeof(skinny_moe_desc))
    return SKINNY_ERR_INVALID_ARG;
  skinny_moe_desc d = *desc;
  if (!half_type(d.dtype) || !float_type(d.out_dtype) || (d.w_dtype != d.dtype && d.w_dtype != SKINNY_W4) ||
      (d.flags & ~SKINNY_MOE_RENORM) != 0)
    return SKINNY_ERR_UNSUPPORTED;
  if (d.w_dtype == SKINNY_W4 ? !group_ok(d.group) : d.group != 0) return SKINNY_ERR_UNSUPPORTED;
  constexpr int64_t kMax = 1 << 20;
  if (d.max_m < 1 || d.max_m > SKINNY_GEMV_MAX_M || d.topk < 1 || d.topk > SKINNY_TOPK_MAX || d.experts < d.topk ||
      d.experts > SKINNY_MOE_MAX_EXPERTS || d.d < 1 || d.d > kMax || d.inter < 1 || d.inter > kMax ||
      d.shared_inter < 0 || d.shared_inter > kMax || d.num_cus < 0)
    return SKINNY_ERR_INVALID_ARG;
  if (d.ldx == 0) d.ldx = d.d;
  if (d.ldo == 0) d.ldo = d.d;
  if (d.ldx > (1LL << 40) || d.ldo > (1LL << 40)) return SKINNY_ERR_INVALID_ARG;
  const int64_t unit = d.group > 32 ? d.group : 32;
  if (d.d % unit != 0 || d.inter % unit != 0 || d.shared_inter % unit != 0 || d.ldx < d.d || d.ldo < d.d)
    return SKINNY_ERR_SHAPE;
  if (d.ldx % 8 != 0) return SKINNY_ERR_ALIGNMENT;

  MoeArgs sizes{};
  sizes.m = (int32_t)d.max_m;
  sizes.topk = d.topk;
  sizes.experts = (int32_t)d.experts;
  sizes.d = d.d;
  sizes.inter = d.inter;
  sizes.shared_inter = d.shared_inter;
  if (!moe_fits(sizes, d.group)) return SKINNY_ERR_UNSUPPORTED;

  skinny_mm_desc r{};
  r.struct_size = sizeof(r);
  r.a_dtype = d.dtype;
  r.w_dtype = d.dtype;
  r.c_dtype = SKINNY_F32;
  r.max_m = d.max_m;
  r.n = d.experts;
  r.k = d.d;
  r.lda = d.ldx;
  r.tile_id = -1;
  r.num_cus = d.num_cus;
  skinny_plan* router = nullptr;
  skinny_status st = skinny_mm_plan(&r, &router);
  if (st != SKINNY_OK) return st;
  size_t rws = 0;
  skinny_mm_workspace_size(router, &rws);
  skinny_moe_plan* p = new (std::nothrow) skinny_moe_plan;
  if (p == nullptr) {
    skinny_mm_plan_destroy(router);
    return SKINNY_ERR_INVALID_ARG;
  }
  p->d = d;
  p->router = router;
  p->max_slots = d.max_m * d.topk < d.experts ? d.max_m * d.topk : d.experts;
  const int64_t planes = moe_planes();
  int64_t at = 0;
  auto region = [&at](int64_t bytes) {
    const int64_t start = at;
    at += round256(bytes);
    return start;
  };
  p->router_ws = (int64_t)rws;
  region(p->router_ws);
  p->logits = region(d.max_m * d.experts * 4);
  p->slots = region(p->max_slots * 4);
  p->slot_rank = region(p->max_slots * kGemvMaxM * 4);
  p->parts = region(d.max_m * d.topk * 16);  // (at most one for each token's expert)
  p->weights = region(d.max_m * (d.topk + 1) * 4);
  p->h = region(d.max_m * (d.topk * d.inter + d.shared_inter) * planes * 2);
  p->y = region(d.max_m * (d.topk + (d.shared_inter > 0 ? 1 : 0)) * d.d * 4);
  p->bytes = at;
  *out_plan = p;
  return SKINNY_OK;
}

void skinny_moe_plan_destroy(skinny_moe_plan* plan) {
  if (plan != nullptr) skinny_mm_plan_destroy(plan->router);
  delete plan;
}

skinny_status skinny_moe_workspace_size(const skinny_moe_plan* plan, size_t* bytes) {
  if (plan == nullptr || bytes == nullptr) return SKINNY_ERR_INVALID_ARG;
  *bytes = (size_t)plan->bytes;
  return SKINNY_OK;
}

skinny_status skinny_moe_run(const skinny_moe_plan* plan, int64_t m, const void* x, const skinny_moe_weights* weights,
                             void* out, int32_t* topk_idx, float* topk_weight, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (plan == nullptr || x == nullptr || weights == nullptr || out == nullptr) return SKINNY_ERR_INVALID_ARG;
  const skinny_moe_desc& d = plan->d;
  if (m < 1 || m > d.max_m) return SKINNY_ERR_INVALID_ARG;
  const bool w4 = d.w_dtype == SKINNY_W4, shared = d.shared_inter > 0;
  const skinny_w4* ws[4] = {&weights->w13, &weights->w2, &weights->shared13, &weights->shared2};
  for (int i = 0; i < 4; ++i) {
    const bool used = i < 2 || shared;
    if (used ? ws[i]->codes == nullptr || (ws[i]->scales != nullptr) != w4 || (!w4 && ws[i]->zeros != nullptr)
             : ws[i]->codes != nullptr || ws[i]->scales != nullptr || ws[i]->zeros != nullptr)
      return SKINNY_ERR_INVALID_ARG;
  }
  // zero points: with every 4-bit weight of the layer, or with none
  const bool zeros = weights->w13.zeros != nullptr;
  for (int i = 1; i < (shared ? 4 : 2); ++i)
    if ((ws[i]->zeros != nullptr) != zeros) return SKINNY_ERR_UNSUPPORTED;
  if (weights->router == nullptr || (weights->shared_gate != nullptr) != shared) return SKINNY_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (!aligned(ws[i]->codes, 16) || !aligned(ws[i]->scales, 2)) return SKINNY_ERR_ALIGNMENT;
  if (!aligned(x, 16) || !aligned(weights->router, 16) || !aligned(weights->shared_gate, 16) ||
      !aligned(out, (uintptr_t)size_of(d.out_dtype)) || !aligned(topk_idx, 4) || !aligned(topk_weight, 4))
    return SKINNY_ERR_ALIGNMENT;
  if (overlap(out, span(m, d.ldo, d.d, size_of(d.out_dtype)), x, span(m, d.ldx, d.d, 2))) return SKINNY_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < (size_t)plan->bytes) return SKINNY_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SKINNY_ERR_ALIGNMENT;

  char* base = (char*)workspace;
  float* logits = (float*)(base + plan->logits);
  const skinny_status st = skinny_mm_run(plan->router, m, x, weights->router, nullptr, logits,
                                         plan->router_ws > 0 ? base : nullptr, (size_t)plan->router_ws, stream);
  if (st != SKINNY_OK) return st;
  auto weight = [](const skinny_w4& w) { return WindowWeight{w.codes, w.scales, w.zeros}; };
  MoeArgs a;
  a.x = x;
  a.ldx = d.ldx;
  a.d = d.d;
  a.inter = d.inter;
  a.shared_inter = d.shared_inter;
  a.w13 = weight(weights->w13);
  a.w2 = weight(weights->w2);
  a.s13 = weight(weights->shared13);
  a.s2 = weight(weights->shared2);
  a.shared_gate = weights->shared_gate;
  a.logits = logits;
  a.slots = (uint32_t*)(base + plan->slots);
  a.slot_rank = (int32_t*)(base + plan->slot_rank);
  a.parts = (uint32_t*)(base + plan->parts);
  a.weights = (float*)(base + plan->weights);
  a.h = (uint16_t*)(base + plan->h);
  a.y = (float*)(base + plan->y);
  a.topk_idx = topk_idx;
  a.topk_weight = topk_weight;
  a.out = out;
  a.ldo = d.ldo;
  a.m = (int32_t)m;
  a.experts = (int32_t)d.experts;
  a.topk = d.topk;
  a.renorm = (d.flags & SKINNY_MOE_RENORM) != 0;
  a.max_slots = (int32_t)plan->max_slots;
  a.out_kind = kind_of(d.out_dtype);
  return hip_status(launch_moe(a, kind_of(d.dtype), d.group, (hipStream_t)stream));
}

skinny_status skinny_token_logprobs_workspace_size(int64_t m, int64_t vocab, int32_t topk, size_t* bytes) {
  if (bytes == nullptr || !logprob_sizes_ok(m, vocab, topk)) return SKINNY_ERR_INVALID_ARG;
  *bytes = (size_t)logprob_bytes(m, vocab, topk);
  return SKINNY_OK;
}

skinny_status skinny_token_logprobs_run(int64_t m, int64_t vocab, const void* logits, int64_t ld, int32_t dtype,
                                        const void* tokens, int32_t tokens64, int32_t topk, float* logprob,
                                        float* entropy, int32_t* rank, int32_t* top_ids, float* top_logprobs,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  if (logits == nullptr || tokens == nullptr || logprob == nullptr || entropy == nullptr || rank == nullptr ||
      !logprob_sizes_ok(m, vocab, topk) || (topk > 0 && (top_ids == nullptr || top_logprobs == nullptr)))
    return SKINNY_ERR_INVALID_ARG;
  if (!float_type(dtype)) return SKINNY_ERR_UNSUPPORTED;
  if (ld == 0) ld = vocab;
  if (ld > (1LL << 40)) return SKINNY_ERR_INVALID_ARG;
  if (ld < vocab) return SKINNY_ERR_SHAPE;
  if (!aligned(logits, (uintptr_t)size_of(dtype)) || !aligned(tokens, tokens64 != 0 ? 8 : 4) || !aligned(logprob, 4) ||
      !aligned(entropy, 4) || !aligned(rank, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
    return SKINNY_ERR_ALIGNMENT;
  const int64_t tb = topk > 0 ? m * topk * 4 : 0;
  const struct {
    const void* p;
    int64_t bytes;
  } out[5] = {{logprob, m * 4}, {entropy, m * 4}, {rank, m * 4}, {tb > 0 ? top_ids : nullptr, tb},
              {tb > 0 ? top_logprobs : nullptr, tb}};
  for (int i = 0; i < 5; ++i) {
    if (overlap(out[i].p, out[i].bytes, logits, span(m, ld, vocab, size_of(dtype))) ||
        overlap(out[i].p, out[i].bytes, tokens, m * (tokens64 != 0 ? 8 : 4)))
      return SKINNY_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return SKINNY_ERR_INVALID_ARG;
  }
  const int64_t need = logprob_bytes(m, vocab, topk);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < (size_t)need) return SKINNY_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SKINNY_ERR_ALIGNMENT;
  }
  const RowSegments seg = row_segments(m, vocab);
  LogprobArgs a;
  a.logits = logits;
  a.ld = ld;
  a.vocab = vocab;
  a.m = m;
  a.tokens = tokens;
  a.tokens64 = tokens64 != 0;
  a.topk = topk;
  a.segments = (int32_t)seg.count;
  a.seg_len = (int32_t)seg.len;
  a.waves = seg.waves;
  a.logprob = logprob;
  a.entropy = entropy;
  a.rank = rank;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.counters = need > 0 ? (uint32_t*)workspace : nullptr;
  a.partial = need > 0 ? (float*)((char*)workspace + kRowCounterBytes) : nullptr;
  return hip_status(launch_logprobs(a, kind_of(dtype), (hipStream_t)stream));
}

}  // extern "C"
