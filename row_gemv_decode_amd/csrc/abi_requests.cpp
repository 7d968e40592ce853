// abi_requests.cpp -- the C ABI of the operators of a batch of requests declared
// in include/skinny_requests.h (residual and norm, low-rank adapters, logit
// adjustments): argument validation, all on the host and before any HIP call,
// and dispatch to the kernels in norm.hip, adapters.hip and adjust.hip.
#include <hip/hip_runtime_api.h>
#include <math.h>

#include "abi_checks.h"
#include "requests.h"
#include "skinny_requests.h"

using namespace skinny;

namespace {

constexpr int64_t kMaxLen = 1 << 24;

// a stride that no memory holds `rows` rows of (their bytes, and so the spans below, stay
// within 2^62)
bool too_far(int64_t rows, int64_t ld) { return ld > (1LL << 40) || ld > (1LL << 60) / rows; }

int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }

// An operand of rows: its bytes, for the checks that outputs overlap nothing.
struct Rows {
  const void* p;
  int64_t rows, ld, len, size;
  int64_t bytes() const { return span(rows, ld, len, size); }
};

bool meet(const Rows& a, const Rows& b) { return overlap(a.p, a.bytes(), b.p, b.bytes()); }

// workspace of the adapters: the inner values, then the tiles and their rows
struct AdaptSizes {
  int splits;
  int64_t split_len, max_tiles, tiles, order, bytes;
};
AdaptSizes adapt_sizes(const skinny_adapters& a, int64_t m) {
  AdaptSizes s;
  s.splits = adapt_splits(m, a.k, a.rank, a.count, &s.split_len);
  s.max_tiles = adapt_max_tiles(m, a.count);
  s.tiles = round16((int64_t)s.splits * m * a.rank * 4) + 16;  // (the tile count is before them)
  s.order = s.tiles + s.max_tiles * 16;
  s.bytes = s.order + s.max_tiles * adapt_tile_rows(m) * 4;
  return s;
}

skinny_status check_adapters(const skinny_adapters* a, int64_t m) {
  if (a == nullptr || a->struct_size < sizeof(skinny_adapters)) return SKINNY_ERR_INVALID_ARG;
  if (!half_type(a->dtype)) return SKINNY_ERR_UNSUPPORTED;
  if (m < 1 || m > (1 << 20) || a->count < 1 || a->count > SKINNY_ADAPTERS_MAX || a->rank < 1 ||
      a->rank > SKINNY_ADAPTER_RANK_MAX || a->k < 1 || a->k > kMaxLen || a->n < 1 || a->n > kMaxLen)
    return SKINNY_ERR_INVALID_ARG;
  if (a->rank % 8 != 0 || a->k % 8 != 0) return SKINNY_ERR_SHAPE;
  return SKINNY_OK;
}

}  // namespace

static_assert(SKINNY_ADAPTERS_MAX == kAdaptersMax && SKINNY_ADAPTER_RANK_MAX == kAdapterRankMax, "adapter limits");

extern "C" {

skinny_status skinny_rms_norm_run(int64_t m, int64_t d, const void* x, int64_t ldx, int32_t x_dtype,
                                  const void* residual, int64_t ldr, int32_t r_dtype, const void* weight,
                                  int32_t w_dtype, float eps, void* residual_out, int64_t ldro, void* out, int64_t ldo,
                                  int32_t out_dtype, void* q, int64_t ldq, float* scales, int32_t group, void* stream) {
  if (x == nullptr || (residual_out != nullptr && residual == nullptr) || (q == nullptr) != (scales == nullptr) ||
      (residual_out == nullptr && out == nullptr && q == nullptr))
    return SKINNY_ERR_INVALID_ARG;
  if (!float_type(x_dtype) || (residual != nullptr && !float_type(r_dtype)) ||
      (weight != nullptr && !float_type(w_dtype)) || (out != nullptr && !float_type(out_dtype)) ||
      (q != nullptr && group != 0 && group != 32 && group != 64 && group != 128))
    return SKINNY_ERR_UNSUPPORTED;
  if (m < 1 || m > (1LL << 31) || d < 1 || d > kMaxLen || !(eps >= 0.0f) || !isfinite(eps)) return SKINNY_ERR_INVALID_ARG;
  int64_t* strides[] = {&ldx, &ldr, &ldro, &ldo, &ldq};
  const bool used[] = {true, residual != nullptr, residual_out != nullptr, out != nullptr, q != nullptr};
  for (int i = 0; i < 5; ++i) {
    if (!used[i] || *strides[i] == 0) *strides[i] = d;
    if (too_far(m, *strides[i])) return SKINNY_ERR_INVALID_ARG;
    if (*strides[i] < d) return SKINNY_ERR_SHAPE;
  }
  const int64_t xs = size_of(x_dtype), rs = size_of(r_dtype), os = size_of(out_dtype);
  if (!aligned(x, xs) || !aligned(residual, rs) || !aligned(residual_out, rs) || !aligned(weight, size_of(w_dtype)) ||
      !aligned(out, os) || !aligned(scales, 4))
    return SKINNY_ERR_ALIGNMENT;
  const int64_t groups = q == nullptr ? 0 : group == 0 ? 1 : (d + group - 1) / group;
  const Rows in[] = {{x, m, ldx, d, xs}, {residual, m, ldr, d, rs}, {weight, 1, d, d, size_of(w_dtype)}};
  const Rows res[] = {{residual_out, m, ldro, d, rs}, {out, m, ldo, d, os}, {q, m, ldq, d, 1}, {scales, m, groups, groups, 4}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 3; ++j) {
      const bool same = (i == 0 && j == 1 && residual_out == residual && ldro == ldr) ||
                        (i == 1 && j == 0 && out == x && ldo == ldx && out_dtype == x_dtype);
      if (!same && meet(res[i], in[j])) return SKINNY_ERR_INVALID_ARG;
    }
    for (int j = 0; j < i; ++j)
      if (meet(res[i], res[j])) return SKINNY_ERR_INVALID_ARG;
  }
  NormArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.residual = residual;
  a.ldr = ldr;
  a.weight = weight;
  a.residual_out = residual_out;
  a.ldro = ldro;
  a.out = out;
  a.ldo = ldo;
  a.q = (uint8_t*)q;
  a.ldq = ldq;
  a.scales = scales;
  a.m = m;
  a.d = (int32_t)d;
  a.group = q == nullptr ? 0 : group;
  a.groups = (int32_t)groups;
  a.w_kind = kind_of(w_dtype);
  a.out_kind = kind_of(out_dtype);
  a.eps = eps;
  return hip_status(launch_norm(a, kind_of(x_dtype), kind_of(r_dtype), (hipStream_t)stream));
}

skinny_status skinny_adapters_workspace_size(const skinny_adapters* adapters, int64_t m, size_t* bytes) {
  const skinny_status st = check_adapters(adapters, m);
  if (st != SKINNY_OK) return st;
  if (bytes == nullptr) return SKINNY_ERR_INVALID_ARG;
  *bytes = (size_t)adapt_sizes(*adapters, m).bytes;
  return SKINNY_OK;
}

skinny_status skinny_adapters_run(const skinny_adapters* adapters, int64_t m, const void* x, int64_t ldx,
                                  const void* ids, int32_t ids64, const void* base, int64_t ldb, int32_t base_dtype,
                                  void* out, int64_t ldo, int32_t out_dtype, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  const skinny_status st = check_adapters(adapters, m);
  if (st != SKINNY_OK) return st;
  const skinny_adapters& d = *adapters;
  if (d.A == nullptr || d.B == nullptr || x == nullptr || ids == nullptr || out == nullptr) return SKINNY_ERR_INVALID_ARG;
  if ((base != nullptr && base_dtype != SKINNY_F32 && base_dtype != d.dtype) ||
      (out_dtype != SKINNY_F32 && out_dtype != d.dtype))
    return SKINNY_ERR_UNSUPPORTED;
  if (ldx == 0) ldx = d.k;
  if (ldb == 0 || base == nullptr) ldb = d.n;
  if (ldo == 0) ldo = d.n;
  if (too_far(m, ldx) || too_far(m, ldb) || too_far(m, ldo)) return SKINNY_ERR_INVALID_ARG;
  if (ldx < d.k || ldb < d.n || ldo < d.n) return SKINNY_ERR_SHAPE;
  const int64_t bs = size_of(base_dtype), os = size_of(out_dtype);
  if (ldx % 8 != 0 || !aligned(x, 16) || !aligned(d.A, 16) || !aligned(d.B, 16) || !aligned(d.ranks, 4) ||
      !aligned(d.scaling, 4) || !aligned(ids, ids64 != 0 ? 8 : 4) || !aligned(base, bs) || !aligned(out, os))
    return SKINNY_ERR_ALIGNMENT;
  const Rows to = {out, m, ldo, d.n, os};
  const Rows in[] = {{x, m, ldx, d.k, 2},
                     {d.A, d.count * d.rank, d.k, d.k, 2},
                     {d.B, d.count * d.n, d.rank, d.rank, 2},
                     {d.ranks, 1, d.count, d.count, 4},
                     {d.scaling, 1, d.count, d.count, 4},
                     {ids, 1, m, m, ids64 != 0 ? 8 : 4}};
  const AdaptSizes s = adapt_sizes(d, m);
  const Rows add = {base, m, ldb, d.n, bs}, ws = {workspace, 1, s.bytes, s.bytes, 1};
  for (const Rows& r : in)
    if (meet(to, r) || meet(ws, r)) return SKINNY_ERR_INVALID_ARG;
  const bool same = base == out && ldb == ldo && base_dtype == out_dtype;
  if ((!same && meet(to, add)) || meet(ws, add) || meet(ws, to)) return SKINNY_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < (size_t)s.bytes) return SKINNY_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SKINNY_ERR_ALIGNMENT;
  AdaptArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.A = d.A;
  a.B = d.B;
  a.ranks = d.ranks;
  a.scaling = d.scaling;
  a.ids = ids;
  a.base = base;
  a.ldb = ldb;
  a.out = out;
  a.ldo = ldo;
  a.m = (int32_t)m;
  a.n = (int32_t)d.n;
  a.k = (int32_t)d.k;
  a.rank = (int32_t)d.rank;
  a.count = (int32_t)d.count;
  a.ids64 = ids64 != 0;
  a.base_kind = kind_of(base_dtype);
  a.out_kind = kind_of(out_dtype);
  a.splits = s.splits;
  a.split_len = (int32_t)s.split_len;
  a.h = (float*)workspace;
  a.tile_count = (uint32_t*)((char*)workspace + s.tiles - 16);
  a.tiles = (uint32_t*)((char*)workspace + s.tiles);
  a.order = (uint32_t*)((char*)workspace + s.order);
  a.max_tiles = (int32_t)s.max_tiles;
  return hip_status(launch_adapters(a, kind_of(d.dtype), (hipStream_t)stream));
}

skinny_status skinny_adjust_logits_run(int64_t m, int64_t vocab, const void* logits, int64_t ld, int32_t dtype,
                                       const skinny_logit_rules* rules, void* out, int64_t ldo, int32_t out_dtype,
                                       void* stream) {
  constexpr int64_t kMax = 1LL << 30;
  if (logits == nullptr || rules == nullptr || out == nullptr || rules->struct_size < sizeof(skinny_logit_rules) || m < 1 ||
      m > kMax || vocab < 1 || vocab > kMax || m > (1LL << 50) / vocab)
    return SKINNY_ERR_INVALID_ARG;
  if (!float_type(dtype) || (out_dtype != dtype && out_dtype != SKINNY_F32)) return SKINNY_ERR_UNSUPPORTED;
  const skinny_logit_rules& u = *rules;
  const bool history = u.history != nullptr, bias = u.biases > 0, mask = u.mask != nullptr;
  const int64_t words = (vocab + 31) / 32, token = u.tokens64 != 0 ? 8 : 4;
  // what goes with a history, a list of biases or a mask does not come without it
  if (u.history_len < 0 || u.history_len > kMaxLen || u.biases < 0 || u.biases > (1 << 16) || (history && u.history_len < 1) ||
      (!history && (u.history_len != 0 || u.lengths != nullptr || u.prompt_lengths != nullptr || u.repetition != nullptr ||
                    u.frequency != nullptr || u.presence != nullptr)) ||
      bias != (u.bias_ids != nullptr) || bias != (u.bias_values != nullptr) ||
      (mask ? u.masks < 1 || u.masks > kMax : u.masks != 0 || u.mask_rows != nullptr))
    return SKINNY_ERR_INVALID_ARG;
  const int64_t ldh = u.ldh == 0 || !history ? u.history_len : u.ldh;
  const int64_t ldm = u.ldm == 0 || !mask ? words : u.ldm;
  if (ld == 0) ld = vocab;
  if (ldo == 0) ldo = vocab;
  if (too_far(m, ld) || too_far(m, ldo) || too_far(m, ldh) || too_far(mask ? u.masks : 1, ldm)) return SKINNY_ERR_INVALID_ARG;
  if (ld < vocab || ldo < vocab || ldh < u.history_len || (mask && ldm < words) ||
      (mask && u.mask_rows == nullptr && u.masks < m))
    return SKINNY_ERR_SHAPE;
  const int64_t xs = size_of(dtype), os = size_of(out_dtype);
  if (!aligned(logits, xs) || !aligned(out, os) || !aligned(u.history, token) || !aligned(u.lengths, 4) ||
      !aligned(u.prompt_lengths, 4) || !aligned(u.repetition, 4) || !aligned(u.frequency, 4) || !aligned(u.presence, 4) ||
      !aligned(u.bias_ids, token) || !aligned(u.bias_values, 4) || !aligned(u.mask, 4) || !aligned(u.mask_rows, 4))
    return SKINNY_ERR_ALIGNMENT;
  const Rows to = {out, m, ldo, vocab, os};
  const Rows in[] = {{u.history, m, ldh, u.history_len, token}, {u.lengths, 1, m, m, 4},   {u.prompt_lengths, 1, m, m, 4},
                     {u.repetition, 1, m, m, 4},                {u.frequency, 1, m, m, 4}, {u.presence, 1, m, m, 4},
                     {u.bias_ids, 1, m, m * u.biases, token},   {u.bias_values, 1, m, m * u.biases, 4},
                     {u.mask, u.masks, ldm, words, 4},          {u.mask_rows, 1, m, m, 4}};
  for (const Rows& r : in)
    if (meet(to, r)) return SKINNY_ERR_INVALID_ARG;
  const bool same = out == logits && ld == ldo && dtype == out_dtype;
  if (!same && meet(to, Rows{logits, m, ld, vocab, xs})) return SKINNY_ERR_INVALID_ARG;
  if (same && !history && !bias && !mask) return SKINNY_OK;  // nothing changes
  AdjustArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.out = out;
  a.ldo = ldo;
  a.m = m;
  a.vocab = (int32_t)vocab;
  a.history = u.history;
  a.ldh = ldh;
  a.history_len = (int32_t)u.history_len;
  a.biases = (int32_t)u.biases;
  a.tokens64 = u.tokens64 != 0;
  a.masks = (int32_t)u.masks;
  a.lengths = u.lengths;
  a.prompt_lengths = u.prompt_lengths;
  a.repetition = u.repetition;
  a.frequency = u.frequency;
  a.presence = u.presence;
  a.bias_ids = u.bias_ids;
  a.bias_values = u.bias_values;
  a.mask = u.mask;
  a.ldm = ldm;
  a.mask_rows = u.mask_rows;
  return hip_status(launch_adjust(a, kind_of(dtype), kind_of(out_dtype), (hipStream_t)stream));
}

}  // extern "C"
