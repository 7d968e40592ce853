// abi_window.cpp -- the C ABI of the decode window's further operators
// declared in include/skinny.h (4-bit grouped GEMV): argument validation, all
// on the host and before any HIP call, and dispatch to the kernels in w4.hip.
#include <hip/hip_runtime_api.h>

#include "internal.h"
#include "skinny.h"

using namespace skinny;

namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int kind_of(int32_t dt) { return dt == SKINNY_F32 ? CK_F32 : dt == SKINNY_F16 ? CK_F16 : CK_BF16; }
bool half_type(int32_t dt) { return dt == SKINNY_F16 || dt == SKINNY_BF16; }
bool float_type(int32_t dt) { return half_type(dt) || dt == SKINNY_F32; }
int64_t size_of(int32_t dt) { return dt == SKINNY_F32 ? 4 : 2; }

// two byte ranges share a byte (a null pointer shares none)
bool overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

skinny_status hip_status(hipError_t e) { return e == hipSuccess ? SKINNY_OK : SKINNY_ERR_HIP; }

constexpr int64_t kMaxDim = (1LL << 31) - 1;

bool group_ok(int32_t group) { return group == 32 || group == 64 || group == 128; }

// bytes from the first element of row 0 to the last of row rows - 1
int64_t span(int64_t rows, int64_t ld, int64_t len, int64_t size) { return ((rows - 1) * ld + len) * size; }

}  // namespace

extern "C" {

skinny_status skinny_w4_mm_run(int64_t m, int64_t n, int64_t k, int32_t group, const void* A, int64_t lda,
                               int32_t a_dtype, const skinny_w4* W, void* C, int64_t ldc, int32_t c_dtype,
                               void* stream) {
  if (A == nullptr || W == nullptr || C == nullptr || W->codes == nullptr || W->scales == nullptr)
    return SKINNY_ERR_INVALID_ARG;
  if (!half_type(a_dtype) || !float_type(c_dtype) || !group_ok(group)) return SKINNY_ERR_UNSUPPORTED;
  if (m < 1 || m > SKINNY_GEMV_MAX_M || n < 1 || n > kMaxDim || k < 1 || k > kMaxDim) return SKINNY_ERR_INVALID_ARG;
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
  g.codes = W->codes;
  g.scales = W->scales;
  g.zeros = W->zeros;
  g.n = n;
  g.k = k;
  g.C = C;
  g.ldc = ldc;
  g.m = (int32_t)m;
  g.c_kind = kind_of(c_dtype);
  return hip_status(launch_w4_mm(g, kind_of(a_dtype), group, (hipStream_t)stream));
}

}  // extern "C"
