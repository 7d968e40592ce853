// abi_checks.h -- what the argument checks of the C entry points share
// (abi_window.cpp, abi_requests.cpp).  Host code; not installed.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "internal.h"
#include "skinny.h"

namespace skinny {

namespace {

[[maybe_unused]] bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

[[maybe_unused]] int kind_of(int32_t dt) { return dt == SKINNY_F32 ? CK_F32 : dt == SKINNY_F16 ? CK_F16 : CK_BF16; }
[[maybe_unused]] bool half_type(int32_t dt) { return dt == SKINNY_F16 || dt == SKINNY_BF16; }
[[maybe_unused]] bool float_type(int32_t dt) { return half_type(dt) || dt == SKINNY_F32; }
[[maybe_unused]] int64_t size_of(int32_t dt) { return dt == SKINNY_F32 ? 4 : 2; }

// two byte ranges share a byte (a null pointer shares none)
[[maybe_unused]] bool overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

[[maybe_unused]] skinny_status hip_status(hipError_t e) { return e == hipSuccess ? SKINNY_OK : SKINNY_ERR_HIP; }

constexpr int64_t kMaxDim = (1LL << 31) - 1;

// bytes from the first element of row 0 to the last of row rows - 1
[[maybe_unused]] int64_t span(int64_t rows, int64_t ld, int64_t len, int64_t size) { return ((rows - 1) * ld + len) * size; }

}  // namespace

}  // namespace skinny
