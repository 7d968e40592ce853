// norm.hip -- the residual's addition and a root-mean-square norm, with a 16-
// or 32-bit output and / or one in 8 bits (e4m3) with scales, for gfx950
// (MI355X).
//
//   h = x + r,  y = h w / sqrt(mean(h^2) + eps),  s_g = max|y| / 448,  q = e4m3(y / s_g)
//
// One pass over the data: a row's h stays in registers between the sum of its
// squares and its outputs, and every load of a row (the weight's too) is issued
// before the first arithmetic.  HBM-bound for many rows; for few, one launch
// and one memory round trip.
//
// A lane holds CH chunks of eight consecutive values.  A row of up to 1024
// values belongs to 8 to 64 lanes of one wave, so that no barrier is needed and
// short rows fill a wave together; a longer one to a workgroup of its own.  The
// largest |h w| of a row or group is found beside the sum of squares: rounding keeps
// order, so its product with 1 / sqrt(..) is the largest |y| exactly, and a row's
// waves meet once.
// Rows past 32768 values do not stay in registers and are read twice
// (norm_long_kernel).
// Measured: 16384 x 5120 bf16 to bf16 sums and 8 bits 113 us (5.2 TB/s, what a large
// copy reaches), 2000 x 7681 bf16 23.3 (5.3), 1983 x 896 bf16 on fp32 sums 5.8,
// 1 x 5120 2.8.
//
// q is the fp32 quotient y / s, rounded to 8 bits.  A product with 1 / s alone, 2^-23
// off, moved 184 of 84 million codes across a border; the remainder's correction costs
// two instructions per value (16384 x 5120 113 us with and without, 8192 x 8192 in groups
// of 32 46.6 -> 47.7; divisions 55.6).  |y / s| is at most 448 (1 + 2^-22), which rounds
// to 448, so nothing has to be clamped and a NaN stays one.
#include "requests.h"
#include "vector_io.h"
#include "wave_ops.h"

namespace skinny {

namespace {

constexpr int kNone = -1;  // RK: no residual
constexpr float kTop8 = 448.0f;  // largest e4m3 value
constexpr float kLargest = 3.40282347e38f;
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126: a group of zeros has codes 0, not NaN

// sum or maximum over `lanes` (8 .. 64) consecutive lanes, in all of them; the
// steps past 8 lanes are uniform branches
template <bool MAX>
__device__ __forceinline__ float lanes_reduce(float v, int lanes) {
  auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  v = join(v, dpp_mov<kDppXor1>(v));
  v = join(v, dpp_mov<kDppXor2>(v));
  if (lanes > 4) v = join(v, dpp_mov<kDppRowHalfMirror>(v));
  if (lanes > 8) v = join(v, dpp_mov<kDppRowMirror>(v));
  if (lanes > 16) {
    auto r = __builtin_amdgcn_permlane16_swap(ubits(v), ubits(v), false, false);
    v = join(fbits(r[0]), fbits(r[1]));
  }
  if (lanes > 32) {
    auto r = __builtin_amdgcn_permlane32_swap(ubits(v), ubits(v), false, false);
    v = join(fbits(r[0]), fbits(r[1]));
  }
  return v;
}

// A row's sum and largest value over the waves of a workgroup.  The sums of 64
// consecutive chunks are added up in the lanes of each wave, by the chunks' places, so
// the result does not depend on how many of a row's chunks a lane has.
template <int CH>
__device__ __forceinline__ void block_reduce(float (&sums)[CH], float& sum, float& top, bool both, float (&parts)[16 * CH + 16],
                                             int waves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int c = 0; c < CH; ++c) sums[c] = lanes_reduce<false>(sums[c], 64);
  if (both) top = lanes_reduce<true>(top, 64);
  if (lane == 0) {
#pragma unroll
    for (int c = 0; c < CH; ++c) parts[c * waves + wave] = sums[c];
    parts[16 * CH + wave] = top;
  }
  __syncthreads();
  sum = lanes_reduce<false>(lane < CH * waves ? parts[lane] : 0.0f, 64);
  if (both) top = lanes_reduce<true>(lane < waves ? parts[16 * CH + lane] : 0.0f, 64);
}

// values e0 .. e0 + 7 of a row, 0 from d on.  In a vector where all lie in the
// row (else any eight of it, where it has eight, so that no load is behind a
// branch), and one by one at the row's end.
template <int K>
__device__ __forceinline__ void load8(const void* row, int e0, int d, float (&x)[8]) {
  Raw<K, 8> raw;
  const bool whole = e0 + 8 <= d;
  if (d >= 8) raw = load_raw<K, 8>(row, whole ? e0 : 0);
  if (whole) {
    unpack_raw<K, 8>(raw, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    if (d % 8 != 0 && e0 < d) {
      // (no load behind a branch of its own, where each would be waited for)
      float v[7];
#pragma unroll
      for (int e = 0; e < 7; ++e) v[e] = value_at<K>(row, min(e0 + e, d - 1));
#pragma unroll
      for (int e = 0; e < 7; ++e) x[e] = e0 + e < d ? v[e] : 0.0f;
    }
  }
}

template <int K>
__device__ __forceinline__ void store8(void* row, int e0, int d, const float (&x)[8]) {
  if (e0 + 8 <= d) {
    store_vec<K, 8, true>(row, e0, x);
  } else if (d % 8 != 0) {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e0 + e < d) store_out<K>(row, e0 + e, x[e]);
  }
}

__device__ __forceinline__ void store8_kind(void* row, int kind, int e0, int d, const float (&x)[8]) {
  if (kind == CK_F32) {
    store8<CK_F32>(row, e0, d, x);
  } else if (kind == CK_F16) {
    store8<CK_F16>(row, e0, d, x);
  } else {
    store8<CK_BF16>(row, e0, d, x);
  }
}

__device__ __forceinline__ void load_weight8(const NormArgs& g, int e0, float (&w)[8]) {
  if (g.weight == nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f;
  } else if (g.w_kind == CK_F32) {
    load8<CK_F32>(g.weight, e0, g.d, w);
  } else if (g.w_kind == CK_F16) {
    load8<CK_F16>(g.weight, e0, g.d, w);
  } else {
    load8<CK_BF16>(g.weight, e0, g.d, w);
  }
}

__device__ __forceinline__ float max8(const float (&y)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
  return m;
}

__device__ __forceinline__ float scale_of(float top) { return fmaxf(top / kTop8, kLeastScale); }

// y / s for inv = 1 / s: the product with inv, less what it misses y by, which an fma
// gives exactly (Markstein 1990) while y is above 2^-103: below, the remainder's last
// bits are lost and the quotient may be that of the product.  The signs keep that of a zero.
__device__ __forceinline__ float quotient(float y, float s, float inv) {
  const float q = y * inv;
  const float past = __builtin_fmaf(q, s, -y);
  return __builtin_fmaf(-past, inv, q);
}

__device__ __forceinline__ void store8_q(uint8_t* row, int e0, int d, const float (&y)[8], float s) {
  const float inv = 1.0f / s;
  s = fminf(s, kLargest);  // (an infinite scale's quotients are 0, or its own NaN: by inv alone)
  uint32_t w[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = quotient(y[4 * q + e], s, inv);
    int v = 0;
    v = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], v, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], v, true);
    w[q] = (uint32_t)v;
  }
  if (e0 + 8 <= d) {
    put8<true>(u32x2{w[0], w[1]}, (char*)row + e0);
  } else if (d % 8 != 0) {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e0 + e < d) row[e0 + e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
  }
}

struct RowPtrs {
  const char *x, *r;
  char *ro, *out;
  uint8_t* q;
  float* scales;
};
template <int XK, int RK>
__device__ __forceinline__ RowPtrs row_ptrs(const NormArgs& g, int64_t row) {
  RowPtrs p;
  p.x = (const char*)g.x + row * g.ldx * kind_size<XK>();
  p.r = RK == kNone ? nullptr : (const char*)g.residual + row * g.ldr * kind_size<RK>();
  p.ro = RK == kNone || g.residual_out == nullptr ? nullptr : (char*)g.residual_out + row * g.ldro * kind_size<RK>();
  p.out = g.out == nullptr ? nullptr : (char*)g.out + row * g.ldo * kind_bytes(g.out_kind);
  p.q = g.q == nullptr ? nullptr : g.q + row * g.ldq;
  p.scales = g.q == nullptr ? nullptr : g.scales + row * g.groups;
  return p;
}

// A row of at most 8 CH lanes values.  BLOCK: the lanes of a workgroup, else
// 2^lanes_log2 of a wave's.
template <int XK, int RK, int CH, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? 1024 : 256) void norm_kernel(NormArgs g) {
  __shared__ float parts_s[16 * CH + 16];
  const int tid = threadIdx.x;
  const int lanes = BLOCK ? 64 : 1 << g.lanes_log2;
  const int step = BLOCK ? (int)blockDim.x : lanes;
  const int place = BLOCK ? tid : tid & (lanes - 1);
  const int waves = BLOCK ? (int)blockDim.x >> 6 : 1;
  const int64_t r = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (256 >> g.lanes_log2) + (tid >> g.lanes_log2);
  const bool active = BLOCK || r < g.m;
  const int d = g.d;
  const RowPtrs p = row_ptrs<XK, RK>(g, active ? r : 0);

  float h[CH][8], w[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) load8<XK>(p.x, (c * step + place) * 8, d, h[c]);
  if constexpr (RK != kNone) {
    float res[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) load8<RK>(p.r, (c * step + place) * 8, d, res[c]);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) h[c][e] += res[c][e];
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) load_weight8(g, (c * step + place) * 8, w[c]);

  // w becomes h w
  float sum = 0.0f, sums[CH], top[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    sums[c] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sums[c] = __builtin_fmaf(h[c][e], h[c][e], sums[c]);
      w[c][e] *= h[c][e];
    }
    top[c] = max8(w[c]);
  }
  const bool row_scale = p.q != nullptr && g.group == 0;
  float row_top = top[0];
#pragma unroll
  for (int c = 1; c < CH; ++c) row_top = fmaxf(row_top, top[c]);
  if constexpr (BLOCK) {
    block_reduce<CH>(sums, sum, row_top, row_scale, parts_s, waves);
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) sum += sums[c];
    sum = lanes_reduce<false>(sum, lanes);
    if (row_scale) row_top = lanes_reduce<true>(row_top, lanes);
  }
  const float inv = 1.0f / sqrtf(sum / (float)d + g.eps);

  // (every load of the row has arrived: its rows may be written in place)
  if constexpr (RK != kNone) {
    if (active && p.ro != nullptr) {
#pragma unroll
      for (int c = 0; c < CH; ++c) store8<RK>(p.ro, (c * step + place) * 8, d, h[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) h[c][e] = w[c][e] * inv;
  if (active && p.out != nullptr) {
#pragma unroll
    for (int c = 0; c < CH; ++c) store8_kind(p.out, g.out_kind, (c * step + place) * 8, d, h[c]);
  }
  if (p.q == nullptr) return;
  if (row_scale) {
    const float s = scale_of(row_top * inv);
    if (active) {
#pragma unroll
      for (int c = 0; c < CH; ++c) store8_q(p.q, (c * step + place) * 8, d, h[c], s);
      if (place == 0) p.scales[0] = s;
    }
  } else {
    // a group is group / 8 lanes of one chunk (fewer where the row has fewer)
    const int mine = min(g.group >> 3, lanes);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * step + place) * 8;
      const float s = scale_of(lanes_reduce<true>(top[c], mine) * inv);
      if (active) {
        store8_q(p.q, e0, d, h[c], s);
        if ((place & (mine - 1)) == 0 && e0 < d) p.scales[e0 / g.group] = s;
      }
    }
  }
}

// Rows that do not fit the registers: one workgroup of 1024 per row, which reads
// the row twice.
template <int XK, int RK>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs g) {
  __shared__ float parts_s[32];
  constexpr int kStep = 8 * 1024;
  const int d = g.d;
  const RowPtrs p = row_ptrs<XK, RK>(g, blockIdx.x);
  auto load_both = [&](int e0, float(&h)[8], float(&hw)[8]) {
    load8<XK>(p.x, e0, d, h);
    if constexpr (RK != kNone) {
      float res[8];
      load8<RK>(p.r, e0, d, res);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] += res[e];
    }
    load_weight8(g, e0, hw);
#pragma unroll
    for (int e = 0; e < 8; ++e) hw[e] *= h[e];
  };
  const int first = (int)threadIdx.x * 8;
  const bool row_scale = p.q != nullptr && g.group == 0;
  float sum = 0.0f, sums[1] = {0.0f}, top = 0.0f;
  for (int e0 = first; e0 < d; e0 += kStep) {
    float h[8], hw[8];
    load_both(e0, h, hw);
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fmaf(h[e], h[e], s);
    sums[0] += s;
    top = fmaxf(top, max8(hw));
  }
  block_reduce<1>(sums, sum, top, row_scale, parts_s, 16);
  const float inv = 1.0f / sqrtf(sum / (float)d + g.eps);
  float s = scale_of(top * inv);
  if (row_scale && threadIdx.x == 0) p.scales[0] = s;
  // (all lanes of a wave, so that groups are whole; a value is read and written
  // by one thread, so rows may be written in place)
  for (int e0 = first; e0 - first < d; e0 += kStep) {
    float h[8], y[8];
    load_both(e0, h, y);
    if constexpr (RK != kNone) {
      if (p.ro != nullptr) store8<RK>(p.ro, e0, d, h);
    }
    const float group_top = max8(y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= inv;
    if (p.out != nullptr) store8_kind(p.out, g.out_kind, e0, d, y);
    if (p.q != nullptr) {
      if (g.group != 0) {
        s = scale_of(lanes_reduce<true>(group_top, g.group >> 3) * inv);
        if ((e0 & (g.group - 1)) == 0 && e0 < d) p.scales[e0 / g.group] = s;
      }
      store8_q(p.q, e0, d, y, s);
    }
  }
}

template <int XK, int RK>
hipError_t launch_kinds(NormArgs a, hipStream_t stream) {
  const int chunks = (a.d + 7) / 8;
  const bool block = chunks > 128;
  int threads = 256;
  int64_t rows = 1;  // of a workgroup
  void (*fn)(NormArgs) = nullptr;
  if (!block) {
    a.lanes_log2 = 3;
    while (a.lanes_log2 < 6 && (1 << a.lanes_log2) < chunks) ++a.lanes_log2;
    rows = 256 >> a.lanes_log2;
    fn = chunks > 64 ? norm_kernel<XK, RK, 2, false> : norm_kernel<XK, RK, 1, false>;
  } else if (chunks <= 4 * 1024) {
    // one chunk per lane; two for many long rows, which makes more rows share a CU:
    // 16384 x 5120 to 8 bits 123 -> 113 us, 8192 x 5120 64.7 -> 62.8, but 1 x 5120
    // 2.8 -> 3.2, 256 x 5120 3.5 -> 3.8 and 4096 x 2560 fp32 36.2 -> 39.5
    const int ch = chunks > 2 * 1024 ? 4 : chunks > 1024 || (chunks > 512 && a.m >= 512) ? 2 : 1;
    threads = ((chunks + ch - 1) / ch + 63) / 64 * 64;
    fn = ch == 1 ? norm_kernel<XK, RK, 1, true> : ch == 2 ? norm_kernel<XK, RK, 2, true> : norm_kernel<XK, RK, 4, true>;
  } else {
    threads = 1024;
    fn = norm_long_kernel<XK, RK>;
  }
  const int64_t most = kMaxLaunchThreads / threads / 2 * rows;  // rows of a launch
  for (int64_t r = 0; r < a.m; r += most) {
    NormArgs part = a;
    part.m = a.m - r < most ? a.m - r : most;
    part.x = (const char*)a.x + r * a.ldx * kind_size<XK>();
    if (RK != kNone) {
      part.residual = (const char*)a.residual + r * a.ldr * kind_size<RK>();
      if (a.residual_out != nullptr) part.residual_out = (char*)a.residual_out + r * a.ldro * kind_size<RK>();
    }
    if (a.out != nullptr) part.out = (char*)a.out + r * a.ldo * (a.out_kind == CK_F32 ? 4 : 2);
    if (a.q != nullptr) {
      part.q = a.q + r * a.ldq;
      part.scales = a.scales + r * a.groups;
    }
    hipLaunchKernelGGL(fn, dim3((unsigned)((part.m + rows - 1) / rows)), dim3(threads), 0, stream, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int XK>
hipError_t launch_residual(const NormArgs& a, int r_kind, hipStream_t stream) {
  return a.residual == nullptr ? launch_kinds<XK, kNone>(a, stream)
         : r_kind == CK_F32    ? launch_kinds<XK, CK_F32>(a, stream)
         : r_kind == CK_F16    ? launch_kinds<XK, CK_F16>(a, stream)
                               : launch_kinds<XK, CK_BF16>(a, stream);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int x_kind, int r_kind, hipStream_t stream) {
  if (a.m < 1 || a.d < 1 || (a.group != 0 && a.group != 32 && a.group != 64 && a.group != 128)) return hipErrorInvalidValue;
  return x_kind == CK_F32   ? launch_residual<CK_F32>(a, r_kind, stream)
         : x_kind == CK_F16 ? launch_residual<CK_F16>(a, r_kind, stream)
                            : launch_residual<CK_BF16>(a, r_kind, stream);
}

}  // namespace skinny
