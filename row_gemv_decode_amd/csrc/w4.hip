// w4.hip -- the multi-row GEMV on 4-bit weights with group scales, for gfx950
// (MI355X):
//
//   C[r][j] = sum over groups g of  s[j][g] * sum over kk in g of (q[j][kk] - z[j][g]) * A[r][kk]
//
// for r < m <= 16.  HBM-bound: the codes and scales are read once per call for
// all rows.  A workgroup owns CT tiles of 16 columns; its waves take the units
// of 128 elements of k in turn (wave w: units w, w + NW, ...), so at any time
// the workgroup reads NW x 64 consecutive bytes of each of its columns, and
// add their sums in LDS in the order of the waves.  Each wave issues the loads
// of several units before the first product.  The split of k depends on k
// alone, so row i of any window equals the one-row call bit for bit.
#include "window_kernel.h"

namespace skinny {

namespace {

constexpr int kW4Waves = 8;

template <int TK, int WQ, int CT, int UB>
__global__ __launch_bounds__(64 * kW4Waves) void w4_rows_kernel(W4Args g) {
  __shared__ f32x4 red[kW4Waves][CT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 4;
  const int k = (int)g.k;
  const int64_t j0 = (int64_t)blockIdx.x * (16 * CT);

  // rows past m repeat row m - 1: their sums are never stored
  const int row = (lane & 15) < g.m ? (lane & 15) : g.m - 1;
  const uint16_t* arow = (const uint16_t*)g.A + row * g.lda + 8 * h;
  WCol<WQ> col[CT];
  f32x4 tot[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int64_t j = j0 + 16 * c + (lane & 15);
    col[c] = w_col<WQ>(g.codes, g.scales, g.zeros, j < g.n ? j : g.n - 1, g.k, h);  // columns past n: not stored
    tot[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const int units = k / kUnit;
  for (int u = wave; u < units; u += kW4Waves * UB) {
    WRaw<WQ> w[UB][CT];
    u32x4 a[UB][1][4];
#pragma unroll
    for (int b = 0; b < UB; ++b) {
      if (u + b * kW4Waves < units) {  // wave-uniform
#pragma unroll
        for (int c = 0; c < CT; ++c) load_unit<WQ, false>(w[b][c], col[c], u + b * kW4Waves, k, h);
        load_a_unit<false>(a[b][0], arow, u + b * kW4Waves, k);
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // every load above is issued before the first product
#pragma unroll
    for (int b = 0; b < UB; ++b)
      if (u + b * kW4Waves < units) mul_unit<TK, WQ, CT, 1, false>(w[b], a[b], tot, u + b * kW4Waves, k);
  }
  if (k % kUnit != 0 && wave == units % kW4Waves) {
    WRaw<WQ> w[CT];
    u32x4 a[1][4];
#pragma unroll
    for (int c = 0; c < CT; ++c) load_unit<WQ, true>(w[c], col[c], units, k, h);
    load_a_unit<true>(a[0], arow, units, k);
    mul_unit<TK, WQ, CT, 1, true>(w, a, tot, units, k);
  }

#pragma unroll
  for (int c = 0; c < CT; ++c) red[wave][c][lane] = tot[c];
  __syncthreads();
  if (wave < CT) {
    f32x4 sum = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kW4Waves; ++w) sum += red[w][wave][lane];
    const int64_t j = j0 + 16 * wave + (lane & 15);
    if (j < g.n) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * h + e < g.m) store_kind(g.C, (4 * h + e) * g.ldc + j, sum[e], g.c_kind);
    }
  }
}

typedef void (*w4_fn)(W4Args);

template <int TK, int WQ>
w4_fn w4_pick_ct(int ct) {
  return ct == 1 ? w4_rows_kernel<TK, WQ, 1, 4> : ct == 2 ? w4_rows_kernel<TK, WQ, 2, 3> : w4_rows_kernel<TK, WQ, 4, 2>;
}

template <int TK>
w4_fn w4_pick(int group, int ct) {
  return group == 32 ? w4_pick_ct<TK, 32>(ct) : group == 64 ? w4_pick_ct<TK, 64>(ct) : w4_pick_ct<TK, 128>(ct);
}

}  // namespace

hipError_t launch_w4_mm(const W4Args& args, int a_kind, int group, hipStream_t stream) {
  if (args.m < 1 || args.m > kGemvMaxM || args.n < 1 || args.k < 32 || args.k % group != 0 ||
      (group != 32 && group != 64 && group != 128) || (a_kind != CK_F16 && a_kind != CK_BF16))
    return hipErrorInvalidValue;
  const int64_t tiles = (args.n + 15) / 16;
  const int ct = tiles >= 4 * 2048 ? 4 : tiles >= 1024 ? 2 : 1;
  const w4_fn fn = a_kind == CK_F16 ? w4_pick<CK_F16>(group, ct) : w4_pick<CK_BF16>(group, ct);
  hipLaunchKernelGGL(fn, dim3((unsigned)((tiles + ct - 1) / ct)), dim3(64 * kW4Waves), 0, stream, args);
  return hipGetLastError();
}

}  // namespace skinny
