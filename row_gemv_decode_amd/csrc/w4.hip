// w4.hip -- the multi-row GEMV on 4-bit weights with group scales, for gfx950
// (MI355X):
//
//   C[r][j] = sum over groups g of  s[j][g] * sum over kk in g of (q[j][kk] - z[j][g]) * A[r][kk]
//
// for r < m <= 16.  HBM-bound: the codes and scales are read once per call for
// all rows (3 x 100003 x 5120, groups of 128, 265 MB: 66 us, 4.0 TB/s, where a
// large copy moves 4.9 TB/s; below about 10 MB the launch and one round trip to
// HBM are the time).  A workgroup of four waves owns CT tiles of 16 columns; each
// wave takes a quarter of k (a run of units of 128) and streams it with two units
// in flight, and the four sums are added in LDS in the order of the waves.
// The split of k depends on k alone, so row i of any window equals the one-row
// call bit for bit.
#include "window_kernel.h"

namespace skinny {

namespace {

constexpr int kW4Waves = 4;

template <int TK, int WQ, int CT>
__global__ __launch_bounds__(64 * kW4Waves, 2) void w4_rows_kernel(W4Args g) {
  __shared__ ScaleLds<WQ, CT> lds;
  __shared__ u32x4 turn_s[kW4Waves][turn_slots<WQ, CT>() * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 4;
  const int k = (int)g.k;
  // the last workgroup's tiles are moved back inside n (CT > 1 implies n >= 16 CT)
  const int64_t own = (int64_t)blockIdx.x * (16 * CT);
  const int64_t j0 = CT > 1 && own > g.n - 16 * CT ? g.n - 16 * CT : own;

  // rows past m repeat row m - 1: their sums are never stored
  const int row = min(lane >> 2, g.m - 1);
  const uint16_t* arow = (const uint16_t*)g.A + row * g.lda + 8 * (lane & 3);
  int64_t j[CT];
  f32x4 tot[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    j[c] = j0 + 16 * c;
    tot[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  block_product<TK, WQ, CT, kW4Waves>(tot, lds, Turn(turn_s[wave], lane), g.w, j,
                                      CT > 1 ? 16 : (int)min(g.n - j0, (int64_t)16), arow, k, wave, lane);

  put_sums(turn_s[wave], tot, lane);
  __syncthreads();
  if (wave < CT) {
    const f32x4 sum = wave_sums(turn_s, wave, lane);
    const int64_t col = j0 + 16 * wave + (lane & 15);
    if (col >= own && col < g.n) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * h + e < g.m) store_kind(g.C, (4 * h + e) * g.ldc + col, sum[e], g.c_kind);
    }
  }
}

typedef void (*w4_fn)(W4Args);

template <int TK, int WQ>
w4_fn w4_pick_ct(int ct) {
  return ct == 1 ? w4_rows_kernel<TK, WQ, 1> : ct == 2 ? w4_rows_kernel<TK, WQ, 2> : w4_rows_kernel<TK, WQ, 4>;
}

template <int TK, int Z>
w4_fn w4_pick(int group, int ct) {
  return group == 32 ? w4_pick_ct<TK, 32 | Z>(ct) : group == 64 ? w4_pick_ct<TK, 64 | Z>(ct) : w4_pick_ct<TK, 128 | Z>(ct);
}

}  // namespace

hipError_t launch_w4_mm(const W4Args& args, int a_kind, int group, hipStream_t stream) {
  if (args.m < 1 || args.m > kGemvMaxM || args.n < 1 || args.k < 32 || args.k % group != 0 || args.k > kW4MaxK ||
      (group != 32 && group != 64 && group != 128) || (a_kind != CK_F16 && a_kind != CK_BF16))
    return hipErrorInvalidValue;
  constexpr int64_t most = kMaxLaunchThreads / (64 * kW4Waves) * 16;  // columns of a launch, by any rule below
  if (args.n > most) {
    W4Args part = args;
    for (int64_t j = 0; j < args.n; j += most) {
      part.n = args.n - j < most ? args.n - j : most;
      part.w.codes = (const char*)args.w.codes + j * (args.k / 2);
      part.w.scales = (const char*)args.w.scales + j * (args.k / group) * 2;
      if (args.w.zeros != nullptr) part.w.zeros = (const char*)args.w.zeros + j * (args.k / group);
      part.C = (char*)args.C + j * (args.c_kind == CK_F32 ? 4 : 2);
      const hipError_t e = launch_w4_mm(part, a_kind, group, stream);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const int64_t tiles = (args.n + 15) / 16;
  // Column tiles per wave: more tiles share the loads of A, fewer make more
  // workgroups.  Three or four workgroups of one tile are resident per CU, three of
  // two and two of four, so: four tiles where their workgroups make one nearly full
  // round; two where one-tile workgroups would need a second round, or, for groups
  // of 128 (the least work per unit), where the two-tile ones are one per CU at
  // most.  Measured (us on the device, 1 / 2 / 4 tiles):
  //   tiles 304   k 5120 g 128 m 16  12.3 / 11.3 / 15.0   k 4096 g 32 m 4  11.3 / 11.7 / 17.2
  //         480                      12.4 / 11.4 / 14.6                    11.8 / 12.3 / 17.3
  //         768                      17.1 / 16.5 / 16.0                    14.2 / 15.8 / 17.9
  //         1024                     23.9 / 17.6 / 17.1                    16.7 / 16.4 / 19.0
  //         1536                     30.1 / 22.9 / 24.7                    24.2 / 20.0 / 24.8
  //         1664                     33.5 / 28.5 / 25.3  (m 16, as below)  28.2 / 27.1 / 25.4
  //         2000                     37.9 / 29.7 / 26.1                    32.6 / 28.2 / 26.1
  //         2250                     42.3 / 33.7 / 34.8                    36.2 / 31.8 / 38.0
  //         6250                     107 / 79.9 / 76.7                     89.7 / 74.2 / 78.3
  //   k 896 g 32 m 1: 304 4.8 / 5.1 / 6.6, 1536 9.2 / 8.2 / 10.1, 2000 10.5 / 10.2 / 10.8
  // Over 148 random shapes the rule loses 0.3 % to the best of the three.
  const int ct = args.k >= 2048 && tiles >= 1640 && tiles <= 2048            ? 4
                 : tiles > 768 || (group == 128 && tiles > 256 && tiles <= 512) ? 2
                                                                               : 1;
  const w4_fn fn = args.w.zeros == nullptr
                       ? (a_kind == CK_F16 ? w4_pick<CK_F16, 0>(group, ct) : w4_pick<CK_BF16, 0>(group, ct))
                       : (a_kind == CK_F16 ? w4_pick<CK_F16, kZeros>(group, ct) : w4_pick<CK_BF16, kZeros>(group, ct));
  hipLaunchKernelGGL(fn, dim3((unsigned)((tiles + ct - 1) / ct)), dim3(64 * kW4Waves), 0, stream, args);
  return hipGetLastError();
}

}  // namespace skinny
