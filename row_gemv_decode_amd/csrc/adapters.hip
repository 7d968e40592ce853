// adapters.hip -- low-rank adapters of many requests beside a shared projection,
// for gfx950 (MI355X).
//
//   out_t = base_t + scaling[a] B[a] (A[a] x_t),   a = ids[t]
//
// Two launches.  The first ("down") gives the inner values A x of every row, the
// second ("up") multiplies them by B and adds the base (a few rows with a small A take
// both in one, see takes_one).  Rows of one adapter are
// gathered into tiles, so that 16 rows share one read of the adapter's weights and a
// matrix-core step has rows to multiply.  In batches of more than kAdaptDirectRows rows a
// tile has 64, which share a read of A, and of B where launch_tiles gives whole tiles to a
// workgroup.  For few rows each workgroup finds its tile in the list of
// ids by itself, which costs no more than reading its own id would: a wave
// compares 64 ids per ballot.  For many, one more launch before the two sorts
// the rows by adapter.
//
// Down: v_mfma_f32_16x16x32 over k, which is split over the workgroup's waves and
// over workgroups; the workgroups' parts go to memory in fp32 and the up launch
// adds them in order.  Up: the inner values keep 24 bits as three bf16 planes
// (each the rounded remainder of the last), so that the result is that of fp32
// products; bf16 weights then take three matrix-core steps, and f16 weights,
// which are the exact sum of two bf16 numbers, five (the product of the two
// lowest parts, at most 2^-24, is left out).  Planes in f16 would lose small inner values.
// The work of both is bound by memory: by latency for a few rows, for many by x
// in the one and base and out in the other.  Measured (bf16): 4096 rows of 12 prompts
// with 8 adapters of rank 32, k 5120, n 7680: sort 5 us, down 11 (4.0 TB/s), up 27 (4.7
// TB/s); 250 rows with 64 adapters of rank 16 to 64, k 4096, n 5003: down 8.3, up 17; 1
// row of rank 16, k 2560, n 7680: 7.0 in one launch.
#include "requests.h"
#include "vector_io.h"
#include "window_kernel.h"

namespace skinny {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kNoBase = -1;

__device__ __forceinline__ int id_at(const AdaptArgs& g, int t) {  // -1: no adapter
  const int64_t a = g.ids64 != 0 ? ((const int64_t*)g.ids)[t] : (int64_t)((const int32_t*)g.ids)[t];
  return a >= 0 && a < g.count ? (int)a : -1;
}

__device__ __forceinline__ int rank_of(const AdaptArgs& g, int a) {
  if (a < 0) return 0;
  if (g.ranks == nullptr) return g.rank;
  const int r = g.ranks[a];
  return r >= 1 && r <= g.rank ? r : 0;
}

// Tile `later` of those past an adapter's first 16 rows, in the order of the
// adapters (rows without one last), for at most 256 rows whose ids the lanes
// hold: a wave counts them in LDS of its own.
__device__ __forceinline__ bool later_tile(const AdaptArgs& g, int later, const int (&a)[kAdaptDirectRows / 64], int& adapter,
                                           int& before) {
  __shared__ uint32_t counts_s[kWaves][kAdaptDirectRows] __attribute__((aligned(16)));
  const int lane = threadIdx.x & 63;
  uint32_t* counts = counts_s[threadIdx.x >> 6];
#pragma unroll
  for (int c = 0; c < kAdaptDirectRows / 64; ++c) counts[c * 64 + lane] = 0;
  wave_lds_order();
#pragma unroll
  for (int c = 0; c < kAdaptDirectRows / 64; ++c)
    if (a[c] >= -1) atomicAdd(&counts[a[c] < 0 ? g.count : a[c]], 1u);
  wave_lds_order();
  const u32x4 mine = *(const u32x4*)&counts[4 * lane];
  int tiles[4], sum = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    tiles[q] = mine[q] > 16 ? ((int)mine[q] - 1) / 16 : 0;
    sum += tiles[q];
  }
  int upto = sum;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const int o = __shfl_up(upto, s);
    if (lane >= s) upto += o;
  }
  const uint64_t past = __builtin_amdgcn_ballot_w64(upto > later);
  if (past == 0) return false;
  const int owner = __builtin_ctzll(past);
  int at = later - __builtin_amdgcn_readlane(upto - sum, owner);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int n = __builtin_amdgcn_readlane(tiles[q], owner);
    if (at >= 0 && at < n) {
      adapter = 4 * owner + q < g.count ? 4 * owner + q : -1;
      before = 16 * (at + 1);
    }
    at -= n;
  }
  return true;
}

// A tile as the launches hand it on: its entry of g.tiles, and its rows in
// g.order from `index` times the tile's size on.
struct Tile {
  int adapter, rows, rank;
  float scale;
};
__device__ __forceinline__ u32x4 tile_entry(const AdaptArgs& g, int adapter, int rows) {
  const int rank = rank_of(g, adapter);
  const float scale = rank == 0 || g.scaling == nullptr ? 1.0f : g.scaling[adapter];
  return u32x4{(uint32_t)adapter, (uint32_t)rows, (uint32_t)rank, ubits(scale)};
}
__device__ __forceinline__ Tile tile_of(u32x4 e) {
  const uint32_t scale = e[3];
  return Tile{(int)e[0], (int)e[1], (int)e[2], fbits(scale)};
}

// Tile `index` and its rows in rows_s; false if there is no such tile (the same in
// every thread).  A tile of the sorted list is read by the workgroup; in the direct
// form each wave finds it, and has rows_s to itself.
template <bool LIST>
__device__ __forceinline__ bool find_tile(const AdaptArgs& g, int index, int* rows_s, Tile& tile) {
  if constexpr (LIST) {
    const int tid = threadIdx.x;
    const int tiles = (int)g.tile_count[0];
    const u32x4 entry = ((const u32x4*)g.tiles)[index];
    if (tid < kAdaptTileRows) rows_s[tid] = (int)g.order[index * kAdaptTileRows + tid];
    tile = tile_of(entry);
    __syncthreads();
    return index < tiles;
  } else {
    constexpr int kChunks = kAdaptDirectRows / 64;
    const int lane = threadIdx.x & 63;
    int a[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) a[c] = c * 64 + lane < g.m ? id_at(g, c * 64 + lane) : -2;
    int mine, before = 0, all = 0;  // the tile's adapter, how many of its rows come before the tile
    if (g.by_adapter == 0) {
      // the tile of row `index`, if that row is the first of 16 of its adapter
      mine = __builtin_amdgcn_readfirstlane(id_at(g, index));
    } else if (index <= g.count) {
      mine = index < g.count ? index : -1;
    } else if (!later_tile(g, index - g.count - 1, a, mine, before)) {
      return false;
    }
    uint64_t same[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      same[c] = __builtin_amdgcn_ballot_w64(a[c] == mine);
      if (g.by_adapter == 0) {
        const int below = index - c * 64;  // rows of this chunk that come first
        before += __builtin_popcountll(same[c] & (below <= 0 ? 0 : below >= 64 ? ~0ull : (1ull << below) - 1));
      }
    }
    if ((before & 15) != 0) return false;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int place = all + __builtin_popcountll(same[c] & ((1ull << lane) - 1)) - before;
      if ((same[c] >> lane & 1) != 0 && place >= 0 && place < 16) rows_s[place] = c * 64 + lane;
      all += __builtin_popcountll(same[c]);
    }
    if (all <= before) return false;
    wave_lds_order();
    tile = tile_of(tile_entry(g, mine, min(16, all - before)));
    return true;
  }
}

// --- sorting the rows of a large batch ---------------------------------------
// One workgroup counts the rows of each adapter (those without one last) and gives
// each as many tiles as it needs, one behind the other.  The order of the rows within an
// adapter is that of the atomics; no row's result depends on it.
constexpr int kSortThreads = 1024;
constexpr int kSortIds = 4;  // ids of a thread that are read once and kept

// adds 1 at counts[a] for every active lane and gives the lane its place; a
// wave of one adapter's rows adds once
__device__ __forceinline__ uint32_t take_places(uint32_t* counts, int a, bool active) {
  const uint64_t on = __builtin_amdgcn_ballot_w64(active);
  if (on == 0) return 0;
  const int lane = threadIdx.x & 63;
  const int leader = __builtin_ctzll(on);
  const int first = __builtin_amdgcn_readlane(a, leader);
  if (__builtin_amdgcn_ballot_w64(active && a == first) == on) {
    uint32_t at = 0;
    if (lane == leader) at = atomicAdd(&counts[first], (uint32_t)__builtin_popcountll(on));
    at = (uint32_t)__builtin_amdgcn_readlane((int)at, leader);
    return at + (uint32_t)__builtin_popcountll(on & ((1ull << lane) - 1));
  }
  return active ? atomicAdd(&counts[a], 1u) : 0;
}

__global__ __launch_bounds__(kSortThreads) void adapter_sort_kernel(AdaptArgs g) {
  extern __shared__ uint32_t counts_s[];  // count + 1
  __shared__ uint32_t tiles_s[kSortThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int places = g.count + 1;
  auto place_of = [&](int t) {
    const int a = id_at(g, min(t, g.m - 1));
    return a < 0 ? g.count : a;
  };
  // (a batch whose ids are kept takes its places while it is counted)
  const bool once = g.m <= kSortIds * kSortThreads;
  int kept[kSortIds];
  uint32_t place[kSortIds];
  if (once) {
#pragma unroll
    for (int i = 0; i < kSortIds; ++i) kept[i] = place_of(i * kSortThreads + tid);
  }
  // each thread's consecutive adapters; the first one's rank and scaling are in flight
  const int each = (places + kSortThreads - 1) / kSortThreads;
  const int a0 = tid * each, a1 = min(a0 + each, places);
  const u32x4 entry0 = tile_entry(g, a0 < g.count ? a0 : -1, 0);
  for (int i = tid; i < places; i += kSortThreads) counts_s[i] = 0;
  __syncthreads();
  if (once) {
#pragma unroll
    for (int i = 0; i < kSortIds; ++i) place[i] = take_places(counts_s, kept[i], i * kSortThreads + tid < g.m);
  } else {
    for (int t0 = 0; t0 < g.m; t0 += kSortThreads) take_places(counts_s, place_of(t0 + tid), t0 + tid < g.m);
  }
  __syncthreads();
  // their tiles, then the sums of the threads before it
  uint32_t tiles = 0;
  for (int a = a0; a < a1; ++a) tiles += (counts_s[a] + kAdaptTileRows - 1) / kAdaptTileRows;
  uint32_t tile_at = tiles;  // inclusive sum over the wave
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const uint32_t t = (uint32_t)__shfl_up((int)tile_at, s);
    if (lane >= s) tile_at += t;
  }
  if (lane == 63) tiles_s[wave] = tile_at;
  __syncthreads();
  tile_at -= tiles;
  for (int i = 0; i < wave; ++i) tile_at += tiles_s[i];
  if (tid == kSortThreads - 1) g.tile_count[0] = tile_at + tiles;
  for (int a = a0; a < a1; ++a) {
    const uint32_t count = counts_s[a];
    counts_s[a] = tile_at * kAdaptTileRows;  // where the adapter's rows start
    if (count == 0) continue;
    u32x4 entry = a == a0 ? entry0 : tile_entry(g, a < g.count ? a : -1, 0);
    for (uint32_t done = 0; done < count; done += kAdaptTileRows) {
      entry[1] = min(count - done, (uint32_t)kAdaptTileRows);
      ((u32x4*)g.tiles)[tile_at++] = entry;
    }
  }
  __syncthreads();
  if (once) {
#pragma unroll
    for (int i = 0; i < kSortIds; ++i)
      if (i * kSortThreads + tid < g.m) g.order[counts_s[kept[i]] + place[i]] = (uint32_t)(i * kSortThreads + tid);
  } else {
    for (int t0 = 0; t0 < g.m; t0 += kSortThreads) {
      const bool on = t0 + tid < g.m;
      const uint32_t at = take_places(counts_s, place_of(t0 + tid), on);
      if (on) g.order[at] = (uint32_t)(t0 + tid);
    }
  }
}

// --- down: the inner values --------------------------------------------------
// A workgroup: 16 TR rows, 16 NR ranks, one split of k.  Its waves take every
// fourth 64 elements of the split (128 bytes of a row), UN of them at once.
template <int TR, int NR>
constexpr int down_units() { return TR == 1 ? (NR == 1 ? 4 : 2) : (NR == 1 ? 2 : 1); }

template <int TK, int TR, int NR>
__global__ __launch_bounds__(kThreads) void adapter_down_kernel(AdaptArgs g) {
  constexpr bool LIST = TR > 1;
  constexpr int UN = down_units<TR, NR>();
  extern __shared__ f32x4 sums_s[];  // the waves' slots, then [waves][TR][NR][64]
  __shared__ int lists_s[LIST ? 16 * TR : 16 * kWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = (int)blockIdx.x % g.splits;
  const int rank0 = (int)blockIdx.x / g.splits * (16 * NR);
  int* rows_s = lists_s + (LIST ? 0 : 16 * wave);
  Tile tile;
  const bool found = find_tile<LIST>(g, blockIdx.y, rows_s, tile);
  if (!LIST && blockIdx.x == 0 && wave == 0) {  // for the up launch
    if (lane < 16 && found) g.order[blockIdx.y * 16 + lane] = (uint32_t)rows_s[lane];
    if (lane == 0)
      ((u32x4*)g.tiles)[blockIdx.y] =
          found ? u32x4{(uint32_t)tile.adapter, (uint32_t)tile.rows, (uint32_t)tile.rank, ubits(tile.scale)} : u32x4{0, 0, 0, 0};
  }
  if (!found || rank0 >= tile.rank) return;
  const int rank = tile.rank;

  // a load gives four consecutive lanes 64 bytes of a row, which pass through the
  // wave's slots of LDS to the lanes that multiply them (see Turn)
  const int row4 = lane >> 2, piece = lane & 3;
  const uint16_t* x[TR];
#pragma unroll
  for (int t = 0; t < TR; ++t) {
    const int i = t * 16 + row4;
    x[t] = (const uint16_t*)g.x + rows_s[i < tile.rows ? i : 0] * g.ldx + 8 * piece;
  }
  const uint16_t* w[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int j = rank0 + n * 16 + row4;
    w[n] = (const uint16_t*)g.A + ((int64_t)tile.adapter * g.rank + (j < rank ? j : 0)) * g.k + 8 * piece;
  }
  const int begin = split * g.split_len;
  const int len = min(g.split_len, g.k - begin);
  const int units = (len + 63) / 64;
  const Turn turn((u32x4*)sums_s + wave * (2 * (TR + NR) * 64), lane);
  f32x4 acc[TR][NR];
#pragma unroll
  for (int t = 0; t < TR; ++t)
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[t][n] = f32x4{0, 0, 0, 0};
  for (int u0 = wave; u0 < units; u0 += kWaves * UN) {
    u32x4 xf[UN][2][TR], wf[UN][2][NR];
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        // past the split: any elements of the row, which count as 0
        const int at = (u0 + u * kWaves) * 64 + b * 32;
        const bool in = at + 8 * piece < len;
        const int k0 = in ? begin + at : -8 * piece;
#pragma unroll
        for (int t = 0; t < TR; ++t) {
          const u32x4 v = *(const u32x4*)(x[t] + k0);
          xf[u][b][t] = in ? v : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) wf[u][b][n] = *(const u32x4*)(w[n] + k0);
      }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      wave_lds_order();
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int t = 0; t < TR; ++t) turn.slots[(b * (TR + NR) + t) * 64 + turn.put] = xf[u][b][t];
#pragma unroll
        for (int n = 0; n < NR; ++n) turn.slots[(b * (TR + NR) + TR + n) * 64 + turn.put] = wf[u][b][n];
      }
      wave_lds_order();
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int t = 0; t < TR; ++t) xf[u][b][t] = turn.slots[(b * (TR + NR) + t) * 64 + turn.get];
#pragma unroll
        for (int n = 0; n < NR; ++n) wf[u][b][n] = turn.slots[(b * (TR + NR) + TR + n) * 64 + turn.get];
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int t = 0; t < TR; ++t)
#pragma unroll
          for (int n = 0; n < NR; ++n) acc[t][n] = mfma16<TK>(wf[u][b][n], xf[u][b][t], acc[t][n]);
    }
  }
  const int low = lane & 15, h = lane >> 4;
  __syncthreads();  // (the slots are the sums' place too)
  // a lane holds ranks 4 h .. 4 h + 3 of row low: the waves' parts are added in
  // the order of the waves
#pragma unroll
  for (int t = 0; t < TR; ++t)
#pragma unroll
    for (int n = 0; n < NR; ++n) sums_s[((wave * TR + t) * NR + n) * 64 + lane] = acc[t][n];
  __syncthreads();
#pragma unroll
  for (int i0 = 0; i0 < TR * NR; i0 += kWaves) {
    const int i = i0 + wave;
    if (TR * NR < kWaves && i >= TR * NR) break;
    f32x4 s = sums_s[i * 64 + lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) s += sums_s[(v * TR * NR + i) * 64 + lane];
    const int row = i / NR * 16 + low, j = rank0 + i % NR * 16 + 4 * h;
    if (row < tile.rows && j < rank)
      *(f32x4*)(g.h + ((int64_t)split * g.m + rows_s[row]) * g.rank + j) = s;
  }
}

// --- up: B's product and the sum ---------------------------------------------
constexpr int kPlanes = 3;
constexpr int kColTiles = 4;               // 16 columns each, per wave
constexpr int kWaveCols = 16 * kColTiles;  // a lane holds kColTiles consecutive columns of its rows
constexpr int kBlockCols = kWaveCols * kWaves;

// the remainder of v past its rounding to bf16, which is left in `bits`
__device__ __forceinline__ float bf16_plane(float v, uint16_t& bits) {
  bits = f32_half<CK_BF16>(v);
  return v - f32_from_bits((uint32_t)bits << 16);
}

// eight f16 weights as the sum of two bf16 numbers each
__device__ __forceinline__ void f16_planes(u32x4 w, u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t u = w[q];
    const h2_t v = as_h2(u);
    const float a = (float)v[0], b = (float)v[1];
    const uint32_t top = pack2<CK_BF16>(a, b);
    hi[q] = top;
    lo[q] = pack2<CK_BF16>(a - f32_from_bits(top << 16), b - f32_from_bits(top & 0xffff0000u));
  }
}

// B's fragments of a wave's 64 columns for one step of 32 ranks.  As loaded: the
// adapter's ranks of the step are `parts` pieces of 16 bytes of each column, and
// consecutive lanes take a column's pieces one after another (so a load of an
// adapter of rank 16 covers 32 columns).  They then pass through the wave's slots of
// LDS (see Turn): lane (low, h) takes piece h of columns 4 low .. 4 low + 3.
template <int TK>
struct WeightFrags {
  u32x4 hi[kColTiles], lo[TK == CK_F16 ? kColTiles : 1];
};
__device__ __forceinline__ int step_parts_log2(int rank, int step) {
  const int left = rank - 32 * step;
  return left > 16 ? 2 : left > 8 ? 1 : 0;
}
template <int TK>
__device__ __forceinline__ void load_frags(const AdaptArgs& g, const uint16_t* wb, int rank, int step, int col, int lane,
                                           WeightFrags<TK>& w) {
  const int log2 = step_parts_log2(rank, step);
  const int piece = 32 * step + 8 * (lane & ((1 << log2) - 1));
  const uint16_t* at = wb + (piece < rank ? piece : 32 * step);
#pragma unroll
  for (int i = 0; i < kColTiles; ++i)
    if (i < 1 << log2) {
      const int c = col + ((i * 64 + lane) >> log2);
      w.hi[i] = *(const u32x4*)(at + (int64_t)min(c, g.n - 1) * g.rank);
    }
}
template <int TK>
__device__ __forceinline__ void finish_frags(int rank, int step, int lane, u32x4* slots, WeightFrags<TK>& w) {
  const int log2 = step_parts_log2(rank, step);
  const int low = lane & 15, h = lane >> 4;
  wave_lds_order();
#pragma unroll
  for (int i = 0; i < kColTiles; ++i)
    if (i < 1 << log2) {
      const int c = (i * 64 + lane) >> log2;
      slots[(c & 3) * 64 + Turn::entry(c >> 2, lane & ((1 << log2) - 1))] = w.hi[i];
    }
  wave_lds_order();
  const int valid = rank - 32 * step - 8 * h;  // elements of this lane's eight that count
  u32x4 keep;
#pragma unroll
  for (int q = 0; q < 4; ++q) keep[q] = valid >= 2 * q + 2 ? ~0u : valid == 2 * q + 1 ? 0xffffu : 0u;
#pragma unroll
  for (int s = 0; s < kColTiles; ++s) {
    w.hi[s] = slots[s * 64 + Turn::entry(low, h)] & keep;
    if constexpr (TK == CK_F16) f16_planes(w.hi[s], w.hi[s], w.lo[s]);
  }
}

// acc[s] += the inner values' planes times one step of column tile s; `planes` is the
// lane's piece of its row's first plane.  The smallest products come first.
template <int TK>
__device__ __forceinline__ void multiply_step(const uint16_t* planes, int plane, const WeightFrags<TK>& f,
                                              f32x4 (&acc)[kColTiles]) {
  u32x4 v[kPlanes];
#pragma unroll
  for (int p = 0; p < kPlanes; ++p) v[p] = *(const u32x4*)(planes + p * plane);
#pragma unroll
  for (int p = kPlanes - 1; p >= 0; --p) {
    if constexpr (TK == CK_F16) {
      if (p < kPlanes - 1) {
#pragma unroll
        for (int s = 0; s < kColTiles; ++s) acc[s] = mfma16<CK_BF16>(v[p], f.lo[s], acc[s]);
      }
    }
#pragma unroll
    for (int s = 0; s < kColTiles; ++s) acc[s] = mfma16<CK_BF16>(v[p], f.hi[s], acc[s]);
  }
}

// four inner values in their planes, at one place of each
__device__ __forceinline__ void store_planes(uint16_t* at, int plane, const float (&v)[4]) {
  uint16_t bits[kPlanes][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float rest = v[q];
#pragma unroll
    for (int p = 0; p < kPlanes; ++p) rest = bf16_plane(rest, bits[p][q]);
  }
#pragma unroll
  for (int p = 0; p < kPlanes; ++p)
    *(u32x2*)(at + p * plane) = u32x2{bits[p][0] | (uint32_t)bits[p][1] << 16, bits[p][2] | (uint32_t)bits[p][3] << 16};
}

// The base of rows 4 h .. 4 h + 3 of the 16 from rows_s on, at columns c0 .. c0 + 3.
// Vectors that pass n are read at column 0 and not used, and so are rows past `rows`.
template <int BK>
using BaseVec = Raw<BK == kNoBase ? CK_F32 : BK, kColTiles>;
template <int BK, typename R>
__device__ __forceinline__ void load_base(const AdaptArgs& g, const R* rows_s, int rows, int h, int c0, BaseVec<BK> (&v)[4]) {
  if constexpr (BK != kNoBase) {
    if (g.n < kColTiles) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t row = rows_s[4 * h + q < rows ? 4 * h + q : 0];
      v[q] = load_raw<BK, kColTiles>(g.base, row * g.ldb + (c0 + kColTiles <= g.n ? c0 : 0));
    }
  }
}

// the lane's rows and columns of the output: the base plus sum[column][row]
template <int TK, int BK, typename R>
__device__ __forceinline__ void store_rows(const AdaptArgs& g, const R* rows_s, int rows, int h, int c0, bool add,
                                           const BaseVec<BK> (&base)[4], const float (&sum)[kColTiles][4]) {
  const bool whole = c0 + kColTiles <= g.n;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (4 * h + q >= rows) continue;
    const int64_t row = rows_s[4 * h + q];
    float v[kColTiles];
#pragma unroll
    for (int s = 0; s < kColTiles; ++s) v[s] = 0.0f;
    if constexpr (BK != kNoBase) {
      if (whole) {
        unpack_raw<BK, kColTiles>(base[q], v);
      } else {
#pragma unroll
        for (int s = 0; s < kColTiles; ++s)
          if (c0 + s < g.n) v[s] = value_at<BK>(g.base, row * g.ldb + c0 + s);
      }
    }
    if (add) {
#pragma unroll
      for (int s = 0; s < kColTiles; ++s) v[s] += sum[s][q];
    }
    const int64_t at = row * g.ldo + c0;
    if (whole) {
      if (g.out_kind == CK_F32) {
        store_vec<CK_F32, kColTiles, true>(g.out, at, v);
      } else {
        store_vec<TK, kColTiles, true>(g.out, at, v);
      }
    } else {
#pragma unroll
      for (int s = 0; s < kColTiles; ++s)
        if (c0 + s < g.n) {
          if (g.out_kind == CK_F32) {
            store_out<CK_F32>(g.out, at + s, v[s]);
          } else {
            store_out<TK>(g.out, at + s, v[s]);
          }
        }
    }
  }
}

constexpr int kLongSteps = 4;  // held of a long rank, where whole tiles of 64 rows take it
// whether the next columns' fragments fit beside those held (else col_blocks is 1)
template <int TK, int HELD>
constexpr bool holds_next() { return HELD > 0 && (HELD < kLongSteps || TK == CK_BF16); }

// A workgroup: 16 TR rows of a tile, col_blocks times kBlockCols columns, 64 of them
// per wave.  HELD: steps of 32 ranks whose fragments of B stay in registers over the
// tile's rows (0: the steps follow one another, with running totals of its 16 rows).
// The matrix core's sums are read in the straight line of code that forms them (the
// hardware does not hold back a read that comes too early, and the compiler has
// missed some behind branches): all HELD steps are multiplied, with zeros past the
// adapter's rank.
template <int TK, int TR, int BK, int HELD>
__global__ __launch_bounds__(kThreads) void adapter_up_kernel(AdaptArgs g, int col_blocks) {
  extern __shared__ uint16_t planes_s[] __attribute__((aligned(16)));  // [planes][16 TR][pitch]
  __shared__ uint32_t rows_s[16 * TR];
  __shared__ u32x4 slots_s[kWaves][64 * kColTiles];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int low = lane & 15, h = lane >> 4;
  const bool list = TR > 1 || g.m > kAdaptDirectRows;
  const uint32_t tiles = list ? g.tile_count[0] : gridDim.y;
  Tile tile = tile_of(((const u32x4*)g.tiles)[blockIdx.y]);
  const int part = (int)blockIdx.z * (16 * TR);  // of the tile's rows
  if (tid < 16 * TR) rows_s[tid] = g.order[blockIdx.y * (list ? kAdaptTileRows : 16) + part + tid];
  tile.rows = min(tile.rows - part, 16 * TR);
  if (blockIdx.y >= tiles || tile.rows <= 0) return;
  const int rank = tile.rank;
  if (rank == 0 && g.out == g.base) return;  // nothing to add
  const float scale = tile.scale;
  const int steps = (rank + 31) / 32;
  const int pitch = (HELD > 0 ? HELD : (g.rank + 31) / 32) * 32 + 8;
  const uint16_t* wb = (const uint16_t*)g.B + (int64_t)max(tile.adapter, 0) * g.n * g.rank;
  __syncthreads();

  const int wave_col = (int)blockIdx.x * col_blocks * kBlockCols + wave * kWaveCols;
  const int first = wave_col + low * kColTiles;
  BaseVec<BK> base[4];
  WeightFrags<TK> w[HELD > 0 ? HELD : 1];
  // (in flight while the inner values are added up)
  load_base<BK>(g, rows_s, tile.rows, h, first, base);
#pragma unroll
  for (int b = 0; b < HELD; ++b)
    if (b < steps) load_frags<TK>(g, wb, rank, b, wave_col, lane, w[b]);

  // the rows' inner values: the splits' parts in order, four ranks per thread
  const int quads = (HELD > 0 ? HELD : steps) * 8;
  for (int e = tid; e < tile.rows * quads; e += kThreads) {
    const int row = e / quads, j = e % quads * 4;
    f32x4 v = f32x4{0, 0, 0, 0};
    if (j < rank) {
      const float* part = g.h + (int64_t)rows_s[row] * g.rank + j;
      const int64_t stride = (int64_t)g.m * g.rank;
      for (int s0 = 0; s0 < g.splits; s0 += 8) {
        f32x4 p[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) p[s] = *(const f32x4*)(part + min(s0 + s, g.splits - 1) * stride);
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s0 + s < g.splits) v += p[s];
      }
    }
    float kept[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) kept[q] = j + q < rank ? v[q] : 0.0f;
    store_planes(planes_s + row * pitch + j, 16 * TR * pitch, kept);
  }
  __syncthreads();

  for (int cb = 0; cb < col_blocks; ++cb) {
    const int col = wave_col + cb * kBlockCols, c0 = col + low * kColTiles;
    if (col >= g.n) break;
    WeightFrags<TK> next_w[HELD > 0 ? HELD : 1];  // the next columns'
    if (holds_next<TK, HELD>() && cb + 1 < col_blocks) {
#pragma unroll
      for (int b = 0; b < HELD; ++b)
        if (b < steps) load_frags<TK>(g, wb, rank, b, col + kBlockCols, lane, next_w[b]);
    }
    auto multiply = [&](int t, int b, const WeightFrags<TK>& f, f32x4(&acc)[kColTiles]) __attribute__((always_inline)) {
      multiply_step<TK>(planes_s + (t * 16 + low) * pitch + b * 32 + 8 * h, 16 * TR * pitch, f, acc);
    };
    float total[kColTiles][4];
    if constexpr (HELD > 0) {
#pragma unroll
      for (int b = 0; b < HELD; ++b) finish_frags<TK>(rank, b, lane, slots_s[wave], w[b]);
    } else {
      static_assert(TR == 1, "running totals are those of 16 rows");
#pragma unroll
      for (int s = 0; s < kColTiles; ++s)
#pragma unroll
        for (int q = 0; q < 4; ++q) total[s][q] = 0.0f;
      if (steps > 0) load_frags<TK>(g, wb, rank, 0, col, lane, w[0]);
      for (int b = 0; b < steps; ++b) {
        if (b + 1 < steps) load_frags<TK>(g, wb, rank, b + 1, col, lane, next_w[0]);
        finish_frags<TK>(rank, b, lane, slots_s[wave], w[0]);
        f32x4 acc[kColTiles];
#pragma unroll
        for (int s = 0; s < kColTiles; ++s) acc[s] = f32x4{0, 0, 0, 0};
        multiply(0, b, w[0], acc);
#pragma unroll
        for (int s = 0; s < kColTiles; ++s)
#pragma unroll
          for (int q = 0; q < 4; ++q) total[s][q] = __builtin_fmaf(scale, acc[s][q], total[s][q]);
#pragma unroll
        for (int s = 0; s < kColTiles; ++s) w[0].hi[s] = next_w[0].hi[s];
      }
    }
    auto sixteen_rows = [&](int t) __attribute__((always_inline)) {
      // the next rows' base, or that of the next columns' first rows
      BaseVec<BK> next[4];
      if (TR > 1 && (t + 1) * 16 < tile.rows) {
        load_base<BK>(g, rows_s + (t + 1) * 16, tile.rows - (t + 1) * 16, h, c0, next);
      } else if (cb + 1 < col_blocks) {
        load_base<BK>(g, rows_s, tile.rows, h, c0 + kBlockCols, next);
      }
      float sum[kColTiles][4];
      if constexpr (HELD > 0) {
        f32x4 acc[kColTiles];
#pragma unroll
        for (int s = 0; s < kColTiles; ++s) acc[s] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < HELD; ++b) multiply(t, b, w[b], acc);
#pragma unroll
        for (int s = 0; s < kColTiles; ++s)
#pragma unroll
          for (int q = 0; q < 4; ++q) sum[s][q] = scale * acc[s][q];
      } else {
#pragma unroll
        for (int s = 0; s < kColTiles; ++s)
#pragma unroll
          for (int q = 0; q < 4; ++q) sum[s][q] = total[s][q];
      }
      store_rows<TK, BK>(g, rows_s + t * 16, tile.rows - t * 16, h, c0, rank != 0, base, sum);
      if (TR > 1 || cb + 1 < col_blocks) {
#pragma unroll
        for (int q = 0; q < 4; ++q) base[q] = next[q];
      }
    };
    if constexpr (TR == 1) {
      sixteen_rows(0);
    } else {
#pragma unroll 1
      for (int t = 0; t * 16 < tile.rows; ++t) sixteen_rows(t);
    }
    if (holds_next<TK, HELD>() && cb + 1 < col_blocks) {
#pragma unroll
      for (int b = 0; b < HELD; ++b)
#pragma unroll
        for (int s = 0; s < kColTiles; ++s) w[b].hi[s] = next_w[b].hi[s];
    }
  }
}

// --- both in one launch --------------------------------------------------------
// For few rows and a small A: each workgroup of the up product computes its tile's
// inner values by itself, which costs a read of the adapter's A from L2 and saves
// the other launch and the way through memory.  The loads of all splits of k, of B
// and of the base are in flight together.  Waves, splits and additions are those of
// the two launches, and so are the bits, so the choice may depend on the rows.
constexpr int kOneSplits = 4;
constexpr int kOnePitch = 32 + 8;
constexpr int64_t kOneReads = 10 << 20;  // elements of A
constexpr int64_t kOneReadsMany = 2 << 20;  // and for more than 64 rows

template <int TK, int BK, int NR>
__global__ __launch_bounds__(kThreads) void adapter_one_kernel(AdaptArgs g) {
  constexpr int UN = NR == 1 ? 4 : 2;  // units of a wave in a split: 1024 or 512 elements
  constexpr int kSlots = 2 * (1 + NR) > kColTiles ? 2 * (1 + NR) : kColTiles;
  __shared__ u32x4 slots_s[kWaves][64 * kSlots];
  __shared__ f32x4 sums_s[kOneSplits][kWaves][NR][64];
  __shared__ uint16_t planes_s[kPlanes * 16 * kOnePitch] __attribute__((aligned(16)));
  __shared__ int lists_s[16 * kWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int low = lane & 15, h = lane >> 4;
  int* rows_s = lists_s + 16 * wave;
  Tile tile;
  if (!find_tile<false>(g, blockIdx.y, rows_s, tile)) return;
  const int rank = tile.rank;
  if (rank == 0 && g.out == g.base) return;  // nothing to add
  const int col = ((int)blockIdx.x * kWaves + wave) * kWaveCols, c0 = col + low * kColTiles;
  BaseVec<BK> base[4];
  WeightFrags<TK> f;

  if (rank > 0) {
    const int row4 = lane >> 2, piece = lane & 3;
    const uint16_t* x = (const uint16_t*)g.x + rows_s[row4 < tile.rows ? row4 : 0] * g.ldx + 8 * piece;
    const uint16_t* w[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int j = n * 16 + row4;
      w[n] = (const uint16_t*)g.A + ((int64_t)tile.adapter * g.rank + (j < rank ? j : 0)) * g.k + 8 * piece;
    }
    const Turn turn(slots_s[wave], lane);
    u32x4 xf[kOneSplits][UN][2], wf[kOneSplits][UN][2][NR];
#pragma unroll
    for (int p = 0; p < kOneSplits; ++p)
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int unit = p * g.split_len + (wave + u * kWaves) * 64;
        if (unit >= g.k) break;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          // past the row: any elements of it, which count as 0
          const int at = unit + b * 32;
          const int k0 = at + 8 * piece < g.k ? at : -8 * piece;
          xf[p][u][b] = *(const u32x4*)(x + k0);
#pragma unroll
          for (int n = 0; n < NR; ++n) wf[p][u][b][n] = *(const u32x4*)(w[n] + k0);
        }
      }
    load_base<BK>(g, rows_s, tile.rows, h, c0, base);
    load_frags<TK>(g, (const uint16_t*)g.B + (int64_t)tile.adapter * g.n * g.rank, rank, 0, col, lane, f);
#pragma unroll
    for (int p = 0; p < kOneSplits; ++p) {
      if (p >= g.splits) break;
      f32x4 acc[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) acc[n] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int unit = p * g.split_len + (wave + u * kWaves) * 64;
        wave_lds_order();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const bool in = unit + b * 32 + 8 * piece < g.k;
          turn.slots[b * (1 + NR) * 64 + turn.put] = in ? xf[p][u][b] : u32x4{0, 0, 0, 0};
#pragma unroll
          for (int n = 0; n < NR; ++n)
            turn.slots[(b * (1 + NR) + 1 + n) * 64 + turn.put] = unit < g.k ? wf[p][u][b][n] : u32x4{0, 0, 0, 0};
        }
        wave_lds_order();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const u32x4 a = turn.slots[b * (1 + NR) * 64 + turn.get];
#pragma unroll
          for (int n = 0; n < NR; ++n) acc[n] = mfma16<TK>(turn.slots[(b * (1 + NR) + 1 + n) * 64 + turn.get], a, acc[n]);
        }
      }
#pragma unroll
      for (int n = 0; n < NR; ++n) sums_s[p][wave][n][lane] = acc[n];
    }
  } else {
    load_base<BK>(g, rows_s, tile.rows, h, c0, base);
  }
  __syncthreads();
  // a wave for each 16 ranks of the step: the waves' parts of a split, then the splits
  if (rank > 0 && wave < 2) {
    f32x4 v = {0, 0, 0, 0};
    if (wave < NR) {
      for (int p = 0; p < g.splits; ++p) {
        f32x4 s = sums_s[p][0][wave < NR ? wave : 0][lane];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) s += sums_s[p][i][wave < NR ? wave : 0][lane];
        v += s;
      }
    }
    float kept[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) kept[q] = 16 * wave + 4 * h + q < rank ? v[q] : 0.0f;
    store_planes(planes_s + low * kOnePitch + 16 * wave + 4 * h, 16 * kOnePitch, kept);
  }
  __syncthreads();
  if (col >= g.n) return;
  finish_frags<TK>(rank, 0, lane, slots_s[wave], f);
  f32x4 acc[kColTiles];
#pragma unroll
  for (int s = 0; s < kColTiles; ++s) acc[s] = f32x4{0, 0, 0, 0};
  multiply_step<TK>(planes_s + low * kOnePitch + 8 * h, 16 * kOnePitch, f, acc);
  float sum[kColTiles][4];
#pragma unroll
  for (int s = 0; s < kColTiles; ++s)
#pragma unroll
    for (int q = 0; q < 4; ++q) sum[s][q] = tile.scale * acc[s][q];
  store_rows<TK, BK>(g, rows_s, tile.rows, h, c0, rank != 0, base, sum);
}

template <int TK, int NR>
auto one_kernel(const AdaptArgs& a) {
  return a.base == nullptr ? adapter_one_kernel<TK, kNoBase, NR>
         : a.base_kind == CK_F32 ? adapter_one_kernel<TK, CK_F32, NR> : adapter_one_kernel<TK, TK, NR>;
}
// Whether the one launch takes a call: its splits are the two launches', and its
// workgroups together read less than 20 MB of A, or 4 MB past 64 rows, whose tiles take
// longer to find.  Measured (us in a graph, and called
// back to back, where the second launch costs the host 2.8 us; one launch / two):
//   1 x 2560 x 7680, rank 16   7.0, 7.2 / 7.6, 8.9      8 x 2560 x 7680  7.4, 7.5 / 7.9, 9.4
//   8 x 4096 x 4096, rank 16   8.6, 8.7 / 8.0, 9.4     16 x 4096 x 4096  9.2, 9.2 / 7.9, 9.4 (34 MB)
//   16 x 2048 x 2048, rank 32  8.1, 8.2 / 8.0, 9.3      1 x 1024 x 1024, rank 8  4.6 / 6.9 in a graph
// and in a graph, for rows of several adapters:
//   64 of 8 x 1024 x 1024, rank 16  5.2 / 7.9          102 of 5 x 504 x 160, rank 8    6.1 / 9.2
//   40 of 4 x 2560 x 7680, rank 16  7.5 / 7.8          64 of 2 x 4096 x 4096, rank 8   9.2 / 8.4
//   256 of 64 x 1024 x 1024, rank 16  8.9 / 8.4 (11 MB)  250 of 2 x 4096 x 1024, rank 16  11.7 / 9.3 (9 MB)
bool takes_one(const AdaptArgs& a) {
  const int64_t blocks = (int64_t)a.max_tiles * ((a.n + kBlockCols - 1) / kBlockCols);
  return a.m <= kAdaptDirectRows && a.rank <= 32 && a.splits <= kOneSplits && a.split_len == (a.rank <= 16 ? 1024 : 512) &&
         blocks * a.rank * a.k <= (a.m <= 64 ? kOneReads : kOneReadsMany);
}

template <int TK>
hipError_t launch_one(const AdaptArgs& a, hipStream_t stream) {
  const auto fn = a.rank <= 16 ? one_kernel<TK, 1>(a) : one_kernel<TK, 2>(a);
  hipLaunchKernelGGL(fn, dim3((unsigned)((a.n + kBlockCols - 1) / kBlockCols), (unsigned)a.max_tiles), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <int TK, int TR, int BK>
auto up_kernel_of(int rank) {
  if (rank > 64) return adapter_up_kernel<TK, TR, BK, TR == 1 ? 0 : kLongSteps>;
  return rank <= 32 ? adapter_up_kernel<TK, TR, BK, 1> : adapter_up_kernel<TK, TR, BK, 2>;
}
template <int TK, int TR>
auto up_kernel(const AdaptArgs& a) {
  return a.base == nullptr       ? up_kernel_of<TK, TR, kNoBase>((int)a.rank)
         : a.base_kind == CK_F32 ? up_kernel_of<TK, TR, CK_F32>((int)a.rank) : up_kernel_of<TK, TR, TK>((int)a.rank);
}

// Workgroups of the up product that take 16 rows of a tile of 64 each: where whole tiles
// would be too few for the chip, and for long ranks, unless rows and columns are many and
// four steps of B can be held: totals of 64 rows would leave a CU too few waves.  Measured
// (us; whole tiles / 16 rows of each):
//   pieces of 256 columns of a tile   48: 3002 x 74 22.1 / 15.7, 172: 2594 x 859 31.3 / 25.8,
//   348: 849 x 1311 22.1 / 16.0, 576: 4096 x 2048 28.2 / 30.1, 924: 2683 x 5178 41.3 / 36.4,
//   2190: 4096 x 7680 48.0 / 55.3
//   rank 128, four steps held  704: 900 x 8192 35.2 / 36.3, 736: 900 x 4096 40.5 / 37.4,
//   1168: 4096 x 4096 62.3 / 61.2, 1504: 1000 x 8192 57.8 / 57.7, 2190: 4096 x 7680 84.6 / 99.3,
//   f16 (one block of columns, two 131) 101 / 118
//   rank 256, none held  4096 x 7680 221 / 180
constexpr int64_t kLongPieces = 1536;
constexpr int64_t kPartPieces = 512;

// A workgroup gets more than 64 KiB of LDS, the launch's part (at most 64 here) and the
// kernel's own, on request.  The request is the same in every call: threads share it.
template <typename F>
hipError_t ask_for_lds(F fn, size_t launch_bytes, size_t own_bytes) {
  if (launch_bytes + own_bytes <= 64 * 1024) return hipSuccess;
  return hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
}

template <int TK, int TR>
hipError_t launch_tiles(const AdaptArgs& a, hipStream_t stream) {
  const unsigned tiles = (unsigned)a.max_tiles;
  const int nr = a.rank > 32 ? 4 : a.rank > 16 ? 2 : 1;
  const unsigned blocks = (unsigned)((a.rank + 16 * nr - 1) / (16 * nr) * a.splits);
  const int entries = TR * nr > 2 * (TR + nr) ? TR * nr : 2 * (TR + nr);  // of 1 KiB, per wave
  const size_t lds = (size_t)kWaves * entries * 64 * sizeof(f32x4);
  const auto down = nr == 1   ? adapter_down_kernel<TK, TR, 1>
                    : nr == 2 ? adapter_down_kernel<TK, TR, 2> : adapter_down_kernel<TK, TR, 4>;
  hipError_t e = ask_for_lds(down, lds, TR > 1 ? 256 : 4352);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(down, dim3(blocks, tiles), dim3(kThreads), lds, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Columns of a workgroup: 256 times what leaves about four workgroups for each CU.
  // 4096 rows x 7680 (2190 pieces of 256 columns) once / twice / three times 49.8 / 48.6 /
  // 50.4 us, 2000 x 2560 (350 pieces) 22.2 / 25.7 / 30.5, 1 x 7680 8.1, four times 10.7.
  const int64_t all = (int64_t)tiles * ((a.n + kBlockCols - 1) / kBlockCols);
  const bool long_steps = TR > 1 && a.rank > 64 && a.rank <= 32 * kLongSteps && all >= kLongPieces;
  const int col_blocks = TR == 1 && all >= 4096 ? 4 : all < 1536 || (long_steps && TK == CK_F16) ? 1 : 2;
  const unsigned cols = (unsigned)((a.n + kBlockCols * col_blocks - 1) / (kBlockCols * col_blocks));
  const int parts = TR > 1 && (a.rank > 64 ? !long_steps : all < kPartPieces) ? TR : 1;
  const size_t planes = (size_t)kPlanes * 16 * (TR / parts) * ((long_steps ? kLongSteps : (a.rank + 31) / 32) * 32 + 8) * 2;
  const auto up = parts > 1 ? up_kernel<TK, 1>(a) : up_kernel<TK, TR>(a);
  e = ask_for_lds(up, planes, kWaves * 64 * kColTiles * sizeof(u32x4) + 16 * TR * sizeof(uint32_t));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(up, dim3(cols, tiles, (unsigned)parts), dim3(kThreads), planes, stream, a, col_blocks);
  return hipGetLastError();
}

// Up to kAdaptDirectRows rows: a place of the grid for each adapter and for each 16
// rows that one may have more, if those are fewer than the rows.
bool adapt_by_adapter(int64_t m, int64_t count) { return count + 1 + m / 16 < m; }

}  // namespace

// Splits of k over workgroups.  The up launch adds their parts again in each of its
// workgroups, so splits are longer where the rank or the rows give workgroups enough.
// For up to 16 rows they depend on k and the rank alone, as a row's bits do.  Measured
// (us): 1 row, rank 16, k 2560 in splits of 256 / 512 / 1024 8.2 / 7.6 / 7.6, 16 rows, k 5120
// 10.1 / 9.0 / 8.5; 8 rows, rank 32, k 8192 512 / 768 8.2 / 9.0; 16 rows, rank 256, k 5120
// 512 / 1024 / 2048 22.2 / 18.9 / 21.9.
int adapt_splits(int64_t m, int64_t k, int64_t rank, int64_t count, int64_t* split_len) {
  int64_t len = m <= 64 && rank > 16 && rank <= 64 ? 512 : 1024;
  if (m > kAdaptDirectRows) {
    // about one workgroup per CU, if one in eight rows begins an adapter's at the most
    const int64_t nr = rank > 32 ? 4 : rank > 16 ? 2 : 1;
    const int64_t starts = count + 1 < m / 8 ? count + 1 : m / 8;
    const int64_t groups = (m / kAdaptTileRows + starts) * ((rank + 16 * nr - 1) / (16 * nr));
    const int64_t want = (256 + groups - 1) / groups;
    len = (k + want - 1) / want;
    len = (len + 255) / 256 * 256;
  }
  while ((k + len - 1) / len > 32) len *= 2;
  *split_len = len;
  return (int)((k + len - 1) / len);
}

int64_t adapt_max_tiles(int64_t m, int64_t count) {
  if (m <= kAdaptDirectRows) return adapt_by_adapter(m, count) ? count + 1 + m / 16 : m;
  const int64_t groups = count + 1 < m ? count + 1 : m;
  return m / kAdaptTileRows + groups;
}

hipError_t launch_adapters(const AdaptArgs& a, int kind, hipStream_t stream) {
  if (a.m < 1 || a.rank < 8 || a.rank % 8 != 0 || a.rank > kAdapterRankMax || a.count < 1 || a.count > kAdaptersMax ||
      a.k % 8 != 0 || a.splits < 1 || (int64_t)a.splits * a.split_len < a.k || a.split_len % 256 != 0 ||
      a.max_tiles > 65535)
    return hipErrorInvalidValue;
  if (a.m <= kAdaptDirectRows) {
    AdaptArgs d = a;
    d.by_adapter = adapt_by_adapter(a.m, a.count);
    if (takes_one(d)) return kind == CK_F16 ? launch_one<CK_F16>(d, stream) : launch_one<CK_BF16>(d, stream);
    return kind == CK_F16 ? launch_tiles<CK_F16, 1>(d, stream) : launch_tiles<CK_BF16, 1>(d, stream);
  }
  hipLaunchKernelGGL(adapter_sort_kernel, dim3(1), dim3(kSortThreads), (size_t)(a.count + 1) * 4, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return kind == CK_F16 ? launch_tiles<CK_F16, 4>(a, stream) : launch_tiles<CK_BF16, 4>(a, stream);
}

}  // namespace skinny
