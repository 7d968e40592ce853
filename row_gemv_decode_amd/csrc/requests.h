// requests.h -- host-side interfaces between the C ABI of the operators of a
// batch of requests (abi_requests.cpp) and their kernels (norm.hip,
// adapters.hip, adjust.hip).  Not installed.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "window.h"

namespace skinny {

// ---------------------------------------------------------------------------
// The residual's addition and the root-mean-square norm (norm.hip)
// ---------------------------------------------------------------------------
struct NormArgs {
  const void* x;         // [m][ldx]
  int64_t ldx;
  const void* residual;  // [m][ldr] or null
  int64_t ldr;
  const void* weight;    // [d] or null
  void* residual_out;    // [m][ldro] or null
  int64_t ldro;
  void* out;             // [m][ldo] or null
  int64_t ldo;
  uint8_t* q;            // [m][ldq] or null
  int64_t ldq;
  float* scales;         // [m][groups]
  int64_t m;
  int32_t d;
  int32_t group;         // columns per scale, 0: the row
  int32_t groups;        // scales per row
  int32_t w_kind, out_kind;
  float eps;
  int32_t lanes_log2;    // (set by the launch) rows within a wave: lanes per row
};

// r_kind: any without a residual
hipError_t launch_norm(const NormArgs& args, int x_kind, int r_kind, hipStream_t stream);

// ---------------------------------------------------------------------------
// Low-rank adapters (adapters.hip)
// ---------------------------------------------------------------------------
constexpr int kAdaptersMax = 8192;
constexpr int kAdapterRankMax = 256;

struct AdaptArgs {
  const void* x;         // [m][ldx]
  int64_t ldx;
  const void* A;         // [count][rank][k]
  const void* B;         // [count][n][rank]
  const int32_t* ranks;  // [count] or null
  const float* scaling;  // [count] or null
  const void* ids;       // [m] int32 or (ids64) int64
  const void* base;      // [m][ldb] or null
  int64_t ldb;
  void* out;             // [m][ldo]
  int64_t ldo;
  int32_t m, n, k, rank, count;
  int32_t ids64;
  int32_t base_kind, out_kind;
  int32_t splits;        // of k over workgroups
  int32_t split_len;     // elements of a split, a multiple of 256
  float* h;              // [splits][m][rank] partial inner values
  uint32_t* tile_count;  // batches past kAdaptDirectRows: how many tiles there are
  uint32_t* tiles;       // [max_tiles][4]: adapter, rows (0: no tile), rank, scaling
  uint32_t* order;       // the tiles' rows, room for adapt_tile_rows each
  int32_t max_tiles;
  int32_t by_adapter;    // (set by the launch) up to kAdaptDirectRows: tiles in the order of the adapters
};

// rows up to which every workgroup finds its adapter's rows by itself
constexpr int kAdaptDirectRows = 256;
constexpr int kAdaptTileRows = 64;  // rows of a tile in larger batches
int adapt_splits(int64_t m, int64_t k, int64_t rank, int64_t count, int64_t* split_len);
constexpr int64_t adapt_tile_rows(int64_t m) { return m <= kAdaptDirectRows ? 16 : kAdaptTileRows; }
int64_t adapt_max_tiles(int64_t m, int64_t count);

hipError_t launch_adapters(const AdaptArgs& args, int kind, hipStream_t stream);

// ---------------------------------------------------------------------------
// Penalties, biases and masks on logits (adjust.hip)
// ---------------------------------------------------------------------------
struct AdjustArgs {
  const void* logits;  // [m][ld]
  int64_t ld;
  void* out;           // [m][ldo], or the logits
  int64_t ldo;
  int64_t m;
  int32_t vocab;
  const void* history;  // [m][ldh] or null
  int64_t ldh;
  int32_t history_len;
  int32_t biases;
  int32_t tokens64;
  int32_t masks;
  const int32_t* lengths;
  const int32_t* prompt_lengths;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const void* bias_ids;  // [m][biases] or null
  const float* bias_values;
  const int32_t* mask;   // [masks][ldm] or null
  int64_t ldm;
  const int32_t* mask_rows;
  int32_t segments;      // (set by the launch) workgroups per row, seg_len tokens each
  int32_t seg_len;
};

hipError_t launch_adjust(const AdjustArgs& args, int x_kind, int out_kind, hipStream_t stream);

}  // namespace skinny
