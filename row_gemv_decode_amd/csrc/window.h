// window.h -- host-side interfaces between the C ABI of the decode window's
// operators (abi_window.cpp) and their kernels (w4.hip, moe.hip,
// logprobs.hip).  Not installed.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "internal.h"

namespace skinny {

// ---------------------------------------------------------------------------
// 4-bit grouped weights (w4.hip, moe.hip): codes [n][k/2] (element kk in byte
// kk/2, the low nibble for even kk), scales [n][k/group] in the rows' type,
// zero points uint8 [n][k/group] or null (8): W = s * (q - z)
// ---------------------------------------------------------------------------
// A launch's grid counts its threads in 32 bits, and a larger one is cut off
// without an error: larger work goes in several launches, or is refused.
constexpr int64_t kMaxLaunchThreads = 1LL << 31;

struct WindowWeight {     // 16-bit weights in `codes`, or a 4-bit grouped weight
  const void* codes;
  const void* scales;
  const void* zeros;
};

// largest k: a lane's offset into its tile of 16 columns has 32 bits
constexpr int64_t kW4MaxK = 1 << 24;

struct W4Args {
  const void* A;       // [m][lda] f16/bf16
  int64_t lda;
  WindowWeight w;
  int64_t n;
  int64_t k;
  void* C;             // [m][ldc]
  int64_t ldc;
  int32_t m;           // <= kGemvMaxM
  int32_t c_kind;      // CK_*
};

// a_kind: CK_F16 or CK_BF16; group 32, 64 or 128
hipError_t launch_w4_mm(const W4Args& args, int a_kind, int group, hipStream_t stream);

// ---------------------------------------------------------------------------
// The whole MoE layer for a decode window (moe.hip): route, up, down, combine
// launches after the router's GEMV.
// ---------------------------------------------------------------------------
constexpr int kMoeMaxExperts = 1024;

struct MoeArgs {
  const void* x;           // [m][ldx]
  int64_t ldx;
  int64_t d;               // row length
  int64_t inter;           // an expert's inner length
  int64_t shared_inter;    // the shared expert's, 0: none
  WindowWeight w13, w2;       // [E][2 inter][d], [E][d][inter]
  WindowWeight s13, s2;       // the shared expert's
  const void* shared_gate; // [d]
  const float* logits;     // [m][experts]
  uint32_t* slots;         // distinct experts, ascending: expert | token mask << 16
  int32_t* slot_rank;      // [max_slots][16]: each slot's place among the experts of a token it serves
  uint32_t* parts;         // [max_parts][4]: expert | tokens << 16, their rows of h (16 bits each)
  float* weights;          // [m][topk + 1]: routing weights, the shared expert's gate last
  uint16_t* h;             // [m][topk][planes][inter], then [m][planes][shared_inter]
  float* y;                // the experts' outputs, [m][topk][d], then the shared expert's, [m][d]
  int32_t* topk_idx;       // [m][topk] or null
  float* topk_weight;      // [m][topk] or null
  void* out;               // [m][ldo]
  int64_t ldo;
  int32_t m, experts, topk, renorm, max_slots, out_kind;
  int32_t max_parts;       // (set by the launch)
};

int moe_planes();  // 16-bit planes that hold one inner value
// whether the layer's launches fit a grid (for args.m, topk, experts, d, inter, shared_inter)
bool moe_fits(const MoeArgs& args, int group);

// kind: CK_F16 or CK_BF16; group: 0 (16-bit weights), 32, 64 or 128
hipError_t launch_moe(const MoeArgs& args, int kind, int group, hipStream_t stream);

// ---------------------------------------------------------------------------
// Token log probabilities (logprobs.hip)
// ---------------------------------------------------------------------------
constexpr int kLogprobMaxSegments = 16;

struct LogprobArgs {
  const void* logits;   // [m][ld]
  int64_t ld;
  int64_t vocab;        // <= 2^30
  int64_t m;
  const void* tokens;   // [m] int32 or (tokens64) int64
  int32_t tokens64;
  int32_t topk;
  int32_t segments;     // workgroups per row, seg_len logits each (the last fewer)
  int32_t seg_len;
  int32_t waves;        // per workgroup: 4 or 8
  float* logprob;       // [m]
  float* entropy;       // [m]
  int32_t* rank;        // [m]
  int32_t* top_ids;     // [m][topk]
  float* top_logprobs;  // [m][topk]
  float* partial;       // segments > 1: [m][segments][4 + 2 topk]
  uint32_t* counters;   // segments > 1: [m] arrivals, zero between calls
};

hipError_t launch_logprobs(const LogprobArgs& args, int x_kind, hipStream_t stream);

}  // namespace skinny
