// Internal declarations of the 8-bit block codes, their products, the routing
// to experts and the experts' sums, shared by their kernels and the C-ABI
// layer.  Nothing here is part of the public interface (include/muon355.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "muon_internal.h"

namespace muon {

constexpr int kCodeBlock = 128;    // MUON_CODE_BLOCK: columns (and rows of a square block) that share a scale
constexpr int kMaxExperts = 512;   // MUON_MAX_EXPERTS
constexpr int kMaxChosen = 16;     // MUON_MAX_CHOSEN
constexpr int kMaxExpertGroups = 32;  // MUON_MAX_EXPERT_GROUPS

// A matrix of e4m3 codes with its scales, as a kernel sees it (muon_codes_t).
struct CodeMat {
  char* codes;
  float* scales;
  int64_t stride, scale_stride;  // bytes, floats between matrices
  int64_t ld, scale_ld;
};

struct QuantizeArgs {
  MatBatch x;
  const int32_t* pairs;   // null, or the pair of each output row (source row = pair / k; < 0: a row of zeros)
  const float* weights;   // null, or a factor for each pair
  int32_t k;
  int32_t in_rows;        // rows of x (bounds pair / k)
  int32_t rows, cols;     // of the codes in x's own order
  int32_t square;         // blocks of 128x128
  CodeMat q, qt;          // codes null: not written
};
hipError_t launch_quantize(const QuantizeArgs& a, int64_t count, hipStream_t stream);

enum GemmMode : int32_t { GEMM_BATCH = 0, GEMM_ROWS = 1, GEMM_REDUCE = 2 };

// C = A B^T over codes; rows(A) = M, rows(B) = N, K columns each.
struct BlockGemmArgs {
  CodeMat a, b;
  MatBatch c;
  const int32_t* offsets;  // device, count + 1 of them, or null
  int64_t count;
  int32_t M, N, K;
  int32_t mode;            // GemmMode
  int32_t square;          // b's blocks are 128x128
  int32_t accumulate;
  int32_t tiles_m, tiles_n;  // set by the launcher
};
hipError_t launch_block_gemm(const BlockGemmArgs& a, hipStream_t stream);

// ------------------------------------------------------------ routing

struct RouteArgs {
  const char* logits;
  int64_t ld;               // elements between tokens
  const float* bias;        // [experts] or null
  const uint8_t* mask;      // [tokens] or null: 0 = the token goes nowhere
  int32_t* chosen;          // [tokens, k]
  float* weights;           // [tokens, k]
  int32_t* slots;           // [tokens, k]; slots, pairs and offsets may all be null
  int32_t* pairs;           // [capacity]
  int32_t* offsets;         // [experts + 1]
  int32_t* loads;           // [experts] or null
  uint8_t* counts;          // [runs of `group` tokens][experts rounded up to 16]
  int64_t capacity;
  int32_t tokens, experts, k;
  int32_t dtype;            // of the logits: 0 = f32, 1 = bf16
  int32_t sigmoid, renormalize;
  int32_t groups, top_groups, group_best;
  int32_t align;
  int32_t group;            // set by the launcher: 16 or 64
  float scale;
};
// Tokens of a run, whose counts are one row of the workspace.
constexpr int64_t kMostInRunsOf16 = 16384;
constexpr int32_t route_group(int64_t tokens, int64_t) { return tokens <= 64 || tokens > kMostInRunsOf16 ? 64 : 16; }
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);

struct RouteBackwardArgs {
  const char* logits;
  int64_t ld;
  const int32_t* chosen;
  const float* weights;
  const float* grad;        // [tokens, k]
  char* out;                // [tokens, experts], as the logits
  int64_t ld_out;
  int32_t tokens, experts, k;
  int32_t dtype;
  int32_t sigmoid, renormalize;
  float scale;
};
hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t stream);

struct BalanceArgs {
  float* bias;
  int32_t* loads;
  int32_t experts;
  float rate;
  const StepControl* control;  // or null
};
hipError_t launch_balance(const BalanceArgs& a, hipStream_t stream);

// ------------------------------------------------------------ sums over a token's experts

struct ExpertSumArgs {
  MatBatch y;               // [rows, cols]
  MatBatch out;             // [tokens, cols]; the gradient of the sums in the dot
  const int32_t* slots;     // [tokens, k]
  const float* weights;     // [tokens, k] or null (ones); the dot writes it
  float* dots;
  int64_t tokens;
  int32_t rows, cols, k;
};
hipError_t launch_expert_sum(const ExpertSumArgs& a, hipStream_t stream);
hipError_t launch_expert_dot(const ExpertSumArgs& a, hipStream_t stream);

}  // namespace muon
