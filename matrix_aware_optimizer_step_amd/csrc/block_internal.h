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
  int64_t total_tiles;       // set by the launcher
};
hipError_t launch_block_gemm(const BlockGemmArgs& a, hipStream_t stream);

}  // namespace muon
