// Each token's weighted sum of its experts' rows, and the gradient of the
// weights:
//
//   out[t] = sum over j of w[t][j] * y[slots[t][j]]     in the order of j, fp32
//   dw[t][j] = <dout[t], y[slots[t][j]]>                 fp32
//
// Both read every row once and are bound by that: bytes in, an element of the
// result for each k of them.  16384 tokens, 8 rows of 2048 bf16: sums 106 us (5.7
// TB/s), dots 112 (5.4).

#include "block_internal.h"

namespace muon {
namespace {

constexpr int kPer = 8;            // columns of a lane
constexpr int kWide = 64 * kPer;   // columns of a wave
constexpr int kAtOnce = 4;         // rows whose loads are in flight together

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// Eight elements at column c of a row, as fp32; zeros behind the last column.
// STREAM: past the caches (nontemporal), where y is more than they hold:
// 16384 tokens of 8 rows of 2048 106 us against 120 for the sums; 1000 tokens of
// 6 rows of 5120 16 against 14.
template <bool STREAM>
__device__ __forceinline__ void load8(float* v, const char* row, int bf16, int64_t c, int64_t cols) {
  if (bf16) {
    const char* p = row + 2 * c;
    uint32_t w[4] = {0, 0, 0, 0};
    if (c + 8 <= cols) {
      const u32x4_any* g = reinterpret_cast<const u32x4_any*>(p);
      const u32x4 t = STREAM ? __builtin_nontemporal_load(g) : *g;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = t[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < cols)
          w[k / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[k]) << (16 * (k % 2));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __builtin_bit_cast(float, k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
  } else {
    const float* p = reinterpret_cast<const float*>(row) + c;
    if (c + 8 <= cols) {
      const u32x4_any* g = reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 t = STREAM ? __builtin_nontemporal_load(g + h) : g[h];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * h + k] = __builtin_bit_cast(float, static_cast<uint32_t>(t[k]));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = c + k < cols ? p[k] : 0.0f;
    }
  }
}

// The row of pair (token, j), null where it has none.
__device__ __forceinline__ const char* row_of(const ExpertSumArgs& a, int64_t pair) {
  const int s = a.slots[pair];
  return s >= 0 && s < a.rows ? a.y.base + static_cast<int64_t>(s) * a.y.ld * (a.y.dtype ? 2 : 4) : nullptr;
}

template <bool STREAM>
__global__ __launch_bounds__(256) void sum_kernel(const ExpertSumArgs a) {
  const int lane = threadIdx.x & 63;
  const uint32_t wide = (static_cast<uint32_t>(a.cols) + kWide - 1) / kWide;
  const uint32_t job = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int64_t token = job / wide;
  const int64_t c = static_cast<int64_t>(job - static_cast<uint32_t>(token) * wide) * kWide + lane * kPer;
  if (token >= a.tokens || c >= a.cols) return;
  float acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.0f;
  for (int j0 = 0; j0 < a.k; j0 += kAtOnce) {
    float v[kAtOnce][kPer], w[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      w[j] = 0.0f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[j][k] = 0.0f;
      if (j0 + j < a.k) {
        const int64_t pair = token * a.k + j0 + j;
        w[j] = a.weights ? a.weights[pair] : 1.0f;
        const char* row = row_of(a, pair);
        if (row) load8<STREAM>(v[j], row, a.y.dtype, c, a.cols);
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = __builtin_fmaf(w[j], v[j][k], acc[k]);
  }
  char* out = a.out.base + token * a.out.ld * (a.out.dtype ? 2 : 4);
  if (a.out.dtype) {
    __bf16 b[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) b[k] = static_cast<__bf16>(acc[k]);
    if (c + kPer <= a.cols) {
      __builtin_memcpy(out + 2 * c, b, sizeof(b));
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (c + k < a.cols) reinterpret_cast<__bf16*>(out)[c + k] = b[k];
    }
  } else {
    float* p = reinterpret_cast<float*>(out) + c;
    if (c + kPer <= a.cols) {
      __builtin_memcpy(p, acc, sizeof(acc));
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (c + k < a.cols) p[k] = acc[k];
    }
  }
}

// A wave for kAtOnce rows of a token: the gradient's columns stay in registers
// while the rows' go by.
template <bool STREAM>
__global__ __launch_bounds__(256) void dot_kernel(const ExpertSumArgs a) {
  const int lane = threadIdx.x & 63;
  const uint32_t parts = (a.k + kAtOnce - 1) / kAtOnce;
  const uint32_t job = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int64_t token = job / parts;
  const int j0 = static_cast<int>(job - static_cast<uint32_t>(token) * parts) * kAtOnce;
  if (token >= a.tokens) return;
  const char* grad = a.out.base + token * a.out.ld * (a.out.dtype ? 2 : 4);
  float acc[kAtOnce];
  const char* row[kAtOnce];
#pragma unroll
  for (int j = 0; j < kAtOnce; ++j) {
    acc[j] = 0.0f;
    row[j] = j0 + j < a.k ? row_of(a, token * a.k + j0 + j) : nullptr;
  }
  for (int64_t c = lane * kPer; c < a.cols; c += kWide) {
    float g[kPer], v[kAtOnce][kPer];
    load8<false>(g, grad, a.out.dtype, c, a.cols);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (row[j]) {
        load8<STREAM>(v[j], row[j], a.y.dtype, c, a.cols);
      } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[j][k] = 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[j] = __builtin_fmaf(g[k], v[j][k], acc[j]);
  }
#pragma unroll
  for (int j = 0; j < kAtOnce; ++j) {
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) acc[j] += __shfl_xor(acc[j], d);
    if (lane == 0 && j0 + j < a.k) a.dots[token * a.k + j0 + j] = row[j] ? acc[j] : 0.0f;
  }
}

bool streams(const ExpertSumArgs& a) {
  return static_cast<int64_t>(a.rows) * a.cols * (a.y.dtype ? 2 : 4) >= int64_t{1} << 27;
}

}  // namespace

hipError_t launch_expert_sum(const ExpertSumArgs& a, hipStream_t s) {
  const int64_t jobs = a.tokens * ((a.cols + kWide - 1) / kWide);
  const uint32_t g = static_cast<uint32_t>((jobs + 3) / 4);
  if (streams(a)) {
    sum_kernel<true><<<g, 256, 0, s>>>(a);
  } else {
    sum_kernel<false><<<g, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_expert_dot(const ExpertSumArgs& a, hipStream_t s) {
  const int64_t jobs = a.tokens * ((a.k + kAtOnce - 1) / kAtOnce);
  const uint32_t g = static_cast<uint32_t>((jobs + 3) / 4);
  if (streams(a)) {
    dot_kernel<true><<<g, 256, 0, s>>>(a);
  } else {
    dot_kernel<false><<<g, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace muon
