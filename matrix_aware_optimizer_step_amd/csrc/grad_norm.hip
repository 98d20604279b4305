// Global 2-norm of a list of gradients, the clip factor and the step count
// of a muon_step_control block.
//
//   norm = sqrt(sum g^2),  scale = min(1, max_norm / norm)
//
// Two launches.  norm_partials_kernel: at most kGradMaxBlocks workgroups walk
// the list's chunks, workgroup b taking the chunks b, b + grid, ..., and each
// writes one fp64 sum.  norm_finish_kernel adds those sums in a fixed order
// and writes the block.  Squares are formed and added in fp64 (v_fma_f64 has
// fp32's rate here), so the largest finite gradients do not overflow and no
// length loses bits.

#include "muon_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = kGradChunk / kThreads;  // 64

__device__ __forceinline__ double sq(float f, double acc) {
  const double d = static_cast<double>(f);
  return fma(d, d, acc);
}

// Sum of squares of this thread's share of one chunk of `len` elements.
template <bool BF16>
__device__ __forceinline__ double chunk_sumsq(const char* p, int64_t len, double acc) {
  constexpr int V = BF16 ? 8 : 4;  // elements in 16 bytes
  constexpr int ES = BF16 ? 2 : 4;
  if (len == kGradChunk && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    uint4 u[kPerThread / V];
#pragma unroll
    for (int k = 0; k < kPerThread / V; ++k)
      u[k] = *reinterpret_cast<const uint4*>(p + (k * kThreads + threadIdx.x) * 16);
#pragma unroll
    for (int k = 0; k < kPerThread / V; ++k) {
      const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (BF16) {
          acc = sq(__builtin_bit_cast(float, w[j] << 16), acc);
          acc = sq(__builtin_bit_cast(float, w[j] & 0xffff0000u), acc);
        } else {
          acc = sq(__builtin_bit_cast(float, w[j]), acc);
        }
      }
    }
    return acc;
  }
  for (int64_t e = threadIdx.x; e < len; e += kThreads) {
    const float f = BF16 ? __builtin_bit_cast(float, static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p + e * ES)) << 16)
                         : *reinterpret_cast<const float*>(p + e * ES);
    acc = sq(f, acc);
  }
  return acc;
}

// Workgroup sum in a fixed order; the result is valid in thread 0.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) s += red[i];
  }
  return s;
}

__global__ __launch_bounds__(kThreads) void norm_partials_kernel(const GradNormArgs a) {
  __shared__ double red[kThreads / 64];
  double acc = 0.0;
  for (int64_t c = blockIdx.x; c < a.total_chunks; c += a.blocks) {
    const int64_t t = a.chunk_tensor[c];
    if (t < 0 || t >= a.count) continue;
    const GradTensor g = a.grads[t];
    const int64_t start = (c - g.first_chunk) * kGradChunk;
    if (start < 0 || start >= g.numel) continue;
    const int64_t len = g.numel - start < kGradChunk ? g.numel - start : kGradChunk;
    acc = g.dtype ? chunk_sumsq<true>(g.data + start * 2, len, acc) : chunk_sumsq<false>(g.data + start * 4, len, acc);
  }
  const double s = block_sum(acc, red);
  if (threadIdx.x == 0) a.partials[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void norm_finish_kernel(const GradNormArgs a) {
  __shared__ double red[kThreads / 64];
  double acc = 0.0;
  for (int i = threadIdx.x; i < a.blocks; i += kThreads) acc += a.partials[i];
  const double s = block_sum(acc, red);
  if (threadIdx.x != 0) return;
  StepControl* c = a.control;
  const float norm = static_cast<float>(sqrt(s));
  c->norm = norm;
  // an infinite norm against an infinite bound is not over it; a NaN is neither
  c->scale = norm > a.max_norm ? a.max_norm / norm : norm <= a.max_norm ? 1.0f : norm;
  const bool skip = a.skip_nonfinite && !(norm <= 3.402823466e38f);
  c->skip = skip;
  if (skip) {
    c->skipped += 1;
  } else {
    c->step += 1;
  }
}

}  // namespace

hipError_t launch_grad_norm(const GradNormArgs& a, hipStream_t stream) {
  if (a.blocks > 0) {
    hipLaunchKernelGGL(norm_partials_kernel, dim3(a.blocks), dim3(kThreads), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_finish_kernel, dim3(1), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace muon
