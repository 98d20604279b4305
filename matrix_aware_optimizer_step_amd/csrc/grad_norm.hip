// Global 2-norm of a list of gradients, the clip factor and the step count
// of a muon_step_control block.
//
//   norm = sqrt(sum g^2),  scale = min(1, max_norm / norm)
//
// At most kGradMaxBlocks workgroups walk the list's chunks, workgroup b taking
// the chunks b, b + grid, ..., and each leaves one fp64 sum; the sums are then
// added in a fixed order.  Up to kGradOneLaunch workgroups the one that draws
// the last ticket does that; with more of them a second launch does it, since
// the tickets are drawn one after another.  One launch against two, us a call
// among others, bf16: 16 workgroups 5.2 and 7.1, 65 5.9 and 7.1, 128 6.7 and
// 7.1, 160 7.1 and 7.2, 200 7.7 and 7.3, 256 8.5 and 7.1, 384 10.6 and 7.6,
// 512 12.7 and 8.7.  The two meet at 160, so between that and 256 a second
// launch would be the faster, by 1.4 us at most.
//
// Bound by HBM: 1.05e9 bf16 gradients in 316 us, 6.6 TB/s.  Two workgroups
// per compute unit with eight 16-byte loads in flight per thread; 4, 8 or 1
// per unit took 340, 353 and 420 us.  Squares are formed and added in fp64
// (v_fma_f64 has fp32's rate here), so no sum of finite gradients overflows
// and no length loses bits; the norm itself is a float and can be infinite.

#include "muon_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kBytes = 16;  // per access

__device__ __forceinline__ double sq(float f, double acc) {
  const double d = static_cast<double>(f);
  return fma(d, d, acc);
}

template <bool BF16>
__device__ __forceinline__ double sq_word(uint32_t w, double acc) {
  if (BF16) return sq(__builtin_bit_cast(float, w & 0xffff0000u), sq(__builtin_bit_cast(float, w << 16), acc));
  return sq(__builtin_bit_cast(float, w), acc);
}

// Sum of squares of this thread's share of one chunk of `len` elements: 16
// bytes at a time wherever the tensor starts (the hardware takes vector
// accesses at any address), kGroup of them in flight, and the elements past
// the last whole 16 bytes one by one.
template <bool BF16>
__device__ __forceinline__ double chunk_sumsq(const char* p, int len, double acc) {
  constexpr int ES = BF16 ? 2 : 4, V = kBytes / ES, kGroup = 8;
  const int whole = len / V;
  int k = threadIdx.x;
  for (; k + (kGroup - 1) * kThreads < whole; k += kGroup * kThreads) {
    uint32_t w[kGroup][4];
#pragma unroll
    for (int j = 0; j < kGroup; ++j) __builtin_memcpy(w[j], p + (k + j * kThreads) * kBytes, kBytes);
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = sq_word<BF16>(w[j][i], acc);
  }
  if (k < whole) {
    uint32_t w[kGroup][4];
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      const int at = k + j * kThreads;
      if (at < whole) {
        __builtin_memcpy(w[j], p + at * kBytes, kBytes);
      } else {
        w[j][0] = w[j][1] = w[j][2] = w[j][3] = 0;
      }
    }
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = sq_word<BF16>(w[j][i], acc);
  }
  const int rest = whole * V + threadIdx.x;
  if (rest < len)
    acc = sq(BF16 ? __builtin_bit_cast(float, static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[rest]) << 16)
                  : reinterpret_cast<const float*>(p)[rest],
             acc);
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

__device__ __forceinline__ void finish(const GradNormArgs& a, double sum) {
  StepControl* c = a.control;
  const float norm = static_cast<float>(sqrt(sum));
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

template <bool ONE>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const GradNormArgs a) {
  __shared__ double red[kThreads / 64];
  double acc = 0.0;
  for (int64_t c = blockIdx.x; c < a.total_chunks; c += a.blocks) {
    const int64_t t = a.chunk_tensor[c];
    if (t < 0 || t >= a.count) continue;
    const GradTensor g = a.grads[t];
    const int64_t start = (c - g.first_chunk) * kGradChunk;
    // (a condition of its own would take 336 us where this takes 316, for 1.05e9 bf16 elements)
    const int64_t numel = known_type(g.dtype) ? g.numel : 0;
    if (start < 0 || start >= numel) continue;
    const int len = static_cast<int>(numel - start < kGradChunk ? numel - start : kGradChunk);
    acc = g.dtype ? chunk_sumsq<true>(g.data + start * 2, len, acc) : chunk_sumsq<false>(g.data + start * 4, len, acc);
  }
  const double s = block_sum(acc, red);
  if (!ONE) {
    if (threadIdx.x == 0) a.partials[blockIdx.x] = s;
    return;
  }
  __shared__ uint32_t last;
  uint32_t* ticket = reinterpret_cast<uint32_t*>(&a.control->reserved[0]);
  if (threadIdx.x == 0) {
    // The exchange takes the sum to memory that every XCD sees, and the
    // ticket is drawn only when its answer is back (the ticket's operand
    // hangs on it): no cache has to be written back for that.
    const auto old = __hip_atomic_exchange(reinterpret_cast<unsigned long long*>(a.partials + blockIdx.x),
                                           __builtin_bit_cast(unsigned long long, s), __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
    uint32_t one = 1;
    asm volatile("" : "+v"(one) : "v"(old) : "memory");
    last = __hip_atomic_fetch_add(ticket, one, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  acc = 0.0;
  for (int i = threadIdx.x; i < a.blocks; i += kThreads)
    acc += __hip_atomic_load(a.partials + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const double sum = block_sum(acc, red);
  if (threadIdx.x == 0) {
    __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next call
    finish(a, sum);
  }
}

__global__ __launch_bounds__(kThreads) void norm_finish_kernel(const GradNormArgs a) {
  __shared__ double red[kThreads / 64];
  double acc = 0.0;
  for (int i = threadIdx.x; i < a.blocks; i += kThreads) acc += a.partials[i];
  const double sum = block_sum(acc, red);
  if (threadIdx.x == 0) finish(a, sum);
}

}  // namespace

hipError_t launch_grad_norm(const GradNormArgs& a, hipStream_t stream) {
  if (a.blocks <= kGradOneLaunch) {
    // an empty list still writes the block: one workgroup, whose sum is 0
    hipLaunchKernelGGL(grad_norm_kernel<true>, dim3(a.blocks > 0 ? a.blocks : 1), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(grad_norm_kernel<false>, dim3(a.blocks), dim3(kThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_finish_kernel, dim3(1), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace muon
