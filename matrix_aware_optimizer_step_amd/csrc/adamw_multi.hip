// AdamW over many tensors of any types in one launch, with 32-bit or 8-bit
// moments ("LLM Optimizers: From SGD and AdamW to SOAP, Muon, and Scalable
// Training", sections 5 and 6):
//
//   m <- b1*m + (1-b1)*g,  v <- b2*v + (1-b2)*g^2
//   theta <- (1 - l*wd)*theta - l * (m*c1) / (sqrt(v*c2) + eps)
//
// A workgroup owns one chunk of kParamChunk elements of one tensor; the
// chunk table names the tensor.  The 8-bit state keeps m and r = sqrt(v) as
// e4m3 codes with a scale per 256 elements (include/muon355.h gives the
// format): a thread holds 16 consecutive elements, so a block is 16 lanes of
// one wave and its maximum four lane exchanges.

#include "muon_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = kParamChunk / kThreads;  // 16 elements per thread
static_assert(kStateBlock == 16 * kPer, "a block of the 8-bit state is 16 lanes");

constexpr float kTop = 448.0f;                      // largest e4m3 value
constexpr float kLeast = 0.001953125f;              // 2^-9, smallest e4m3 value above zero
constexpr float kTiny = 7.888609052210118e-31f;     // 2^-100

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
// two values rounded to nearest even, the first in the low half
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, bf16x2));
}

// 8 values starting at element e of p, all of them inside (vec) or the first n.
template <bool BF16>
__device__ __forceinline__ void load8(const char* p, bool vec, int n, float* x) {
  if (vec) {
    if (BF16) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[2 * k] = bf16_lo(w[k]);
        x[2 * k + 1] = bf16_hi(w[k]);
      }
    } else {
      const float4 a = reinterpret_cast<const float4*>(p)[0];
      const float4 b = reinterpret_cast<const float4*>(p)[1];
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = 0.0f;
      if (k < n)
        x[k] = BF16 ? bf16_lo(reinterpret_cast<const uint16_t*>(p)[k]) : reinterpret_cast<const float*>(p)[k];
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(char* p, bool vec, int n, const float* x) {
  if (vec) {
    if (BF16) {
      uint4 u;
      u.x = bf16_pair(x[0], x[1]);
      u.y = bf16_pair(x[2], x[3]);
      u.z = bf16_pair(x[4], x[5]);
      u.w = bf16_pair(x[6], x[7]);
      *reinterpret_cast<uint4*>(p) = u;
    } else {
      reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k < n) {
        if (BF16) {
          reinterpret_cast<uint16_t*>(p)[k] = static_cast<uint16_t>(bf16_pair(x[k], 0.0f));
        } else {
          reinterpret_cast<float*>(p)[k] = x[k];
        }
      }
    }
  }
}

// What one step does to one element, after g has been scaled.
struct Rule {
  float gs, b1, omb1, b2, omb2, sc2, eps, decay, lr;  // sc2 = sqrt(c2); lr includes c1

  // m and v in, m, v and r = sqrt(v) out, theta updated
  __device__ __forceinline__ void operator()(float& p, float g, float& m, float& v, float& r) const {
    g *= gs;
    m = b1 * m + omb1 * g;
    v = b2 * v + omb2 * g * g;
    r = sqrtf(v);
    p = decay * p - lr * m / (r * sc2 + eps);
  }
};

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0xBB67AE85u;
  x ^= x >> 15;
  x *= 0x9E3779B9u;
  return x ^ (x >> 16);
}

// The larger of two magnitudes; a NaN on either side gives NaN.
__device__ __forceinline__ float max_abs(float a, float b) {
  return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b));
}

template <bool PB, bool GB>
__device__ __forceinline__ void chunk32(const ParamTensor& t, const Rule& rule, int64_t start, int len, bool aligned) {
  char* P = t.param + start * (PB ? 2 : 4);
  const char* G = t.grad + start * (GB ? 2 : 4);
  char* M = t.m + start * 4;
  char* V = t.v + start * 4;
#pragma unroll
  for (int u = 0; u < kPer / 8; ++u) {
    const int e = (u * kThreads + threadIdx.x) * 8;
    const int n = len - e;
    if (n <= 0) continue;
    const bool full = n >= 8, vec = full && aligned;
    float p[8], g[8], m[8], v[8];
    load8<PB>(P + e * (PB ? 2 : 4), vec, n, p);
    load8<GB>(G + e * (GB ? 2 : 4), vec, n, g);
    load8<false>(M + e * 4, full, n, m);
    load8<false>(V + e * 4, full, n, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float r;
      rule(p[k], g[k], m[k], v[k], r);
    }
    store8<PB>(P + e * (PB ? 2 : 4), vec, n, p);
    store8<false>(M + e * 4, full, n, m);
    store8<false>(V + e * 4, full, n, v);
  }
}

// 16 codes of one lane (four words), the first n inside the tensor.
__device__ __forceinline__ void load_codes(const char* p, int n, uint32_t* w) {
  if (n >= 16) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (k < n) w[k / 4] |= static_cast<uint32_t>(reinterpret_cast<const uint8_t*>(p)[k]) << (8 * (k & 3));
  }
}

__device__ __forceinline__ void store_codes(char* p, int n, const uint32_t* w) {
  if (n >= 16) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (k < n) reinterpret_cast<uint8_t*>(p)[k] = static_cast<uint8_t>(w[k / 4] >> (8 * (k & 3)));
  }
}

__device__ __forceinline__ void decode4(uint32_t w, float s, float* x) {
  x[0] = s * __builtin_amdgcn_cvt_f32_fp8(w, 0);
  x[1] = s * __builtin_amdgcn_cvt_f32_fp8(w, 1);
  x[2] = s * __builtin_amdgcn_cvt_f32_fp8(w, 2);
  x[3] = s * __builtin_amdgcn_cvt_f32_fp8(w, 3);
}

// v_cvt_sr_fp8_f32 is floor(|y|/q + (seed >> 12) / 2^20) * q with y's sign,
// for normal and subnormal codes (checked on the hardware over the range).
__device__ __forceinline__ uint32_t encode4(const float* y, const uint32_t* rnd) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], rnd[0], w, 0);
  w = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], rnd[1], w, 1);
  w = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], rnd[2], w, 2);
  return __builtin_amdgcn_cvt_sr_fp8_f32(y[3], rnd[3], w, 3);
}

template <bool PB, bool GB>
__device__ __forceinline__ void chunk8(const ParamTensor& t, const Rule& rule, int64_t start, int len, bool aligned,
                                       uint32_t key) {
  const int e = threadIdx.x * kPer;
  const int n = len - e;  // <= 0: a lane of the last block past the tensor's end, or a block past it
  const bool vec = n >= kPer && aligned;
  char* P = t.param + (start + e) * (PB ? 2 : 4);
  const char* G = t.grad + (start + e) * (GB ? 2 : 4);
  char* CM = t.m + start + e;
  char* CR = t.v + start + e;
  float2* S = reinterpret_cast<float2*>(t.scales) + (start + e) / kStateBlock;
  float p[16], m[16], r[16];
  float am = 0.0f, ar = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) p[k] = m[k] = r[k] = 0.0f;
  if (n > 0) {
    float g[16];
    uint32_t wm[4], wr[4];
    const float2 s = *S;
    load8<PB>(P, vec, n, p);
    load8<PB>(P + 8 * (PB ? 2 : 4), vec, n - 8, p + 8);
    load8<GB>(G, vec, n, g);
    load8<GB>(G + 8 * (GB ? 2 : 4), vec, n - 8, g + 8);
    load_codes(CM, n, wm);
    load_codes(CR, n, wr);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      decode4(wm[k], s.x, m + 4 * k);
      decode4(wr[k], s.y, r + 4 * k);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float v = r[k] * r[k];
      rule(p[k], g[k], m[k], v, r[k]);
    }
    if (n < kPer) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (k >= n) m[k] = r[k] = 0.0f;  // an element past the end has no part in the block's maximum
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      am = max_abs(am, m[k]);
      ar = max_abs(ar, r[k]);
    }
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    am = max_abs(am, __shfl_xor(am, o, 16));
    ar = max_abs(ar, __shfl_xor(ar, o, 16));
  }
  if (n <= 0) return;
  const float im = am < kTiny ? 0.0f : kTop / am;
  const float ir = ar < kTiny ? 0.0f : kTop / ar;
  const uint32_t ra = mix(static_cast<uint32_t>((t.counter + start + e) >> 4) ^ key);
  const uint32_t rb = mix(ra + 0x6A09E667u);
  uint32_t wm[4], wr[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float ym[4], yr[4];
    uint32_t rm[4], rr[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t x = ra + (4 * q + k) * rb;
      rm[k] = x;
      rr[k] = (x << 16) | (x >> 16);
      // the scaled maximum may round past 448; a NaN stays in the scale
      ym[k] = fminf(fmaxf(m[4 * q + k] * im, -kTop), kTop);
      const float y = r[4 * q + k] * ir;
      yr[k] = y == 0.0f ? 0.0f : fminf(fmaxf(y, kLeast), kTop);
    }
    wm[q] = encode4(ym, rm);
    wr[q] = encode4(yr, rr);
  }
  store8<PB>(P, vec, n, p);
  store8<PB>(P + 8 * (PB ? 2 : 4), vec, n - 8, p + 8);
  store_codes(CM, n, wm);
  store_codes(CR, n, wr);
  if ((threadIdx.x & 15) == 0)
    *S = make_float2(am < kTiny ? 0.0f : am / kTop, ar < kTiny ? 0.0f : ar / kTop);
}

__global__ __launch_bounds__(kThreads) void adamw_multi_kernel(const AdamWMultiArgs a) {
  const int64_t chunk = blockIdx.x;
  const int64_t i = a.chunk_tensor[chunk];
  if (i < 0 || i >= a.count) return;  // a wrong chunk table: nothing to do here
  const ParamTensor t = a.params[i];
  const int64_t start = (chunk - t.first_chunk) * kParamChunk;
  if (start < 0 || start >= t.numel) return;
  const int len = t.numel - start < kParamChunk ? static_cast<int>(t.numel - start) : static_cast<int>(kParamChunk);

  double lr = a.lr * static_cast<double>(t.lr_factor);
  int64_t step = a.step;
  float c1 = a.c1, c2 = a.c2;
  Rule rule{1.0f, a.b1, a.omb1, a.b2, a.omb2, 0.0f, a.eps, 0.0f, 0.0f};
  if (a.control != nullptr) {
    if (a.control->skip) return;
    step = a.control->step < 1 ? 1 : a.control->step;
    rule.gs = a.control->scale;
    lr *= static_cast<double>(a.control->lr_factor);
    // 1 - beta^t = -(e^(t log beta) - 1): expm1 keeps its bits for small t
    c1 = -1.0f / expm1f(static_cast<float>(static_cast<double>(step) * a.log_b1));
    c2 = -1.0f / expm1f(static_cast<float>(static_cast<double>(step) * a.log_b2));
  }
  rule.sc2 = sqrtf(c2);
  rule.decay = static_cast<float>(1.0 - lr * static_cast<double>(t.weight_decay));
  rule.lr = static_cast<float>(lr) * c1;

  const bool aligned = ((reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad)) & 15) == 0;
  if (t.state_bits == 8) {
    const uint32_t key = mix(mix(static_cast<uint32_t>(step)) ^ a.seed);
    if (t.param_dtype) {
      t.grad_dtype ? chunk8<true, true>(t, rule, start, len, aligned, key)
                   : chunk8<true, false>(t, rule, start, len, aligned, key);
    } else {
      t.grad_dtype ? chunk8<false, true>(t, rule, start, len, aligned, key)
                   : chunk8<false, false>(t, rule, start, len, aligned, key);
    }
  } else {
    if (t.param_dtype) {
      t.grad_dtype ? chunk32<true, true>(t, rule, start, len, aligned)
                   : chunk32<true, false>(t, rule, start, len, aligned);
    } else {
      t.grad_dtype ? chunk32<false, true>(t, rule, start, len, aligned)
                   : chunk32<false, false>(t, rule, start, len, aligned);
    }
  }
}

}  // namespace

hipError_t launch_adamw_multi(const AdamWMultiArgs& a, int64_t total_chunks, hipStream_t stream) {
  if (total_chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(adamw_multi_kernel, dim3(static_cast<unsigned>(total_chunks)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace muon
