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
// format).

#include "muon_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = kParamChunk / kThreads;  // 16 elements per thread
constexpr int kPiece = 8;                     // contiguous elements of a thread
static_assert(kStateBlock == 16 * kPer, "a block of the 8-bit state is 16 lanes");

constexpr float kTop = 448.0f;                      // largest e4m3 value
constexpr float kLeast = 0.001953125f;              // 2^-9, smallest e4m3 value above zero
constexpr float kTiny = 7.888609052210118e-31f;     // 2^-100

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// A piece of a tensor: 8 values of bf16 or fp32 as they lie in memory.  Whole
// pieces move 16 bytes per access whatever the tensor's alignment: the
// hardware takes vector accesses at any address, so views that start anywhere
// in a flat buffer need no path of their own.
template <bool BF16>
struct Piece {
  uint32_t w[BF16 ? kPiece / 2 : kPiece];

  __device__ __forceinline__ void load(const char* p) { __builtin_memcpy(w, p, sizeof(w)); }
  // the first n >= 1 of them, then zeros (element 0 is read in their place and
  // dropped: no branch between the loads)
  __device__ __forceinline__ void load_first(const char* p, int n) {
#pragma unroll
    for (int k = 0; k < kPiece; ++k) {
      const int i = k < n ? k : 0;
      if (BF16) {
        const uint32_t h = reinterpret_cast<const uint16_t*>(p)[i], x = k < n ? h : 0;
        w[k / 2] = k % 2 ? w[k / 2] | (x << 16) : x;
      } else {
        const uint32_t x = reinterpret_cast<const uint32_t*>(p)[i];
        w[k] = k < n ? x : 0;
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (uint32_t& x : w) x = 0;
  }
  __device__ __forceinline__ float get(int k) const {
    if (!BF16) return __builtin_bit_cast(float, w[k]);
    return __builtin_bit_cast(float, k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
  }
  // bf16 rounds to nearest even
  __device__ __forceinline__ void set(const float* x) {
#pragma unroll
    for (int k = 0; k < kPiece; k += 2) {
      if (BF16) {
        w[k / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x[k], x[k + 1]}, bf16x2));
      } else {
        w[k] = __builtin_bit_cast(uint32_t, x[k]);
        w[k + 1] = __builtin_bit_cast(uint32_t, x[k + 1]);
      }
    }
  }
  __device__ __forceinline__ void store(char* p) const { __builtin_memcpy(p, w, sizeof(w)); }
  __device__ __forceinline__ void store_first(char* p, int n) const {
#pragma unroll
    for (int k = 0; k < kPiece; ++k) {
      if (k >= n) continue;
      if (BF16) {
        reinterpret_cast<uint16_t*>(p)[k] = static_cast<uint16_t>(w[k / 2] >> (k % 2 * 16));
      } else {
        reinterpret_cast<uint32_t*>(p)[k] = w[k];
      }
    }
  }
};

// The same at element e of a tensor's chunk of len elements; `full`: the
// chunk is whole (uniform).
template <bool BF16>
__device__ __forceinline__ void load(Piece<BF16>& x, const char* base, int e, int len, bool full) {
  const char* p = base + e * (BF16 ? 2 : 4);
  if (full || len - e >= kPiece) {
    x.load(p);
  } else if (len - e > 0) {
    x.load_first(p, len - e);
  } else {
    x.clear();
  }
}
template <bool BF16>
__device__ __forceinline__ void store(const Piece<BF16>& x, char* base, int e, int len, bool full) {
  char* p = base + e * (BF16 ? 2 : 4);
  if (full || len - e >= kPiece) {
    x.store(p);
  } else if (len - e > 0) {
    x.store_first(p, len - e);
  }
}

// What one step does to one element.  Every product and sum of the moments is
// rounded by itself (no contraction): both moments then round as the formula
// is written, whichever way the compiler schedules it, and it costs nothing
// beside the memory accesses (equal times for 1.05e9 elements with 8-bit states).
struct Rule {
  float gs, b1, omb1, b2, omb2, sc2, eps, decay, lr;  // sc2 = sqrt(c2); lr includes c1

  __device__ __forceinline__ float first(float m, float g) const {
#pragma clang fp contract(off)
    const float old = b1 * m, add = omb1 * g;
    return old + add;
  }
  __device__ __forceinline__ float second(float v, float g) const {
#pragma clang fp contract(off)
    const float old = b2 * v, add = omb2 * (g * g);
    return old + add;
  }
  // v_rcp_f32 (off by 1.5 ulp, a 1e-7 of the step): the IEEE division took 7 %
  // of the time with 8-bit states
  __device__ __forceinline__ float theta(float p, float m, float r) const {
    return decay * p - lr * m * __builtin_amdgcn_rcpf(r * sc2 + eps);
  }
};

// 32-bit moments: two pieces per thread, 256 pieces apart, so that a wave's
// access covers one contiguous run.  The state is padded, so only the
// parameter and the gradient end inside a piece.
template <bool PB, bool GB>
__device__ __forceinline__ void chunk32(const ParamTensor& t, const Rule& rule, int64_t start, int len, bool full) {
  constexpr int N = kPer / kPiece;
  char* P = t.param + start * (PB ? 2 : 4);
  const char* G = t.grad + start * (GB ? 2 : 4);
  char* M = t.m + start * 4;
  char* V = t.v + start * 4;
  Piece<PB> p[N];
  Piece<GB> g[N];
  Piece<false> m[N], v[N];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int e = (q * kThreads + threadIdx.x) * kPiece;
    load(p[q], P, e, len, full);
    load(g[q], G, e, len, full);
    if (full || e < len) {
      m[q].load(M + e * 4);
      v[q].load(V + e * 4);
    }
  }
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int e = (q * kThreads + threadIdx.x) * kPiece;
    float np[kPiece], nm[kPiece], nv[kPiece];
#pragma unroll
    for (int k = 0; k < kPiece; ++k) {
      const float x = rule.gs * g[q].get(k);
      nm[k] = rule.first(m[q].get(k), x);
      nv[k] = rule.second(v[q].get(k), x);
      np[k] = rule.theta(p[q].get(k), nm[k], sqrtf(nv[k]));
      if (!full && e + k >= len) nm[k] = nv[k] = 0.0f;  // behind the tensor, also where the clip factor is a NaN
    }
    p[q].set(np);
    m[q].set(nm);
    v[q].set(nv);
    store(p[q], P, e, len, full);
    if (full || e < len) {
      m[q].store(M + e * 4);
      v[q].store(V + e * 4);
    }
  }
}

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

// The largest of x >= 0 over a row of 16 lanes, in every one of them, by
// rotations inside the row.  Such floats order as their bits, a NaN above all.
template <int CTRL>
__device__ __forceinline__ uint32_t max_rotated(uint32_t x) {
  const uint32_t y = __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false);
  return x > y ? x : y;
}
__device__ __forceinline__ float row_max(float x) {
  uint32_t u = __builtin_bit_cast(uint32_t, x);
  u = max_rotated<0x128>(u);  // by 8, 4, 2 and 1 lanes
  u = max_rotated<0x124>(u);
  u = max_rotated<0x122>(u);
  u = max_rotated<0x121>(u);
  return __builtin_bit_cast(float, u);
}

// Four values to codes.  v_cvt_sr_fp8_f32 is floor(|y|/q + (seed >> 12) / 2^20) * q
// with y's sign, for normal and subnormal codes (checked on the hardware over
// the range).
__device__ __forceinline__ uint32_t encode4(const float* y, const uint32_t* rnd) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], rnd[0], w, 0);
  w = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], rnd[1], w, 1);
  w = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], rnd[2], w, 2);
  return __builtin_amdgcn_cvt_sr_fp8_f32(y[3], rnd[3], w, 3);
}

// 8-bit moments.  A block of 256 elements is a row of 16 lanes; lane j holds
// the pieces at 8j and 128 + 8j of it, so every access of a wave is
// contiguous within a block (16 elements in one run were 11 % slower with
// fp32 tensors, 88 against 80 us for 25e6 elements, and equal with bf16).
// Everything between the loads and the stores stays in registers: the
// block's maxima are four lane rotations, the codes come and go through the
// e4m3 conversions.  The codes are padded to whole blocks, so only the
// parameter and the gradient end inside a piece; the gap's codes are zero and
// stay zero whatever the block holds, and add nothing to a maximum.
//
// What bounds it is its memory accesses, 5.4 TB/s over three read and three
// written streams (1.94 ms for 1.05e9 bf16 elements): without its arithmetic the
// kernel takes the same time.  Its pointers come out of a descriptor, so the
// accesses are flat ones; what global ones would take is not measured.  The
// first version spent 67 vector instructions on an element and was bound by
// those (2.44 ms): what went is the step's IEEE division, lane exchanges through
// LDS, and bounds checks in whole chunks.  Whole and partial chunks share their
// arithmetic: as two instantiations the kernel had twice the code (now 58 KB),
// and a launch of 300,000 elements in 40 tensors of both types took 10.3 us
// and not 6.1.
template <bool PB, bool GB>
__device__ __forceinline__ void chunk8(const ParamTensor& t, const Rule& rule, int64_t start, int len, bool full,
                                       uint32_t key) {
  constexpr int N = kPer / kPiece;
  const int row = (threadIdx.x >> 4) * kStateBlock;
  const int e = row + (threadIdx.x & 15) * kPiece;
  const bool inside = full || row < len;  // the row's block has elements of this tensor
  char* P = t.param + start * (PB ? 2 : 4);
  const char* G = t.grad + start * (GB ? 2 : 4);
  char* CM = t.m + start + e;
  char* CR = t.v + start + e;
  float2* S = reinterpret_cast<float2*>(t.scales) + (start + row) / kStateBlock;
  Piece<PB> p[N];
  Piece<GB> g[N];
  uint2 wm[N], wr[N];
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int q = 0; q < N; ++q) wm[q] = wr[q] = make_uint2(0, 0);
  if (inside) {
    s = *S;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int o = q * 16 * kPiece;
      wm[q] = *reinterpret_cast<const uint2*>(CM + o);
      wr[q] = *reinterpret_cast<const uint2*>(CR + o);
    }
  }
#pragma unroll
  for (int q = 0; q < N; ++q) {
    load(p[q], P, e + q * 16 * kPiece, len, full);
    load(g[q], G, e + q * 16 * kPiece, len, full);
  }
  float m[kPer], v[kPer];
  float am = 0.0f, av = 0.0f;
#pragma unroll
  for (int z = 0; z < kPer; z += 2) {
    const int q = z / kPiece, k = z % kPiece;
    const uint32_t a = k < 4 ? wm[q].x : wm[q].y, b = k < 4 ? wr[q].x : wr[q].y;
    const f32x2 cm = (k & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8(a, true) : __builtin_amdgcn_cvt_pk_f32_fp8(a, false);
    const f32x2 cr = (k & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8(b, true) : __builtin_amdgcn_cvt_pk_f32_fp8(b, false);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float x = rule.gs * g[q].get(k + j);
      const float r = s.y * cr[j];
      m[z + j] = rule.first(s.x * cm[j], x);
      v[z + j] = rule.second(r * r, x);
      // behind the tensor, also where the block's scale or the clip factor is a NaN
      if (!full && e + q * 16 * kPiece + k + j >= len) m[z + j] = v[z + j] = 0.0f;
    }
    am = max_abs(am, max_abs(m[z], m[z + 1]));
    av = max_abs(av, max_abs(v[z], v[z + 1]));
  }
  am = row_max(am);
  av = row_max(av);
  const float ar = sqrtf(av);
  // 448 * (1 / largest) and largest * (1 / 448), as tensor code computes such
  // quotients: plain elementwise operations give the same codes and scales
  const float im = am < kTiny ? 0.0f : kTop * (1.0f / am);
  const float ir = ar < kTiny ? 0.0f : kTop * (1.0f / ar);
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int o = q * 16 * kPiece;
    const int64_t pos = t.counter + start + e + o;
    const uint32_t ra = mix(static_cast<uint32_t>(pos >> 4) ^ key);
    const uint32_t rb = mix(ra + 0x6A09E667u);
    uint32_t rnd = ra + (static_cast<uint32_t>(pos) & 15u) * rb;
    uint32_t cm[2], cr[2];
    float np[kPiece];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float ym[4], yr[4];
      uint32_t rm[4], rr[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int z = q * kPiece + 4 * i + k;
        const float r = sqrtf(v[z]);
        np[4 * i + k] = rule.theta(p[q].get(4 * i + k), m[z], r);
        rm[k] = rnd;
        rr[k] = (rnd << 16) | (rnd >> 16);
        rnd += rb;
        // the scaled maximum may round past 448; a NaN is in the scale
        ym[k] = __builtin_amdgcn_fmed3f(m[z] * im, -kTop, kTop);
        const float y = __builtin_amdgcn_fmed3f(r * ir, kLeast, kTop);
        yr[k] = v[z] > 0.0f ? y : 0.0f;
        if (!full && e + o + 4 * i + k >= len) ym[k] = 0.0f;  // 0 times a NaN's scale
      }
      cm[i] = encode4(ym, rm);
      cr[i] = encode4(yr, rr);
    }
    p[q].set(np);
    store(p[q], P, e + o, len, full);
    if (inside) {
      *reinterpret_cast<uint2*>(CM + o) = make_uint2(cm[0], cm[1]);
      *reinterpret_cast<uint2*>(CR + o) = make_uint2(cr[0], cr[1]);
    }
  }
  if (inside && (threadIdx.x & 15) == 0)
    *S = make_float2(am < kTiny ? 0.0f : am * (1.0f / kTop), ar < kTiny ? 0.0f : ar * (1.0f / kTop));
}

// One workgroup per chunk beat workgroups that take several (2 to 8 in turn,
// or a grid of 1024 to 16384 that walks the table: 4 to 16 % slower).  The
// chunks run from the last to the first: a norm before the step reads the
// gradients first to last, and what it read last is still in the cache
// (clipped steps over 60e6 to 300e6 elements 0.3 to 3.6 % faster, others equal).
__global__ __launch_bounds__(kThreads) void adamw_multi_kernel(const AdamWMultiArgs a) {
  const int64_t chunk = static_cast<int64_t>(gridDim.x) - 1 - blockIdx.x;
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

  const uint32_t key = mix(mix(static_cast<uint32_t>(step)) ^ a.seed);
  const bool full = len == kParamChunk;
  switch (param_form(t.state_bits, t.param_dtype, t.grad_dtype)) {
    case 0: chunk32<false, false>(t, rule, start, len, full); break;
    case 1: chunk32<false, true>(t, rule, start, len, full); break;
    case 2: chunk32<true, false>(t, rule, start, len, full); break;
    case 3: chunk32<true, true>(t, rule, start, len, full); break;
    case 4: chunk8<false, false>(t, rule, start, len, full, key); break;
    case 5: chunk8<false, true>(t, rule, start, len, full, key); break;
    case 6: chunk8<true, false>(t, rule, start, len, full, key); break;
    case 7: chunk8<true, true>(t, rule, start, len, full, key); break;
  }
}

}  // namespace

hipError_t launch_adamw_multi(const AdamWMultiArgs& a, int64_t total_chunks, hipStream_t stream) {
  if (total_chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(adamw_multi_kernel, dim3(static_cast<unsigned>(total_chunks)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace muon
