// A matrix as e4m3 codes with an fp32 scale for each block of 128: 128
// elements of one row, or a square of 128x128 (include/muon355.h gives the
// format).
//
//   scale = max|x| / 448,   code = round((448 * x) / max|x|)   over a block
//
// The quotient is rounded once, after a correction of the reciprocal's product
// by its remainder, so a quotient that lies half-way between two codes is a
// tie also here: with bf16 inputs, whose quotients are ratios of short
// integers, one in a thousand is.  Written as x * (448 / max|x|) these ties
// fell to either side, and so did those of fp32 inputs with 0.875 x rounded
// before the division.
//
// Both kernels are bound by memory: bytes in plus one byte for each order out.
// 16384 x 4096 bf16: one order 38 us (5.3 TB/s), the transposed one 48, both 60 to
// 67 (4.0 to 4.5 TB/s), both with square blocks 54.  Workgroups that fetch their
// next tile while they work on one were no faster (75), nor were fewer registers
// for more waves (83).

#include "block_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100: a block below it holds zeros
constexpr float kTop = 448.0f;                   // largest e4m3 value

// The larger of two magnitudes; a NaN on either side gives NaN.
__device__ __forceinline__ float max_abs(float a, float b) {
  return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b));
}
// The larger of two floats >= 0, ordered as their bits (a NaN is above all).
__device__ __forceinline__ float max_bits(float a, float b) {
  const uint32_t x = __builtin_bit_cast(uint32_t, a), y = __builtin_bit_cast(uint32_t, b);
  return __builtin_bit_cast(float, x > y ? x : y);
}
// The largest of x >= 0 over a row of 16 lanes, in every one of them.
template <int CTRL>
__device__ __forceinline__ float max_rotated(float x) {
  const int u = __builtin_bit_cast(int, x);
  return max_bits(x, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(u, u, CTRL, 0xf, 0xf, false)));
}
__device__ __forceinline__ float row_max(float x) {
  x = max_rotated<0x128>(x);  // by 8, 4, 2 and 1 lanes
  x = max_rotated<0x124>(x);
  x = max_rotated<0x122>(x);
  return max_rotated<0x121>(x);
}

// a / b from a reciprocal of b: a quotient that fp32 holds comes out as it is,
// another within its last place.
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return __builtin_fmaf(__builtin_fmaf(-q, b, a), r, q);
}
// The same of a + rest, where rest is what fp32 does not hold of a dividend.
__device__ __forceinline__ float quotient(float a, float rest, float b, float r) {
  const float q = a * r;
  return __builtin_fmaf(__builtin_fmaf(-q, b, a) + rest, r, q);
}
// What a block's values are divided by: d = max / 512 (of values times 0.875:
// no product leaves the range) and its reciprocal, the hardware's (off by an
// ulp) corrected by its remainder; 0 for a block of zeros.  (IEEE divisions here
// took 10 % of the time of both orders.)  LONG: the values may have 24
// significant bits, which times 0.875 are up to 27: what its product loses
// joins the remainder (16384 x 4096 in both orders: fp32 84 us against 83
// without, bf16 rows gathered and weighted, whose columns are such products, 91
// against 87).  Values that are bf16 lose nothing.
template <bool LONG>
struct Divisor {
  float d, r;
  __device__ __forceinline__ explicit Divisor(float top) {
    d = top * 0.001953125f;
    const float x = __builtin_amdgcn_rcpf(d);
    r = top < kTiny ? 0.0f : __builtin_fmaf(__builtin_fmaf(-d, x, 1.0f), x, x);
  }
  __device__ __forceinline__ float operator()(float x) const {
    const float a = 0.875f * x;
    return LONG ? quotient(a, __builtin_fmaf(0.875f, x, -a), d, r) : quotient(a, d, r);
  }
};
// top / 448, correctly rounded (the reciprocal of 448 is).
__device__ __forceinline__ float scale_of(float top) {
  return top < kTiny ? 0.0f : quotient(top, kTop, 1.0f / kTop);
}

// A block of one row times its weight w: the weight falls out of the quotients,
// so the codes are the row's own (a tie stays one, which products rounded to
// fp32 lose), with w's sign.  Not where the block is zeros or not finite by its
// weight, or too small without it: the products' there.
struct Weighted {
  float all;     // the largest product
  float factor;  // the values' on their way to the codes
  float top;     // what the codes' values are at most
  __device__ __forceinline__ Weighted(float most, float w) {
    all = __builtin_fabsf(most * w);
    const bool falls_out = most >= kTiny && all >= kTiny && all < __builtin_inff();
    factor = falls_out ? __builtin_copysignf(1.0f, w) : w;
    top = falls_out ? most : all;
  }
};

// Four quotients as codes, to nearest, ties to even.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(4)));  // 16 bytes at the alignment of an fp32 element
typedef u32x4 u32x4_any2 __attribute__((aligned(2)));

// Large matrices go past the caches in both directions (nontemporal accesses):
// 16384 x 4096 bf16 in both orders 66 us against 72.  Small ones stay, for the
// product that reads them next.
// (A matrix's address may come out of a table, and would be read by flat
// accesses: it is global memory.)
template <bool STREAM, typename T>
__device__ __forceinline__ T read(const T* p) {
  const auto g = (__attribute__((address_space(1))) const T*)(p);
  return STREAM ? __builtin_nontemporal_load(g) : *g;
}
template <bool STREAM, typename T>
__device__ __forceinline__ void write(T* p, const T& v) {
  if (STREAM) {
    __builtin_nontemporal_store(v, p);
  } else {
    *p = v;
  }
}

// Eight consecutive elements of a row at any alignment (the hardware takes
// vector accesses at any address), zeros from column `left` on.
template <bool BF16, bool STREAM>
__device__ __forceinline__ void load8(float* v, const char* p, int left) {
  if (BF16) {
    uint32_t w[4] = {0, 0, 0, 0};
    if (left >= 8) {
      const u32x4 t = read<STREAM>(reinterpret_cast<const u32x4_any2*>(p));
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = t[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left)
          w[k / 2] |= static_cast<uint32_t>(read<STREAM>(reinterpret_cast<const uint16_t*>(p) + k)) << (16 * (k % 2));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __builtin_bit_cast(float, k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
    if (left >= 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 t = read<STREAM>(reinterpret_cast<const u32x4_any*>(p) + h);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * h + k] = __builtin_bit_cast(float, static_cast<uint32_t>(t[k]));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) v[k] = read<STREAM>(reinterpret_cast<const float*>(p) + k);
    }
  }
}

__device__ __forceinline__ const char* matrix(const MatBatch& m, int64_t i) {
  return m.ptrs ? static_cast<const char*>(m.ptrs[i]) : m.base + i * m.stride_bytes;
}

// The source of output row r: its address (null: a row of zeros) and factor.
template <bool BF16, bool PAIRS>
__device__ __forceinline__ const char* source(const QuantizeArgs& a, const char* base, int r, float& w) {
  w = 1.0f;
  int64_t s = r;
  if (PAIRS) {
    const int p = a.pairs[r];
    if (p < 0 || p / a.k >= a.in_rows) return nullptr;
    s = p / a.k;
    if (a.weights) w = a.weights[p];
  }
  return base + s * a.x.ld * (BF16 ? 2 : 4);
}

// Blocks of one row, in x's own order only: 16 lanes for a block, 16 rows for
// a workgroup, which walks four blocks of them (1 KB of each row).
template <bool BF16, bool PAIRS, bool STREAM>
__global__ __launch_bounds__(kThreads) void rows_kernel(const QuantizeArgs a) {
  constexpr int kBlocks = 4;
  const int lane = threadIdx.x & 15;
  const uint32_t wide = static_cast<uint32_t>((a.cols + kBlocks * kCodeBlock - 1) / (kBlocks * kCodeBlock));
  const uint32_t by = blockIdx.x / wide, bx = blockIdx.x - by * wide;
  const int64_t r = static_cast<int64_t>(by) * 16 + (threadIdx.x >> 4);
  const int64_t mat = blockIdx.y;
  if (r >= a.rows) return;
  float w;
  const char* src = source<BF16, PAIRS>(a, matrix(a.x, mat), static_cast<int>(r), w);
  char* out = a.q.codes + mat * a.q.stride + r * a.q.ld;
  float* scales = a.q.scales + mat * a.q.scale_stride + r;
  float v[kBlocks][8];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    const int64_t c = (static_cast<int64_t>(bx) * kBlocks + b) * kCodeBlock + 8 * lane;
    const int64_t left = src ? a.cols - c : 0;
    if (left > 0) {
      load8<BF16, STREAM>(v[b], src + c * (BF16 ? 2 : 4), left < 8 ? static_cast<int>(left) : 8);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[b][k] = 0.0f;
    }
  }
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    const int64_t block = static_cast<int64_t>(bx) * kBlocks + b;
    if (block * kCodeBlock >= a.cols) return;
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max_abs(top, v[b][k]);
    top = row_max(top);
    float all = top;
    if (PAIRS) {
      const Weighted x(top, w);
      all = x.all;
      top = x.top;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[b][k] *= x.factor;
    }
    const Divisor<!BF16> div(top);
    const u32x2 u = {encode4(div(v[b][0]), div(v[b][1]), div(v[b][2]), div(v[b][3])),
                     encode4(div(v[b][4]), div(v[b][5]), div(v[b][6]), div(v[b][7]))};
    write<STREAM>(reinterpret_cast<u32x2*>(out + block * kCodeBlock + 8 * lane), u);
    if (lane == 0) scales[block * a.q.scale_ld] = scale_of(all);
  }
}

// A tile of 128x128: a thread holds 8 rows x 8 columns, so a row's maximum is
// over 16 neighbouring lanes and a column's over the threads 16 apart (in LDS
// across waves).  The transposed codes go through LDS, eight rows of a column
// at a time, so that both orders are written in whole rows of 128 codes.
template <bool BF16, bool PAIRS, bool SQUARE, bool STREAM>
__global__ __launch_bounds__(kThreads) void tile_kernel(const QuantizeArgs a) {
  __shared__ __attribute__((aligned(16))) char turned[128 * 128];
  __shared__ float part[4][128];
  const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int64_t mat = blockIdx.y;
  const uint32_t wide = static_cast<uint32_t>((a.cols + 127) / 128);
  const uint32_t by = blockIdx.x / wide, bx = blockIdx.x - by * wide;
  const int64_t r0 = static_cast<int64_t>(by) * 128, c0 = static_cast<int64_t>(bx) * 128;
  const char* base = matrix(a.x, mat);
  const int64_t c = c0 + 8 * tc;
  const int left = static_cast<int>(a.cols - c < 8 ? a.cols - c : 8);
  float v[8][8], w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 8 * tr + i;
    w[i] = 1.0f;
    const char* src = r < a.rows ? source<BF16, PAIRS>(a, base, static_cast<int>(r), w[i]) : nullptr;
    if (src && left > 0) {
      load8<BF16, STREAM>(v[i], src + c * (BF16 ? 2 : 4), left);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = 0.0f;
    }
  }
  char* q = a.q.codes ? a.q.codes + mat * a.q.stride : nullptr;
  char* qt = a.qt.codes ? a.qt.codes + mat * a.qt.stride : nullptr;
  float all = 0.0f;  // SQUARE: the block's maximum
  if (SQUARE) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) all = max_abs(all, v[i][k]);
    all = row_max(all);
    if (tc == 0) part[0][tr] = all;
    __syncthreads();
    all = row_max(part[0][tc]);
    const float s = scale_of(all);
    if (threadIdx.x == 0) {
      if (q) a.q.scales[mat * a.q.scale_stride + bx * a.q.scale_ld + by] = s;
      if (qt) a.qt.scales[mat * a.qt.scale_stride + by * a.qt.scale_ld + bx] = s;
    }
  }
  if (q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + 8 * tr + i;
      float top = all;
      if (!SQUARE) {
        top = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max_abs(top, v[i][k]);
        top = row_max(top);
      }
      float most = top, f = 1.0f;
      if (PAIRS) {
        const Weighted x(top, w[i]);
        most = x.all;
        top = x.top;
        f = x.factor;
      }
      const Divisor<!BF16> div(top);
      auto code4 = [&](const float* p) {
        return PAIRS ? encode4(div(p[0] * f), div(p[1] * f), div(p[2] * f), div(p[3] * f))
                     : encode4(div(p[0]), div(p[1]), div(p[2]), div(p[3]));
      };
      if (r < a.rows) {
        const u32x2 u = {code4(v[i]), code4(v[i] + 4)};
        write<STREAM>(reinterpret_cast<u32x2*>(q + r * a.q.ld + c), u);
        if (!SQUARE && tc == 0)
          a.q.scales[mat * a.q.scale_stride + bx * a.q.scale_ld + r] = scale_of(most);
      }
    }
  }
  if (!qt) return;
  if (PAIRS) {  // a column's values have weights of their own
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] *= w[i];
  }
  float top[8];
  if (!SQUARE) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) t = max_abs(t, v[i][k]);
      t = max_bits(t, __shfl_xor(t, 16));
      top[k] = max_bits(t, __shfl_xor(t, 32));
    }
    if ((threadIdx.x & 48) == 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) part[wave][8 * tc + k] = top[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      top[k] = max_bits(max_bits(part[0][8 * tc + k], part[1][8 * tc + k]),
                        max_bits(part[2][8 * tc + k], part[3][8 * tc + k]));
    if (threadIdx.x < 16) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) a.qt.scales[mat * a.qt.scale_stride + by * a.qt.scale_ld + c + k] = scale_of(top[k]);
    }
  }
  // 16-byte chunk j of column k lies in slot j ^ (k / 8 % 8): the columns that
  // a wave writes together spread over the banks
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const Divisor<!BF16 || PAIRS> div(SQUARE ? all : top[k]);
    uint2 u;
    u.x = encode4(div(v[0][k]), div(v[1][k]), div(v[2][k]), div(v[3][k]));
    u.y = encode4(div(v[4][k]), div(v[5][k]), div(v[6][k]), div(v[7][k]));
    *reinterpret_cast<uint2*>(turned + (8 * tc + k) * 128 + (((tr >> 1) ^ (tc & 7)) << 4) + 8 * (tr & 1)) = u;
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int col = s * 32 + (threadIdx.x >> 3), j = threadIdx.x & 7;
    if (c0 + col >= a.cols) continue;
    const u32x4 u = *reinterpret_cast<const u32x4*>(turned + col * 128 + ((j ^ ((col >> 3) & 7)) << 4));
    write<STREAM>(reinterpret_cast<u32x4*>(qt + (c0 + col) * a.qt.ld + r0 + 16 * j), u);
  }
}

template <bool BF16, bool PAIRS, bool STREAM>
void launch_sized(const QuantizeArgs& a, uint32_t count, hipStream_t s) {
  // the columns of a row of tiles are consecutive workgroups
  if (!a.square && !a.qt.codes) {
    const uint32_t n = static_cast<uint32_t>((a.cols + 511) / 512) * static_cast<uint32_t>((a.rows + 15) / 16);
    rows_kernel<BF16, PAIRS, STREAM><<<dim3(n, count), kThreads, 0, s>>>(a);
    return;
  }
  const dim3 grid(static_cast<uint32_t>((a.cols + 127) / 128) * static_cast<uint32_t>((a.rows + 127) / 128), count);
  if constexpr (!PAIRS) {
    if (a.square) {
      tile_kernel<BF16, false, true, STREAM><<<grid, kThreads, 0, s>>>(a);
      return;
    }
  }
  tile_kernel<BF16, PAIRS, false, STREAM><<<grid, kThreads, 0, s>>>(a);
}

template <bool BF16, bool PAIRS>
void launch(const QuantizeArgs& a, uint32_t count, hipStream_t s) {
  if (static_cast<int64_t>(a.rows) * a.cols * count >= int64_t{1} << 25) {
    launch_sized<BF16, PAIRS, true>(a, count, s);
  } else {
    launch_sized<BF16, PAIRS, false>(a, count, s);
  }
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs& a, int64_t count, hipStream_t s) {
  const uint32_t n = static_cast<uint32_t>(count);
  if (a.x.dtype) {
    a.pairs ? launch<true, true>(a, n, s) : launch<true, false>(a, n, s);
  } else {
    a.pairs ? launch<false, true>(a, n, s) : launch<false, false>(a, n, s);
  }
  return hipGetLastError();
}

}  // namespace muon
