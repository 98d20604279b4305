// Products of 8-bit block codes on CDNA4 matrix cores (gfx950).
//
//   C[m][n] = sum over blocks b of 128 columns:
//             sa[b][m] * sb[b][n or n/128] * (sum over k in b of A[m][k] * B[n][k])
//
// v_mfma_f32_16x16x128_f8f6f4 sums one block of a 16x16 tile in fp32, exactly
// one block's worth, so a scale meets each partial sum once, in an fp32
// multiply-add into the running sums.  That is one vector instruction per
// output element and block (two where B has a scale for each row), half the
// (the whole) time of the matrix instructions, which run beside them.
//
// B's rows are the instruction's rows and A's rows its columns, and the row
// that a lane's four results belong to is chosen freely when B is read from
// LDS: a lane ends up with one row m and 4*NT consecutive columns n of the
// result, which it stores in whole 16-byte pieces without a detour.
//
// A workgroup computes a tile of BM x BN from k-tiles of one block, double
// buffered in LDS by global_load_lds_dwordx4.  Rows are 128 bytes; the 16-byte
// chunks of a row are XOR-permuted (a_swizzle, b_swizzle) so that the 16 rows
// of a fragment's read cover all 64 banks.

#include "block_internal.h"

namespace muon {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t lds_address(const void* l) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)(l)));
}
// Global -> LDS copies of 16 or 4 bytes per lane: lane i's bytes at base + off
// land at LDS address l + 16 i (4 i).  Inline asm, as the compiler would
// otherwise wait for them at LDS reads that have nothing to do with them; the
// kernels order them with wait_all() and a barrier.
__device__ __forceinline__ void copy16(const char* base, uint32_t off, uint32_t l) {
  asm volatile("global_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(__builtin_amdgcn_readfirstlane(l))
               : "memory");
}
__device__ __forceinline__ void copy4(const char* base, uint32_t off, uint32_t l) {
  asm volatile("global_load_lds_dword %0, %1" ::"v"(off), "s"(base), "{m0}"(__builtin_amdgcn_readfirstlane(l))
               : "memory");
}
// All vector loads and LDS accesses of this wave are done, then the barrier.
__device__ __forceinline__ void wait_all() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// One block's worth of a 16x16 tile from the 32 codes that each lane holds of a
// row.  WIDE: a bf16 instruction sums the codes, which bf16 holds exactly.
//
// The instruction for 8-bit floats adds eight neighbouring products at a time
// after cutting each off 13 bits below the leading bit of the largest one's
// exponents (measured: of a product 2^-13 of the largest all remains, of one
// 2^-14 nothing).  A result is off by 5e-5 of its size from this, a fortieth of
// a bf16 result's own rounding but a hundred times fp32's.  So a BF16 result
// takes that instruction, 4.36 PFLOP/s by itself here, and an F32 result, a
// gradient that many batches add to, the bf16 one, 2.29 PFLOP/s.
template <bool WIDE>
struct Fragment;
template <>
struct Fragment<false> {
  i32x8 v;
  __device__ __forceinline__ void set(const i32x4& lo, const i32x4& hi) {
    v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  __device__ __forceinline__ f32x4 operator*(const Fragment& o) const {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, o.v, zero, 0, 0, 0, 0, 0, 0);
  }
};
template <>
struct Fragment<true> {
  bf16x8 v[4];
  __device__ __forceinline__ static bf16x8 eight(int a, int b) {
    const bf16x2 w0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const bf16x2 w1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const bf16x2 w2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const bf16x2 w3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    return __builtin_shufflevector(__builtin_shufflevector(w0, w1, 0, 1, 2, 3),
                                   __builtin_shufflevector(w2, w3, 0, 1, 2, 3), 0, 1, 2, 3, 4, 5, 6, 7);
  }
  __device__ __forceinline__ void set(const i32x4& lo, const i32x4& hi) {
    v[0] = eight(lo[0], lo[1]);
    v[1] = eight(lo[2], lo[3]);
    v[2] = eight(hi[0], hi[1]);
    v[3] = eight(hi[2], hi[3]);
  }
  __device__ __forceinline__ f32x4 operator*(const Fragment& o) const {
    f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[q], o.v[q], p, 0, 0, 0);
    return p;
  }
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// N consecutive results of a row, `left` of them inside the matrix.
template <int N>
__device__ __forceinline__ void store_row(const MatBatch& c, char* row, int64_t col, int left, const float* v,
                                          int accumulate) {
  if (left <= 0) return;
  if (c.dtype) {
    char* p = row + col * 2;
    if (left >= N && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
#pragma unroll
      for (int k = 0; k < N; k += 8) {
        uint4 u;
        u.x = bf16_pair(v[k], v[k + 1]);
        u.y = bf16_pair(v[k + 2], v[k + 3]);
        u.z = bf16_pair(v[k + 4], v[k + 5]);
        u.w = bf16_pair(v[k + 6], v[k + 7]);
        *reinterpret_cast<uint4*>(p + 2 * k) = u;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < left) reinterpret_cast<__bf16*>(p)[k] = static_cast<__bf16>(v[k]);
    }
    return;
  }
  float* p = reinterpret_cast<float*>(row) + col;
  if (left >= N && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
#pragma unroll
    for (int k = 0; k < N; k += 4) {
      float4 u = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      if (accumulate) {
        const float4 o = *reinterpret_cast<const float4*>(p + k);
        u = make_float4(o.x + u.x, o.y + u.y, o.z + u.z, o.w + u.w);
      }
      *reinterpret_cast<float4*>(p + k) = u;
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < left) p[k] = accumulate ? p[k] + v[k] : v[k];
  }
}

// The permutation of the 16-byte chunks of a row in LDS.  Sixteen lanes read a
// chunk of 16 rows together; two rows are 256 bytes, one pass over the banks,
// so the chunks of the 8 pairs of rows have to differ: consecutive rows for A,
// rows {0, 1, 2, 3} + 4 j + SPAN * {0, 1, 2, 3} for B.
__device__ __forceinline__ int a_swizzle(int row) { return (row >> 1) & 7; }
template <int SPAN>
__device__ __forceinline__ int b_swizzle(int row) {
  return ((row >> 1) & 1) | ((row / SPAN & 3) << 1);
}

// Row offset i of the list, kept inside [0, most] and above the one before.
__device__ __forceinline__ int offset_at(const int32_t* offsets, int64_t i, int most) {
  const int o = offsets[i];
  return o < 0 ? 0 : o > most ? most : o;
}

// Which expert and which rows the m-tile `tile` of a list of segments is:
// every segment is cut into tiles of BM rows by itself.  A wave scans the
// segments, 64 at a time.  False: behind the last tile.
template <int BM>
__device__ __forceinline__ bool find_rows(const BlockGemmArgs& a, int tile, int& expert, int& first, int& end) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int64_t e0 = 0; e0 < a.count; e0 += 64) {
    const int64_t e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < a.count) {
      lo = offset_at(a.offsets, e, a.M);
      hi = offset_at(a.offsets, e + 1, a.M);
    }
    const int mine = hi > lo ? (hi - lo + BM - 1) / BM : 0;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int x = __shfl_up(sum, d);
      if (lane >= d) sum += x;
    }
    const int start = before + sum - mine;
    const uint64_t hit = __ballot(tile >= start && tile < start + mine);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      expert = static_cast<int>(e0) + l;
      first = __builtin_amdgcn_readlane(lo, l) + (tile - __builtin_amdgcn_readlane(start, l)) * BM;
      end = __builtin_amdgcn_readlane(hi, l);
      return true;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

constexpr int kGroupRows = 8;  // tile rows that are walked together, column by column

// BM x BN tile, WM x WN waves of (BM/WM) x (BN/WN) each.  SB: B has a scale
// for each row.
template <int BM, int BN, int WM, int WN, bool SB, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN, 2) void gemm_kernel(const BlockGemmArgs a) {
  constexpr int NW = WM * WN;
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16;  // 16x16 tiles of a wave
  constexpr int SPAN = 4 * NT;                         // consecutive columns of a lane
  constexpr int OPB = BM * 128;
  constexpr int SCALES = (BM + BN) * 128;              // scales of A's rows, then of B's
  constexpr int STAGE = SCALES + (BM + (SB ? BN : 0)) * 4;
  constexpr int IA = BM / 8 / NW, IB = BN / 8 / NW;    // copies of 8 rows, per wave
  static_assert(IA * 8 * NW == BM && IB * 8 * NW == BN && 2 * STAGE <= 160 * 1024, "tile");
  static_assert(BM / 64 + (SB ? BN / 64 : 0) <= 2 * NW && BN / WN <= 128, "scale copies");
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // workgroup ids reach the 8 XCDs round-robin: each XCD takes a contiguous
  // range of the tiles, so that tiles that share rows share its L2
  const int total = static_cast<int>(a.total_tiles);
  const int xcd = blockIdx.x & 7;
  int t = (blockIdx.x >> 3) + xcd * (total >> 3) + (xcd < (total & 7) ? xcd : (total & 7));
  const int per = a.tiles_m * a.tiles_n;
  const int mat = t / per;
  t -= mat * per;
  const int span = kGroupRows * a.tiles_n;
  const int grp = t / span, in = t - grp * span;
  const int high = min(kGroupRows, a.tiles_m - grp * kGroupRows);
  const int tj = in / high, ti = grp * kGroupRows + in - tj * high;

  // the tile's rows [m0, m1) of A, the matrix of B and C, and its blocks of k
  int m0 = ti * BM, m1 = a.M, which = mat, kb0 = 0, nk = (a.K + 127) >> 7;
  if (a.mode == GEMM_ROWS) {
    if (!find_rows<BM>(a, ti, which, m0, m1)) return;
  } else if (a.mode == GEMM_REDUCE) {
    const int lo = offset_at(a.offsets, mat, a.K) >> 7, hi = (offset_at(a.offsets, mat + 1, a.K) + 127) >> 7;
    kb0 = lo;
    nk = hi > lo ? hi - lo : 0;
    if (nk == 0 && a.accumulate) return;
  }
  const int n0 = tj * BN;
  const int64_t amat = a.mode == GEMM_BATCH ? mat : 0, bmat = a.mode == GEMM_REDUCE ? 0 : which;
  const char* A = a.a.codes + amat * a.a.stride + m0 * a.a.ld + static_cast<int64_t>(kb0) * 128;
  const char* B = a.b.codes + bmat * a.b.stride + n0 * a.b.ld + static_cast<int64_t>(kb0) * 128;
  const float* SA = a.a.scales + amat * a.a.scale_stride + kb0 * a.a.scale_ld + m0;
  const float* SB0 = a.b.scales + bmat * a.b.scale_stride + kb0 * a.b.scale_ld;

  // copies: lane l of an instruction fills slot l % 8 of row l / 8, and a
  // wave's instructions are STEP rows apart; rows behind the matrix repeat its
  // last one (their results are not stored).  The offsets are computed where
  // they are used, two instructions each: held, they cost the registers that
  // keep the loop free of scratch memory.
  constexpr int STEP = 8 * NW;
  static_assert(STEP % 16 == 0 && (STEP / SPAN == 2 || STEP / SPAN == 4), "the swizzles repeat");
  const int row8 = wave * 8 + (lane >> 3);
  const uint32_t chunk_a = ((lane & 7) ^ a_swizzle(row8)) << 4;
  const uint32_t chunk_b = ((lane & 7) ^ b_swizzle<SPAN>(row8)) << 4;
  const int last_a = a.M - 1 - m0, last_b = a.N - 1 - n0;
  const uint32_t lda = static_cast<uint32_t>(a.a.ld), ldb = static_cast<uint32_t>(a.b.ld);
  const uint32_t lds0 = lds_address(smem);
  auto copy = [&](int kt, int stage) {
    const char* pa = A + static_cast<int64_t>(kt) * 128;
    const char* pb = B + static_cast<int64_t>(kt) * 128;
    const uint32_t l = lds0 + stage * STAGE + wave * 1024;
#pragma unroll
    for (int r = 0; r < IA; ++r)
      copy16(pa, __umul24(min(row8 + r * STEP, last_a), lda) + chunk_a, l + r * STEP * 128);
#pragma unroll
    for (int r = 0; r < IB; ++r)
      copy16(pb, __umul24(min(row8 + r * STEP, last_b), ldb) + (chunk_b ^ (STEP / SPAN == 2 && r % 2 ? 64 : 0)),
             l + OPB + r * STEP * 128);
    // the scales, 64 rows an instruction
#pragma unroll
    for (int r = 0; r < (BM / 64 + (SB ? BN / 64 : 0) + NW - 1) / NW; ++r) {
      const int q = wave + r * NW;
      if (q < BM / 64) {
        copy4(reinterpret_cast<const char*>(SA + kt * a.a.scale_ld), 4 * min(q * 64 + lane, last_a),
              lds0 + stage * STAGE + SCALES + q * 256);
      } else if (SB && q < BM / 64 + BN / 64) {
        copy4(reinterpret_cast<const char*>(SB0 + kt * a.b.scale_ld + n0), 4 * min(q * 64 - BM + lane, last_b),
              lds0 + stage * STAGE + SCALES + q * 256);
      }
    }
  };

  const int wm = wave / WN, wn = wave - wm * WN;
  const int l15 = lane & 15, g = lane >> 4;
  const int arow = wm * (BM / WM) + l15;
  const int brow = wn * (BN / WN) + (l15 >> 2) * SPAN + (l15 & 3);  // tile j adds 4 j
  const int sbn = min(n0 + wn * (BN / WN), a.N - 1) >> 7;  // block row of B, square blocks
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

  // a lane's 32 codes of a row: chunks g and g + 4.  (Tile rows 16 apart, and
  // B's rows 4 j apart, share the swizzle up to b_swizzle's lowest bit, which
  // 4 j leaves alone.)
  const uint32_t a_lo = arow * 128 + ((g ^ a_swizzle(arow)) << 4), a_hi = a_lo ^ 64;
  const uint32_t b_lo = OPB + brow * 128 + ((g ^ b_swizzle<SPAN>(brow)) << 4), b_hi = b_lo ^ 64;
  const uint32_t a_scale = SCALES + arow * 4, b_scale = SCALES + (BM + wn * (BN / WN) + g * SPAN) * 4;

  if (nk > 0) copy(0, 0);
  float sq = 0.0f;
  if (!SB && nk > 0) sq = SB0[sbn];
  wait_all();
  for (int kt = 0; kt < nk; ++kt) {
    const char* s = smem + (kt & 1) * STAGE;
    const float sb = sq;
    if (kt + 1 < nk) {
      copy(kt + 1, (kt + 1) & 1);
      if (!SB) sq = SB0[(kt + 1) * a.b.scale_ld + sbn];
    }
    Fragment<WIDE> fa[MT], fb[2];
    float sa[MT];
    f32x4 p[2][MT], w[2];
    auto read_b = [&](int j) {
      fb[j & 1].set(*reinterpret_cast<const i32x4*>(s + b_lo + 512 * j),
                    *reinterpret_cast<const i32x4*>(s + b_hi + 512 * j));
    };
    auto add = [&](int i, int j) {  // a tile's sums, times their scales
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[i][j][r] = __builtin_fmaf(SB ? p[j & 1][i][r] * w[j & 1][r] : p[j & 1][i][r], sa[i], acc[i][j][r]);
    };
#pragma unroll
    for (int i = 0; i < MT; ++i)
      fa[i].set(*reinterpret_cast<const i32x4*>(s + a_lo + 2048 * i),
                *reinterpret_cast<const i32x4*>(s + a_hi + 2048 * i));
    read_b(0);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      sa[i] = *reinterpret_cast<const float*>(s + a_scale + 64 * i);
      if (!SB) sa[i] *= sb;
    }
    // The products of tile column j run while the sums of j - 1 are added and
    // the codes of j + 1 come from LDS.  The order is pinned: left to itself
    // the compiler adds each product at once and waits for it.
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j + 1 < NT) read_b(j + 1);
      if (SB) w[j & 1] = *reinterpret_cast<const f32x4*>(s + b_scale + 16 * j);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        p[j & 1][i] = fb[j & 1] * fa[i];
        if (j > 0) add(i, j - 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) add(i, NT - 1);
    wait_all();
  }

  const int64_t cmat = a.mode == GEMM_ROWS ? 0 : mat;
  char* C = a.c.ptrs ? static_cast<char*>(a.c.ptrs[cmat]) : a.c.base + cmat * a.c.stride_bytes;
  const int n = n0 + wn * (BN / WN) + g * SPAN;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + arow + i * 16;
    if (m >= m1) continue;
    float v[SPAN];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[4 * j + r] = acc[i][j][r];
    store_row<SPAN>(a.c, C + m * a.c.ld * (a.c.dtype ? 2 : 4), n, a.N - n, v, a.accumulate);
  }
}

// Tiles of a launch: in ROWS every segment may end inside a tile.
int64_t count_tiles(BlockGemmArgs& a, int bm, int bn) {
  a.tiles_n = (a.N + bn - 1) / bn;
  a.tiles_m = a.mode == GEMM_ROWS ? static_cast<int32_t>(a.M / bm + a.count) : (a.M + bm - 1) / bm;
  a.total_tiles = static_cast<int64_t>(a.tiles_m) * a.tiles_n * (a.mode == GEMM_ROWS ? 1 : a.count);
  return a.total_tiles;
}

template <int BM, int BN, int WM, int WN, bool WIDE>
void launch(BlockGemmArgs& a, hipStream_t s) {
  const uint32_t g = static_cast<uint32_t>(count_tiles(a, BM, BN));
  if (a.square) {
    gemm_kernel<BM, BN, WM, WN, false, WIDE><<<g, 64 * WM * WN, 0, s>>>(a);
  } else {
    gemm_kernel<BM, BN, WM, WN, true, WIDE><<<g, 64 * WM * WN, 0, s>>>(a);
  }
}

}  // namespace

hipError_t launch_block_gemm(const BlockGemmArgs& args, hipStream_t s) {
  BlockGemmArgs a = args;
  if (a.c.dtype) {
    if (count_tiles(a, 256, 256) >= 200) {
      launch<256, 256, 4, 2, false>(a, s);
    } else {
      launch<128, 128, 2, 2, false>(a, s);
    }
  } else if (count_tiles(a, 256, 128) >= 200) {
    launch<256, 128, 4, 2, true>(a, s);
  } else {
    launch<128, 128, 2, 2, true>(a, s);
  }
  return hipGetLastError();
}

}  // namespace muon
