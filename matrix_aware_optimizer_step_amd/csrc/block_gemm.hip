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
// B's rows are the instruction's rows and A's rows its columns, and which row
// of B the instruction's row stands for is chosen when B is read from LDS
// (b_row): a lane ends up with 16 bytes of one row of the result, and four
// lanes with 64, stored without a detour.
//
// A workgroup computes a tile of BM x BN from k-tiles of one block, STAGES of
// them in LDS, filled by global_load_lds_dwordx4.  Rows are 128 bytes; the
// 16-byte chunks of a row are XOR-permuted (a_swizzle, b_swizzle) so that the 16
// rows of a fragment's read cover all 64 banks (no conflict is counted).
//
// Measured: 8192 x 14336 x 4096 into bf16 442 to 485 us (2.0 to 2.2 PFLOP/s,
// by the card's clock; a plain 8-bit product with one scale runs in the library
// in 382), 8192^3 443 (2.5; 355).  The matrix pipes are busy 57 % of the time.
// Without the copies the loop is 17 % faster, without the scales' multiply-adds
// 7 %, without the results' stores 13 % at K = 4096.  Prefetching lines into L2,
// persistent workgroups whose first copies run behind the last tile's stores,
// and copies spread over the steps of a k-tile changed nothing.
// Into fp32 8192 x 8192 x 4096 takes 510 to 550 us (1.0 to 1.1 PFLOP/s): there the
// conversions and the scales are as many instruction cycles as the products.

#include "block_internal.h"

namespace muon {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t lds_address(const void* l) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)(l)));
}
// Global -> LDS copies of 16 or 4 bytes per lane: lane i's bytes at base + off
// land at LDS address l + 16 i (4 i).  Inline asm, as the compiler would
// otherwise wait for them at LDS reads that have nothing to do with them; the
// kernels order them with wait_all_but() and a barrier.  The instruction reads
// m0, which needs a wait state after its write (the compiler adds it to its own
// instructions only).
__device__ __forceinline__ void copy16(const char* base, uint32_t off, uint32_t l) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(__builtin_amdgcn_readfirstlane(l))
               : "memory");
}
__device__ __forceinline__ void copy4(const char* base, uint32_t off, uint32_t l) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "{m0}"(__builtin_amdgcn_readfirstlane(l))
               : "memory");
}
// All LDS accesses of this wave are done and all but its N newest vector loads,
// then the barrier.
template <int N>
__device__ __forceinline__ void wait_all_but() {
  static_assert(N >= 0 && N < 64, "vmcnt has six bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// One block's worth of a 16x16 tile from the 32 codes that each lane holds of a
// row.  WIDE: a bf16 instruction sums the codes, which bf16 holds exactly.
//
// The instruction for 8-bit floats adds eight neighbouring products at a time
// after cutting each off 13 bits below the leading bit of the largest one's
// exponents (measured: of a product 2^-13 of the largest all remains, of one
// 2^-14 nothing).  A result whose products have random signs is off by 5e-5 of its
// size from this, a fortieth of a bf16 result's own rounding but a hundred times
// fp32's; one whose products cancel by less than 2^-10 of each eight's largest,
// far below what the codes themselves are off by (2^-4).  So a BF16 result
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
  static constexpr int kSteps = 1;
  __device__ __forceinline__ f32x4 step(int, const Fragment& o, const f32x4&) const {
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
  static constexpr int kSteps = 4;
  __device__ __forceinline__ f32x4 step(int q, const Fragment& o, const f32x4& p) const {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[q], o.v[q], q ? p : zero, 0, 0, 0);
  }
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// Results lie in global memory, also where the address comes out of a table
// (flat accesses otherwise), at the alignment of their elements.
template <typename T>
using Global = __attribute__((address_space(1))) T*;
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef i32x4 i32x4_any __attribute__((aligned(2)));
typedef i32x2 i32x2_any __attribute__((aligned(2)));

// 16 bytes of a row of the result from column n on, `left` elements of them
// inside the matrix.
template <bool WIDE>
__device__ __forceinline__ void store_run(char* row, int64_t n, int left, const float* v, int accumulate) {
  if (WIDE) {
    Global<float> p = (Global<float>)(reinterpret_cast<float*>(row) + n);
    if (left >= 4) {
      f32x4 u = {v[0], v[1], v[2], v[3]};
      if (accumulate) u += *(Global<const f32x4_any>)(p);
      *(Global<f32x4_any>)(p) = u;
    } else {
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k < left) p[k] = accumulate ? p[k] + v[k] : v[k];
    }
  } else {
    Global<uint16_t> p = (Global<uint16_t>)(reinterpret_cast<uint16_t*>(row) + n);
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = bf16_pair(v[2 * k], v[2 * k + 1]);
    if (left >= 8) {
      *(Global<i32x4_any>)(p) = (i32x4){static_cast<int>(u[0]), static_cast<int>(u[1]), static_cast<int>(u[2]),
                                        static_cast<int>(u[3])};
    } else {
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (k < left) p[k] = static_cast<uint16_t>(u[k / 2] >> (16 * (k % 2)));
    }
  }
}
// The same for four elements.
template <bool WIDE>
__device__ __forceinline__ void store_few(char* row, int64_t n, int left, const float* v, int accumulate) {
  if (WIDE) {
    store_run<true>(row, n, left, v, accumulate);
    return;
  }
  Global<uint16_t> p = (Global<uint16_t>)(reinterpret_cast<uint16_t*>(row) + n);
  const uint32_t u[2] = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
  if (left >= 4) {
    *(Global<i32x2_any>)(p) = (i32x2){static_cast<int>(u[0]), static_cast<int>(u[1])};
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < left) p[k] = static_cast<uint16_t>(u[k / 2] >> (16 * (k % 2)));
  }
}

// B's row (a column of the result) that row r of the instruction's tile j
// stands for.  A lane has four consecutive rows of the instruction, r = 4 g ..
// 4 g + 3, of every j.  F32 results take them as they are: four lanes write 64
// bytes of a row.  BF16 results make two j neighbours, eight consecutive
// columns of a lane, so that four lanes again write 64 bytes together.
template <bool WIDE>
__device__ __forceinline__ int b_row(int j, int r) {
  return WIDE ? 16 * j + r : 32 * (j / 2) + 8 * (r >> 2) + 4 * (j % 2) + (r & 3);
}
// The permutation of the 16-byte chunks of a row in LDS.  Sixteen lanes read a
// chunk of 16 rows together; two rows are 256 bytes, one pass over the banks,
// so the chunks of the 8 pairs of rows have to differ: of consecutive rows, or
// of rows b_row(j, 0 .. 15).
__device__ __forceinline__ int a_swizzle(int row) { return (row >> 1) & 7; }
template <bool WIDE>
__device__ __forceinline__ int b_swizzle(int row) {
  return WIDE ? a_swizzle(row) : ((row >> 1) & 1) | ((row >> 3 & 3) << 1);
}

__device__ __forceinline__ char* c_matrix(const MatBatch& c, int64_t i) {
  return c.ptrs ? static_cast<char*>(c.ptrs[i]) : c.base + i * c.stride_bytes;
}

// Row offset i of the list, kept inside [0, most].
__device__ __forceinline__ int offset_at(const int32_t* offsets, int64_t i, int most) {
  const int o = offsets[i];
  return o < 0 ? 0 : o > most ? most : o;
}

// Segments of rows, each cut into tiles of BM rows by itself.  A wave scans the
// segments, 64 at a time.
template <int BM>
__device__ __forceinline__ int segment_tiles(const BlockGemmArgs& a, int64_t e, int& lo, int& hi) {
  lo = hi = 0;
  if (e < a.count) {
    lo = offset_at(a.offsets, e, a.M);
    hi = offset_at(a.offsets, e + 1, a.M);
  }
  return hi > lo ? (hi - lo + BM - 1) / BM : 0;
}
// The tiles of all segments.
template <int BM>
__device__ __forceinline__ int count_rows(const BlockGemmArgs& a) {
  int lo, hi, sum = 0;
  for (int64_t e = threadIdx.x & 63; e < a.count; e += 64) sum += segment_tiles<BM>(a, e, lo, hi);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
  return __builtin_amdgcn_readfirstlane(sum);
}
// Which segment and which rows the m-tile `tile` is.  False: behind the last.
template <int BM>
__device__ __forceinline__ bool find_rows(const BlockGemmArgs& a, int tile, int& expert, int& first, int& end) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int64_t e0 = 0; e0 < a.count; e0 += 64) {
    int lo, hi;
    const int mine = segment_tiles<BM>(a, e0 + lane, lo, hi);
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
constexpr int kChunkCols = 2;  // REDUCE: tile columns of a chunk of tiles that one XCD takes

// BM x BN tile, WM x WN waves of (BM/WM) x (BN/WN) each.  SB: B has a scale
// for each row.
template <int BM, int BN, int WM, int WN, int STAGES, bool SB, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN, 2) void gemm_kernel(const BlockGemmArgs a) {
  constexpr int NW = WM * WN;
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16;  // 16x16 tiles of a wave
  constexpr int OPB = BM * 128;
  constexpr int STAGE = (BM + BN) * 128;
  constexpr int SCALES = STAGES * STAGE;               // scales of A's rows, then of B's, of STAGES + 1 k-tiles
  constexpr int SCALE_STAGE = BM * 4 + (SB ? BN * 4 : 256);
  constexpr int IA = BM / 8 / NW, IB = BN / 8 / NW;    // copies of 8 rows, per wave
  static_assert(IA * 8 * NW == BM && IB * 8 * NW == BN && SCALES + (STAGES + 1) * SCALE_STAGE <= 160 * 1024, "tile");
  static_assert(BN / WN <= 128 && NT % 2 == 0, "a wave's columns lie in one block of B");
  __shared__ __attribute__((aligned(1024))) char smem[SCALES + (STAGES + 1) * SCALE_STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // Workgroup ids reach the 8 XCDs round-robin: each XCD takes a contiguous
  // range of the tiles, so that tiles that share rows share its L2.  The range
  // is of the tiles that there are: with segments of rows the launch has more.
  // Segments of k have tiles of unequal length: there the XCDs take small
  // chunks of every segment in turn, and their shares come out even.
  const int xcd = blockIdx.x & 7, turn = blockIdx.x >> 3;
  int mat, ti, tj;
  if (a.mode == GEMM_REDUCE) {
    const int high = min(kGroupRows, a.tiles_m), size = high * kChunkCols;
    const int across = (a.tiles_n + kChunkCols - 1) / kChunkCols, down = (a.tiles_m + high - 1) / high;
    const int chunk = turn / size * 8 + xcd, in = turn % size;
    mat = chunk / (across * down);
    const int c = chunk - mat * (across * down);
    ti = c / across * high + in % high;
    tj = c % across * kChunkCols + in / high;
    if (mat >= a.count || ti >= a.tiles_m || tj >= a.tiles_n) return;
  } else {
    const int tiles_m = a.mode == GEMM_ROWS ? count_rows<BM>(a) : a.tiles_m;
    const int per = tiles_m * a.tiles_n;
    const int total = per * (a.mode == GEMM_ROWS ? 1 : static_cast<int>(a.count));
    if (turn >= (total >> 3) + (xcd < (total & 7) ? 1 : 0)) return;
    int t = turn + xcd * (total >> 3) + min(xcd, total & 7);
    mat = t / per;
    t -= mat * per;
    const int span = kGroupRows * a.tiles_n;
    const int grp = t / span, in = t - grp * span;
    const int high = min(kGroupRows, tiles_m - grp * kGroupRows);
    tj = in / high;
    ti = grp * kGroupRows + in - tj * high;
  }

  // the tile's rows [m0, m1) of A, the matrix of B and C, and its blocks of k
  int m0 = ti * BM, m1 = a.M, which = mat, kb0 = 0, nk = (a.K + 127) >> 7;
  int cut_from = 0, cut_to = 128;  // the columns that count, from those of the first block to those of the last
  if (a.mode == GEMM_ROWS) {
    if (!find_rows<BM>(a, ti, which, m0, m1)) return;
  } else if (a.mode == GEMM_REDUCE) {
    const int lo = offset_at(a.offsets, mat, a.K), hi = offset_at(a.offsets, mat + 1, a.K);
    kb0 = lo >> 7;
    nk = hi > lo ? ((hi + 127) >> 7) - kb0 : 0;
    if (nk == 0 && a.accumulate) return;
    cut_from = lo & 127;
    cut_to = hi - ((kb0 + nk - 1) << 7);
  }
  const int n0 = tj * BN;
  const int64_t amat = a.mode == GEMM_BATCH ? mat : 0, bmat = a.mode == GEMM_REDUCE ? 0 : which;
  const char* A = a.a.codes + amat * a.a.stride + m0 * a.a.ld + static_cast<int64_t>(kb0) * 128;
  const char* B = a.b.codes + bmat * a.b.stride + n0 * a.b.ld + static_cast<int64_t>(kb0) * 128;
  const float* SA = a.a.scales + amat * a.a.scale_stride + kb0 * a.a.scale_ld + m0;
  const float* SB0 = a.b.scales + bmat * a.b.scale_stride + kb0 * a.b.scale_ld + (SB ? n0 : n0 >> 7);

  // copies: lane l of an instruction fills slot l % 8 of row l / 8, and a
  // wave's instructions are STEP rows apart; rows behind the matrix repeat its
  // last one (their results are not stored).  The offsets are computed where
  // they are used, two instructions each: held, they cost the registers that
  // keep the loop free of scratch memory.
  constexpr int STEP = 8 * NW;
  static_assert(STEP % 32 == 0, "the swizzles repeat");
  const int row8 = wave * 8 + (lane >> 3);
  const uint32_t chunk_a = ((lane & 7) ^ a_swizzle(row8)) << 4;
  const uint32_t chunk_b = ((lane & 7) ^ b_swizzle<WIDE>(row8)) << 4;
  const int last_a = a.M - 1 - m0, last_b = a.N - 1 - n0;
  const uint32_t lda = static_cast<uint32_t>(a.a.ld), ldb = static_cast<uint32_t>(a.b.ld);
  const uint32_t lds0 = lds_address(smem);
  // scales: 64 of A's rows, or of B's, for a wave (256 x 256 and 128 x 128: one
  // instruction each); waves that are left repeat the last one's
  constexpr int kScaleCopies = BM / 64 + (SB ? BN / 64 : 1);
  static_assert(kScaleCopies <= NW, "one copy of scales for a wave");
  const int slot = min(wave, kScaleCopies - 1);
  const bool of_a = slot < BM / 64;
  const float* const scales = of_a ? SA : SB0;
  const int64_t scale_ld = of_a ? a.a.scale_ld : a.b.scale_ld;
  const uint32_t ofs_s = 4 * (of_a ? min(slot * 64 + lane, last_a)
                                   : SB ? min(slot * 64 - BM + lane, last_b) : min(lane, last_b >> 7));
  auto copy = [&](int kt, uint32_t stage, uint32_t scale_stage) __attribute__((always_inline)) {
    const char* pa = A + static_cast<int64_t>(kt) * 128;
    const char* pb = B + static_cast<int64_t>(kt) * 128;
    const uint32_t l = lds0 + stage;
    int row = row8;
    asm volatile("" : "+v"(row));  // not before the loop: eight registers
#pragma unroll
    for (int r = 0; r < IA; ++r)
      copy16(pa, __umul24(min(row + r * STEP, last_a), lda) + chunk_a, l + wave * 1024 + r * STEP * 128);
#pragma unroll
    for (int r = 0; r < IB; ++r)
      copy16(pb, __umul24(min(row + r * STEP, last_b), ldb) + chunk_b, l + OPB + wave * 1024 + r * STEP * 128);
    copy4(reinterpret_cast<const char*>(scales + kt * scale_ld), ofs_s, lds0 + scale_stage + slot * 256);
  };

  const int wm = wave / WN, wn = wave - wm * WN;
  const int l15 = lane & 15, g = lane >> 4;
  const int arow = wm * (BM / WM) + l15;
  const int brow = wn * (BN / WN) + b_row<WIDE>(0, l15);
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

  // a lane's 32 codes of a row: chunks g and g + 4
  const uint32_t a_lo = arow * 128 + ((g ^ a_swizzle(arow)) << 4), a_hi = a_lo ^ 64;
  const uint32_t b_lo = OPB + brow * 128 + ((g ^ b_swizzle<WIDE>(brow)) << 4), b_hi = b_lo ^ 64;
  const uint32_t a_scale = arow * 4;
  const uint32_t b_scale = BM * 4 + (SB ? (wn * (BN / WN) + b_row<WIDE>(0, 4 * g)) * 4 : wn * (BN / WN) / 128 * 4);

  Fragment<WIDE> fa[MT], fb[2];
  f32x4 p[2][MT], w[2];
  float sa[MT], sa_next[MT];
  // codes as they lie in LDS, and as the matrix instruction takes them (for F32
  // results that is a conversion, which waits for them: it comes later)
  i32x4 raw_a[MT][2], raw_b[2];
  auto read_a = [&](const char* s, int i) {
    raw_a[i][0] = *reinterpret_cast<const i32x4*>(s + a_lo + 2048 * i);
    raw_a[i][1] = *reinterpret_cast<const i32x4*>(s + a_hi + 2048 * i);
  };
  auto set_a = [&](int i) { fa[i].set(raw_a[i][0], raw_a[i][1]); };
  auto read_b = [&](const char* s, int j) {
    const int row = b_row<WIDE>(j, 0);  // 4 more rows, or 16 or 32 more, have the same swizzle
    raw_b[0] = *reinterpret_cast<const i32x4*>(s + b_lo + 128 * row);
    raw_b[1] = *reinterpret_cast<const i32x4*>(s + b_hi + 128 * row);
  };
  auto set_b = [&](int j) { fb[j & 1].set(raw_b[0], raw_b[1]); };
  auto read_scales = [&](const char* s) {
    const float sb = SB ? 1.0f : *reinterpret_cast<const float*>(s + b_scale);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      sa_next[i] = *reinterpret_cast<const float*>(s + a_scale + 64 * i);
      if (!SB) sa_next[i] *= sb;
    }
  };
  // A segment of k may start or end inside a block: A's codes there that belong
  // to its neighbours become zeros, in LDS before a wave reads them for good.  (Where
  // its borders are those of blocks this is two comparisons a tile; 16384 tokens,
  // 8 of 128, 768 x 2048, added: 748 us with borders of blocks, 756 without.  Masks on the
  // fragments inside the loop cost 30 registers and, at 128 x 128, scratch memory.)
  auto cut = [&](uint32_t stage, int from, int to) __attribute__((always_inline)) {
#pragma unroll 1
    for (int x = threadIdx.x; x < BM * 32; x += 64 * NW) {  // four codes of a row
      const int row = x >> 5, at = 4 * (x & 31);
      const int lo = min(max(from - at, 0), 4), hi = max(min(max(to - at, 0), 4), lo);
      *reinterpret_cast<uint32_t*>(smem + stage + row * 128 + (((at >> 4) ^ a_swizzle(row)) << 4) + (at & 15)) &=
          static_cast<uint32_t>((uint64_t{1} << 8 * hi) - (uint64_t{1} << 8 * lo));
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  auto add = [&](int i, int j) {  // a tile's sums, times their scales
#pragma unroll
    for (int r = 0; r < 4; ++r)
      acc[i][j][r] = __builtin_fmaf(SB ? p[j & 1][i][r] * w[j & 1][r] : p[j & 1][i][r], sa[i], acc[i][j][r]);
  };

  // The products of tile column j run while the sums of j - 1 are added and
  // the codes of j + 1 come from LDS.  In the last column's step every wave
  // has read its k-tile: it waits for its copies of the next one, joins the
  // barrier and reads the next one's first codes behind the last products.
  // The order is pinned: left to itself the compiler adds each product at once
  // and waits for it.
  //
  // (A wave may be one barrier ahead of another that still reads its k-tile's
  // scales for B in the last step: scales have a stage more than codes.)
  constexpr int COPIES = IA + IB + 1;  // of a wave for a k-tile
  auto after = [](uint32_t x, uint32_t step, uint32_t from, int n) { return x == from + (n - 1) * step ? from : x + step; };
  uint32_t cs = 0, ss = SCALES;                    // stages that are read
  uint32_t cw = 0, sw = SCALES;                    // and that are copied into
  auto copy_next = [&](int kt) __attribute__((always_inline)) {
    copy(kt, cw, sw);
    cw = after(cw, STAGE, 0, STAGES);
    sw = after(sw, SCALE_STAGE, SCALES, STAGES + 1);
  };
  auto block = [&](int kt, auto last) __attribute__((always_inline)) {
    constexpr bool kMore = !decltype(last)::value;
    const char* s = smem + cs;
    const uint32_t cs_next = after(cs, STAGE, 0, STAGES), ss_next = after(ss, SCALE_STAGE, SCALES, STAGES + 1);
#pragma unroll
    for (int i = 0; i < MT; ++i) sa[i] = sa_next[i];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j + 1 < NT) {
        read_b(s, j + 1);
        if (!WIDE) set_b(j + 1);
      } else if (kMore) {
        if (STAGES > 2 && kt + STAGES - 1 < nk) {
          wait_all_but<(STAGES - 2) * COPIES>();
        } else {
          wait_all_but<0>();
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (SB) w[j & 1] = *reinterpret_cast<const f32x4*>(smem + ss + b_scale + 4 * b_row<WIDE>(j, 0));
      constexpr int Q = Fragment<WIDE>::kSteps;
      if (WIDE && kMore && j + 1 == NT) {
#pragma unroll
        for (int i = 0; i < MT; ++i) read_a(smem + cs_next, i);
        read_b(smem + cs_next, 0);
        read_scales(smem + ss_next);
      }
#pragma unroll
      for (int q = 0; q < Q; ++q) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          p[j & 1][i] = fb[j & 1].step(q, fa[i], p[j & 1][i]);  // (MT sums in turn: none waits for its own last one)
          if (!WIDE) {
            if (j > 0) add(i, j - 1);
            if (kMore && j + 1 == NT) {
              read_a(smem + cs_next, i);
              set_a(i);
              if (i == 0) {
                read_b(smem + cs_next, 0);
                set_b(0);
              }
              if (i == 1) read_scales(smem + ss_next);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          if (kMore && j == 0 && q == 0 && i == 0) {
            if (STAGES == 2 || kt + STAGES - 1 < nk) copy_next(kt + STAGES - 1);
          }
        }
        if (WIDE) {
#pragma unroll
          for (int i = q * MT / Q; i < (q + 1) * MT / Q; ++i)
            if (j > 0) add(i, j - 1);
          if (q + 2 == Q && j + 1 < NT) set_b(j + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) add(i, NT - 1);
    if (WIDE && kMore) {
#pragma unroll
      for (int i = 0; i < MT; ++i) set_a(i);
      set_b(0);
    }
    cs = cs_next;
    ss = ss_next;
  };
  if (nk > 0) {
#pragma unroll
    for (int q = 0; q < STAGES - 1; ++q)
      if (q < nk) copy_next(q);
    if (STAGES > 2 && nk >= STAGES - 1) {
      wait_all_but<(STAGES - 2) * COPIES>();
    } else {
      wait_all_but<0>();
    }
    if (cut_from > 0 || (nk == 1 && cut_to < 128)) cut(0, cut_from, nk == 1 ? cut_to : 128);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      read_a(smem, i);
      set_a(i);
    }
    read_b(smem, 0);
    set_b(0);
    read_scales(smem + ss);
    for (int kt = 0; kt + 1 < nk; ++kt) block(kt, std::false_type{});
    if (nk > 1 && cut_to < 128) {  // what the last step has read of it is read again
      cut(cs, 0, cut_to);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        read_a(smem + cs, i);
        set_a(i);
      }
    }
    block(nk - 1, std::true_type{});
  }

  const int64_t cmat = a.mode == GEMM_ROWS ? 0 : mat;
  char* C = c_matrix(a.c, cmat);
  constexpr int RUN = WIDE ? 4 : 8;  // consecutive columns of a lane
  const int n_first = n0 + wn * (BN / WN);
  if (WIDE && a.accumulate && n_first + BN / WN <= a.N) {
    // a row's old values are all on their way before the first is needed
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int m = m0 + arow + i * 16;
      if (m >= m1) continue;
      char* row = C + m * a.c.ld * 4 + static_cast<int64_t>(n_first) * 4;
      f32x4 old[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) old[j] = *(Global<const f32x4_any>)(row + 4 * b_row<true>(j, 4 * g));
#pragma unroll
      for (int j = 0; j < NT; ++j) *(Global<f32x4_any>)(row + 4 * b_row<true>(j, 4 * g)) = old[j] + acc[i][j];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + arow + i * 16;
    if (m >= m1) continue;
    char* row = C + m * a.c.ld * (WIDE ? 4 : 2);
#pragma unroll
    for (int j = 0; j < NT; j += RUN / 4) {
      const int n = n_first + b_row<WIDE>(j, 4 * g);
      float v[RUN];
#pragma unroll
      for (int r = 0; r < RUN; ++r) v[r] = acc[i][j + r / 4][r % 4];
      store_run<WIDE>(row, n, a.N - n, v, a.accumulate);
    }
  }
}

// Few rows (a token being decoded, or a few for each expert): B is read once
// and that is the time.  A workgroup takes 16 rows of B; its W waves take the
// blocks of k in turn, each straight from memory into the registers that the
// matrix instruction reads, kAhead blocks in flight, and their sums are added
// in the order of the waves in LDS.  All of a 4096 x 4096 matrix is on its way
// at once: 1 x 4096 x 4096 takes 6.7 us from cold memory (2.4 of them an empty
// launch), 1 x 14336 x 4096 15.2 (3.9 TB/s).  The rows of A, MT * 16 at a time,
// come out of L2.  32 tokens to 8 of 128 experts of 768 x 2048 take 36 us from
// cold memory, 5.6 TB/s, with four waves (eight, two blocks each: 49).
//
// In ROWS a workgroup belongs to one expert, so that it needs two offsets and
// no search; an expert with more than MT * 16 rows takes several passes: 1024
// rows to 128 experts of 768 x 2048 take 39 us if each has 8, 42 if one has 135,
// 56 if one has 262 and 159 if one has them all.
template <int MT, int W, bool SB, bool WIDE>
__global__ __launch_bounds__(64 * W) void few_rows_kernel(const BlockGemmArgs a) {
  constexpr int kAhead = MT == 1 ? 4 : 2;
  __shared__ f32x4 part[W][MT][64];
  const int lane = threadIdx.x & 63, l15 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mat = blockIdx.x / a.tiles_n, n0 = (blockIdx.x - mat * a.tiles_n) * 16;
  int first = 0, end = a.M;
  if (a.mode == GEMM_ROWS) {
    first = offset_at(a.offsets, mat, a.M);
    end = offset_at(a.offsets, mat + 1, a.M);
  }
  const int nk = (a.K + 127) >> 7;
  const int64_t amat = a.mode == GEMM_ROWS ? 0 : mat;
  const char* B = a.b.codes + mat * a.b.stride + static_cast<int64_t>(min(n0 + l15, a.N - 1)) * a.b.ld + 16 * g;
  const float* SB0 = a.b.scales + mat * a.b.scale_stride;
  char* C = c_matrix(a.c, amat);
  const int n = n0 + 4 * g;  // this lane's columns of the result
  for (int m0 = first; m0 < end; m0 += MT * 16) {
    const char* A[MT];
    const float* SA[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int64_t m = min(m0 + i * 16 + l15, end - 1);
      A[i] = a.a.codes + amat * a.a.stride + m * a.a.ld + 16 * g;
      SA[i] = a.a.scales + amat * a.a.scale_stride + m;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb0 = wave; kb0 < nk; kb0 += W * kAhead) {
      i32x4 bl[kAhead], bh[kAhead], al[kAhead][MT], ah[kAhead][MT];
      float sa[kAhead][MT], sb[kAhead][SB ? 4 : 1];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int kb = kb0 + u * W;
        if (kb >= nk) break;
        const int64_t k = static_cast<int64_t>(kb) * 128;
        bl[u] = *reinterpret_cast<const i32x4*>(B + k);
        bh[u] = *reinterpret_cast<const i32x4*>(B + k + 64);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          al[u][i] = *reinterpret_cast<const i32x4*>(A[i] + k);
          ah[u][i] = *reinterpret_cast<const i32x4*>(A[i] + k + 64);
          sa[u][i] = SA[i][kb * a.a.scale_ld];
        }
        if (SB) {
#pragma unroll
          for (int r = 0; r < 4; ++r) sb[u][r] = SB0[kb * a.b.scale_ld + min(n + r, a.N - 1)];
        } else {
          sb[u][0] = SB0[kb * a.b.scale_ld + (n0 >> 7)];
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (kb0 + u * W >= nk) break;
        Fragment<WIDE> fb;
        fb.set(bl[u], bh[u]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          Fragment<WIDE> fa;
          fa.set(al[u][i], ah[u][i]);
          f32x4 p;
#pragma unroll
          for (int q = 0; q < Fragment<WIDE>::kSteps; ++q) p = fb.step(q, fa, p);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][r] = __builtin_fmaf(SB ? p[r] * sb[u][r] : p[r], SB ? sa[u][i] : sa[u][i] * sb[u][0], acc[i][r]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave < MT) {
      f32x4 sum = part[0][wave][lane];
#pragma unroll
      for (int q = 1; q < W; ++q) sum += part[q][wave][lane];
      const int m = m0 + wave * 16 + l15;
      if (m < end) {
        const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
        store_few<WIDE>(C + m * a.c.ld * (WIDE ? 4 : 2), n, a.N - n, v, a.accumulate);
      }
    }
    if (m0 + MT * 16 < end) __syncthreads();
  }
}

// Tiles of a launch: in ROWS every segment may end inside a tile.
int64_t count_tiles(BlockGemmArgs& a, int bm, int bn) {
  a.tiles_n = (a.N + bn - 1) / bn;
  a.tiles_m = a.mode == GEMM_ROWS ? static_cast<int32_t>(a.M / bm + a.count) : (a.M + bm - 1) / bm;
  return static_cast<int64_t>(a.tiles_m) * a.tiles_n * (a.mode == GEMM_ROWS ? 1 : a.count);
}
// Workgroups of a launch (gemm_kernel's numbering of the tiles).
int64_t count_workgroups(BlockGemmArgs& a, int bm, int bn) {
  const int64_t tiles = count_tiles(a, bm, bn);
  if (a.mode != GEMM_REDUCE) return tiles;
  const int64_t high = a.tiles_m < kGroupRows ? a.tiles_m : kGroupRows;
  const int64_t chunks = (a.tiles_n + kChunkCols - 1) / kChunkCols * ((a.tiles_m + high - 1) / high) * a.count;
  return (chunks + 7) / 8 * 8 * high * kChunkCols;
}

template <int BM, int BN, int WM, int WN, int STAGES, bool WIDE>
void launch(BlockGemmArgs& a, hipStream_t s) {
  const uint32_t g = static_cast<uint32_t>(count_workgroups(a, BM, BN));
  if (a.square) {
    gemm_kernel<BM, BN, WM, WN, STAGES, false, WIDE><<<g, 64 * WM * WN, 0, s>>>(a);
  } else {
    gemm_kernel<BM, BN, WM, WN, STAGES, true, WIDE><<<g, 64 * WM * WN, 0, s>>>(a);
  }
}

template <int MT, int W, bool WIDE>
void launch_few(BlockGemmArgs& a, hipStream_t s) {
  a.tiles_n = (a.N + 15) / 16;
  const uint32_t g = static_cast<uint32_t>(a.tiles_n * a.count);
  if (a.square) {
    few_rows_kernel<MT, W, false, WIDE><<<g, 64 * W, 0, s>>>(a);
  } else {
    few_rows_kernel<MT, W, true, WIDE><<<g, 64 * W, 0, s>>>(a);
  }
}

// Which kernel and tile, by what was measured (us, bf16 results unless noted):
//   1 .. 32 rows (8 .. 24 on an expert's average): few_rows_kernel; 16 x 4096 x
//     4096 7.7 against 13.9 with tiles of 64; with eight waves from K = 4096 on
//     (one row and 4096 of B, from memory: K = 4096 6.7 against 8.0 with four,
//     8192 10.0 against 12.1), with four below, where eight gain less than a
//     microsecond (2048: 5.0 against 5.2) and lose with many experts (8 rows each
//     of 128 experts of 768 x 2048: 50.6 against 39.2);
//   256 x 256 from 200 tiles on (4096^3: 64 against 82 with 128 x 128; at 128
//     tiles, 2048 x 4096 x 4096, 59 against 43); with segments of rows from 512
//     rows a segment on (512: 189 against 194; 128: 87 against 65);
//   128 x 128 from 128 tiles on, with four stages in flight while there is no
//     more than one tile for a compute unit (1024 x 4096 x 4096: 26 against 38
//     with two, 35 with tiles of 64), with two stages and two workgroups on a
//     compute unit above (2048 x 4096 x 4096: 43 against 49);
//   64 x 64, four stages, below (256 x 4096 x 4096: 14 against 23 and 38).
// F32 results gain nothing from larger tiles than 128 x 128 (8192 x 8192 x
// 4096: 553 against 570 with 256 x 128).
template <bool WIDE>
void launch_typed(BlockGemmArgs& a, hipStream_t s) {
  const int64_t rows = a.mode == GEMM_ROWS ? a.M / a.count : a.M;  // of a segment, on average
  const bool few = a.mode != GEMM_REDUCE && a.count * ((a.N + 15) / 16) < int64_t{1} << 23;
  const bool deep = a.K >= 4096;
  const bool large = count_tiles(a, 256, 256) >= 200 && (a.mode != GEMM_ROWS || rows >= 512);
  if (few && rows <= (a.mode == GEMM_ROWS ? 8 : 16)) {
    deep ? launch_few<1, 8, WIDE>(a, s) : launch_few<1, 4, WIDE>(a, s);
  } else if (few && rows <= (a.mode == GEMM_ROWS ? 24 : 32)) {
    deep ? launch_few<2, 8, WIDE>(a, s) : launch_few<2, 4, WIDE>(a, s);
  } else if (!WIDE && large) {
    launch<256, 256, 4, 2, 2, false>(a, s);
  } else if (count_tiles(a, 128, 128) > 256) {
    launch<128, 128, 2, 2, 2, WIDE>(a, s);
  } else if (count_tiles(a, 128, 128) > 128) {
    launch<128, 128, 4, 2, 4, WIDE>(a, s);
  } else {
    launch<64, 64, 2, 2, 4, WIDE>(a, s);
  }
}

}  // namespace

hipError_t launch_block_gemm(const BlockGemmArgs& args, hipStream_t s) {
  BlockGemmArgs a = args;
  a.c.dtype ? launch_typed<false>(a, s) : launch_typed<true>(a, s);
  return hipGetLastError();
}

}  // namespace muon
