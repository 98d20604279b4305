// C-ABI layer of the expert layers: 8-bit block codes, their products, the
// routing to experts and the experts' sums.  Contracts are in
// include/muon355.h.

#include "../../include/muon355.h"

#include <cstddef>
#include <cstdint>

#include "abi_common.h"
#include "block_internal.h"

namespace {

using namespace muon;

static_assert(kCodeBlock == MUON_CODE_BLOCK, "code block");

constexpr int64_t kMaxExtent = (int64_t{1} << 31) - 128;
// a launch has fewer than 2^32 work-items; workgroups have at most 512
constexpr int64_t kMaxWorkgroups = (int64_t{1} << 23) - 1;

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A batch of dense matrices.  `gathered`: pairs name its rows.
muon_status_t check_dense(const muon_batch_t* b, const char* name) {
  if (!b) return fail(MUON_ERR_INVALID_VALUE, "%s: descriptor is NULL", name);
  if (b->dtype != MUON_F32 && b->dtype != MUON_BF16)
    return fail(MUON_ERR_INVALID_VALUE, "%s: dtype %d is not MUON_F32 or MUON_BF16", name, b->dtype);
  if (b->reserved != 0) return fail(MUON_ERR_INVALID_VALUE, "%s: reserved field must be 0", name);
  if (b->count < 1 || b->count > 65535)
    return fail(MUON_ERR_INVALID_VALUE, "%s: count %lld outside [1, 65535]", name, (long long)b->count);
  if (b->rows < 1 || b->rows > kMaxExtent || b->cols < 1 || b->cols > kMaxExtent)
    return fail(MUON_ERR_INVALID_VALUE, "%s: %lld x %lld outside [1, 2^31-128]", name, (long long)b->rows,
                (long long)b->cols);
  if (b->ld < b->cols || b->ld > kMaxExtent)
    return fail(MUON_ERR_INVALID_VALUE, "%s: ld %lld outside [cols, 2^31-128]", name, (long long)b->ld);
  if (!b->ptrs && !b->base) return fail(MUON_ERR_INVALID_VALUE, "%s: both ptrs and base are NULL", name);
  if (!b->ptrs && b->count > 1 && b->stride < (b->rows - 1) * b->ld + b->cols)
    return fail(MUON_ERR_INVALID_VALUE, "%s: stride %lld overlaps consecutive matrices", name, (long long)b->stride);
  if (!b->ptrs && !aligned(b->base, b->dtype == MUON_BF16 ? 2 : 4))
    return fail(MUON_ERR_INVALID_VALUE, "%s: base is not aligned to its element size", name);
  return MUON_OK;
}

MatBatch to_mat(const muon_batch_t* b) {
  MatBatch m{};
  m.base = static_cast<char*>(b->base);
  m.stride_bytes = b->stride * (b->dtype == MUON_BF16 ? 2 : 4);
  m.ptrs = b->ptrs;
  m.ld = b->ld;
  m.dtype = b->dtype;
  return m;
}

muon_status_t check_codes(const muon_codes_t* q, const char* name) {
  if (!q) return fail(MUON_ERR_INVALID_VALUE, "%s: descriptor is NULL", name);
  if (q->reserved != 0) return fail(MUON_ERR_INVALID_VALUE, "%s: reserved field must be 0", name);
  if (!q->codes || !q->scales) return fail(MUON_ERR_INVALID_VALUE, "%s: codes or scales are NULL", name);
  if (!aligned(q->codes, 16) || !aligned(q->scales, 4))
    return fail(MUON_ERR_INVALID_VALUE, "%s: codes must be 16-byte, scales 4-byte aligned", name);
  if (q->count < 1 || q->count > 65535)
    return fail(MUON_ERR_INVALID_VALUE, "%s: count %lld outside [1, 65535]", name, (long long)q->count);
  if (q->rows < 1 || q->rows > kMaxExtent || q->cols < 1 || q->cols > kMaxExtent)
    return fail(MUON_ERR_INVALID_VALUE, "%s: %lld x %lld outside [1, 2^31-128]", name, (long long)q->rows,
                (long long)q->cols);
  if (q->block_rows != 1 && q->block_rows != MUON_CODE_BLOCK)
    return fail(MUON_ERR_INVALID_VALUE, "%s: block_rows %d is not 1 or 128", name, q->block_rows);
  const int64_t wide = ceil_div(q->cols, MUON_CODE_BLOCK) * MUON_CODE_BLOCK;
  if (q->ld < wide || q->ld % 16 != 0 || q->ld >= int64_t{1} << 31)
    return fail(MUON_ERR_INVALID_VALUE, "%s: ld %lld must be a multiple of 16, at least cols in whole blocks (%lld) and "
                "below 2^31", name, (long long)q->ld, (long long)wide);
  const int64_t high = ceil_div(q->rows, q->block_rows);
  if (q->scale_ld < high || q->scale_ld >= int64_t{1} << 31)
    return fail(MUON_ERR_INVALID_VALUE, "%s: scale_ld %lld outside [%lld, 2^31)", name, (long long)q->scale_ld,
                (long long)high);
  if (q->count > 1) {
    if (q->stride % 16 != 0 || q->stride < (q->rows - 1) * q->ld + wide)
      return fail(MUON_ERR_INVALID_VALUE, "%s: stride %lld must be a multiple of 16 and not overlap matrices", name,
                  (long long)q->stride);
    if (q->scale_stride < (wide / MUON_CODE_BLOCK - 1) * q->scale_ld + high)
      return fail(MUON_ERR_INVALID_VALUE, "%s: scale_stride %lld overlaps consecutive matrices", name,
                  (long long)q->scale_stride);
  }
  return MUON_OK;
}

CodeMat to_codes(const muon_codes_t* q) {
  CodeMat m{};
  m.codes = static_cast<char*>(q->codes);
  m.scales = q->scales;
  m.stride = q->stride;
  m.scale_stride = q->scale_stride;
  m.ld = q->ld;
  m.scale_ld = q->scale_ld;
  return m;
}

}  // namespace

extern "C" {

muon_status_t muon_block_quantize(const muon_batch_t* x, const int32_t* pairs, const float* weights, int64_t k,
                                  const muon_codes_t* q, const muon_codes_t* qt, void* stream) {
  muon_status_t st;
  if ((st = check_dense(x, "x")) != MUON_OK) return st;
  if (!q && !qt) return fail(MUON_ERR_INVALID_VALUE, "q and qt are both NULL");
  if (q && (st = check_codes(q, "q")) != MUON_OK) return st;
  if (qt && (st = check_codes(qt, "qt")) != MUON_OK) return st;
  const int64_t rows = q ? q->rows : qt->cols, cols = q ? q->cols : qt->rows;
  if (q && qt && (qt->cols != rows || qt->rows != cols || qt->count != q->count || qt->block_rows != q->block_rows))
    return fail(MUON_ERR_INVALID_VALUE, "q and qt are not of one matrix");
  const int32_t block_rows = q ? q->block_rows : qt->block_rows;
  const int64_t count = q ? q->count : qt->count;
  if (cols != x->cols || count != x->count || (!pairs && rows != x->rows))
    return fail(MUON_ERR_INVALID_VALUE, "the codes' shape is not x's");
  if (k < 1 || k > (int64_t{1} << 31) - 1) return fail(MUON_ERR_INVALID_VALUE, "k %lld outside [1, 2^31)", (long long)k);
  if (!pairs && (weights || k != 1)) return fail(MUON_ERR_INVALID_VALUE, "weights and k need pairs");
  if (pairs && (count != 1 || x->ptrs)) return fail(MUON_ERR_INVALID_VALUE, "pairs take one matrix");
  if (pairs && block_rows != 1) return fail(MUON_ERR_UNSUPPORTED, "pairs take blocks of one row");
  if (pairs && (!aligned(pairs, 4) || !aligned(weights, 4)))
    return fail(MUON_ERR_INVALID_VALUE, "pairs and weights must be 4-byte aligned");
  if (ceil_div(rows, 16) * ceil_div(cols, 128) > kMaxWorkgroups)
    return fail(MUON_ERR_UNSUPPORTED, "%lld x %lld is too large for one launch", (long long)rows, (long long)cols);
  QuantizeArgs a{};
  a.x = to_mat(x);
  a.pairs = pairs;
  a.weights = weights;
  a.k = static_cast<int32_t>(k);
  a.in_rows = static_cast<int32_t>(x->rows);
  a.rows = static_cast<int32_t>(rows);
  a.cols = static_cast<int32_t>(cols);
  a.square = block_rows == MUON_CODE_BLOCK;
  if (q) a.q = to_codes(q);
  if (qt) a.qt = to_codes(qt);
  const hipError_t e = launch_quantize(a, count, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return launch_status(e, "quantize");
  return done(static_cast<hipStream_t>(stream), "muon_block_quantize");
}

muon_status_t muon_block_matmul(const muon_codes_t* a, const muon_codes_t* b, const muon_batch_t* c,
                                const int32_t* offsets, int32_t product, int32_t accumulate, void* stream) {
  muon_status_t st;
  if ((st = check_codes(a, "a")) != MUON_OK) return st;
  if ((st = check_codes(b, "b")) != MUON_OK) return st;
  if ((st = check_dense(c, "c")) != MUON_OK) return st;
  if (product < MUON_PRODUCT_BATCH || product > MUON_PRODUCT_REDUCE)
    return fail(MUON_ERR_INVALID_VALUE, "unknown product %d", product);
  if (accumulate != 0 && accumulate != 1) return fail(MUON_ERR_INVALID_VALUE, "accumulate must be 0 or 1");
  if (accumulate && c->dtype != MUON_F32) return fail(MUON_ERR_UNSUPPORTED, "only an F32 result accumulates");
  if (a->block_rows != 1) return fail(MUON_ERR_UNSUPPORTED, "a's blocks must have one row");
  if (a->cols != b->cols) return fail(MUON_ERR_INVALID_VALUE, "a and b differ in columns");
  if (c->rows != a->rows || c->cols != b->rows) return fail(MUON_ERR_INVALID_VALUE, "c is not rows(a) x rows(b)");
  // 256 rows of codes are within reach of a 32-bit offset
  if (a->ld >= int64_t{1} << 24 || b->ld >= int64_t{1} << 24)
    return fail(MUON_ERR_UNSUPPORTED, "rows of 2^24 bytes and more");
  const int64_t many = product == MUON_PRODUCT_REDUCE ? c->count : b->count;
  if (product == MUON_PRODUCT_BATCH) {
    if (a->count != many || c->count != many) return fail(MUON_ERR_INVALID_VALUE, "counts differ");
    if (offsets) return fail(MUON_ERR_INVALID_VALUE, "offsets go with ROWS and REDUCE");
  } else {
    if (!offsets || !aligned(offsets, 4))
      return fail(MUON_ERR_INVALID_VALUE, "offsets must be a 4-byte aligned device address");
    if (a->count != 1 || (product == MUON_PRODUCT_ROWS ? c->count : b->count) != 1)
      return fail(MUON_ERR_INVALID_VALUE, "one matrix each where the offsets divide it");
  }
  const int64_t tiles = (ceil_div(a->rows, 128) + (product == MUON_PRODUCT_ROWS ? many : 0)) * ceil_div(b->rows, 128) *
                        (product == MUON_PRODUCT_ROWS ? 1 : many);
  if (tiles > kMaxWorkgroups) return fail(MUON_ERR_UNSUPPORTED, "the product is too large for one launch");
  BlockGemmArgs g{};
  g.a = to_codes(a);
  g.b = to_codes(b);
  g.c = to_mat(c);
  g.offsets = offsets;
  g.count = many;
  g.M = static_cast<int32_t>(a->rows);
  g.N = static_cast<int32_t>(b->rows);
  g.K = static_cast<int32_t>(a->cols);
  g.mode = product;
  g.square = b->block_rows == MUON_CODE_BLOCK;
  g.accumulate = accumulate;
  const hipError_t e = launch_block_gemm(g, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return launch_status(e, "block matmul");
  return done(static_cast<hipStream_t>(stream), "muon_block_matmul");
}

}  // extern "C"
