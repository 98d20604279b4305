// C-ABI layer of the expert layers: 8-bit block codes, their products, the
// routing to experts and the experts' sums.  Contracts are in
// include/muon355.h.

#include "../../include/muon355.h"

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "abi_common.h"
#include "block_internal.h"

namespace {

using namespace muon;

static_assert(kCodeBlock == MUON_CODE_BLOCK && kMaxExperts == MUON_MAX_EXPERTS && kMaxChosen == MUON_MAX_CHOSEN &&
                  kMaxExpertGroups == MUON_MAX_EXPERT_GROUPS,
              "limits");

constexpr int64_t kMaxExtent = (int64_t{1} << 31) - 128;
// a launch has fewer than 2^32 work-items; workgroups have at most 512
constexpr int64_t kMaxWorkgroups = (int64_t{1} << 23) - 1;

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A batch of dense matrices.
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

// Rows of the order by expert, 0 where it has more than 2^31-1.
int64_t route_rows(int64_t tokens, int64_t experts, int64_t k, int64_t align) {
  const int64_t n = ceil_div(tokens * k + experts * (align - 1), align) * align;
  return n < int64_t{1} << 31 ? n : 0;
}
bool route_sizes_ok(int64_t tokens, int64_t experts, int64_t k, int64_t align) {
  return tokens >= 1 && tokens < int64_t{1} << 31 && experts >= 1 && experts <= MUON_MAX_EXPERTS && k >= 1 &&
         k <= MUON_MAX_CHOSEN && k <= experts && align >= 1 && align <= 65536 && tokens * k < int64_t{1} << 31;
}

muon_status_t check_route(const muon_route_t* r) {
  if (!r) return fail(MUON_ERR_INVALID_VALUE, "description is NULL");
  if (r->dtype != MUON_F32 && r->dtype != MUON_BF16)
    return fail(MUON_ERR_INVALID_VALUE, "dtype %d is not MUON_F32 or MUON_BF16", r->dtype);
  if (!r->logits || !aligned(r->logits, r->dtype == MUON_BF16 ? 2 : 4))
    return fail(MUON_ERR_INVALID_VALUE, "logits are NULL or not aligned to their element size");
  if (!route_sizes_ok(r->tokens, r->experts, r->k, r->align))
    return fail(MUON_ERR_INVALID_VALUE, "tokens %lld, experts %lld, k %lld or align %d is out of range",
                (long long)r->tokens, (long long)r->experts, (long long)r->k, r->align);
  if (r->ld < r->experts || r->ld > kMaxExtent)
    return fail(MUON_ERR_INVALID_VALUE, "ld %lld outside [experts, 2^31-128]", (long long)r->ld);
  if (r->score != MUON_SCORE_SOFTMAX && r->score != MUON_SCORE_SIGMOID)
    return fail(MUON_ERR_INVALID_VALUE, "unknown score %d", r->score);
  if (r->renormalize != 0 && r->renormalize != 1) return fail(MUON_ERR_INVALID_VALUE, "renormalize must be 0 or 1");
  if (r->groups < 1 || r->groups > MUON_MAX_EXPERT_GROUPS || r->experts % r->groups != 0)
    return fail(MUON_ERR_INVALID_VALUE, "groups %d outside [1, %d] or no divisor of the experts", r->groups,
                MUON_MAX_EXPERT_GROUPS);
  if (r->top_groups < 1 || r->top_groups > r->groups)
    return fail(MUON_ERR_INVALID_VALUE, "top_groups %d outside [1, groups]", r->top_groups);
  if (r->k > r->experts / r->groups * r->top_groups)
    return fail(MUON_ERR_INVALID_VALUE, "k %lld is more than the experts of the groups that stay", (long long)r->k);
  if (r->group_best != 1 && r->group_best != 2) return fail(MUON_ERR_INVALID_VALUE, "group_best must be 1 or 2");
  if (!std::isfinite(r->scale)) return fail(MUON_ERR_INVALID_VALUE, "scale must be finite");
  return MUON_OK;
}

// y, the tokens' matrix and the slots of a sum or a dot.
muon_status_t check_sum(const muon_batch_t* y, const muon_batch_t* t, const char* name, const int32_t* slots,
                        int64_t k, int64_t jobs_per_token) {
  muon_status_t st;
  if ((st = check_dense(y, "y")) != MUON_OK) return st;
  if ((st = check_dense(t, name)) != MUON_OK) return st;
  if (y->count != 1 || t->count != 1 || y->ptrs || t->ptrs)
    return fail(MUON_ERR_INVALID_VALUE, "y and %s must be one matrix each, given by base", name);
  if (y->cols != t->cols) return fail(MUON_ERR_INVALID_VALUE, "y and %s differ in columns", name);
  if (k < 1 || k > MUON_MAX_CHOSEN)
    return fail(MUON_ERR_INVALID_VALUE, "k %lld outside [1, %d]", (long long)k, MUON_MAX_CHOSEN);
  if (!slots || !aligned(slots, 4)) return fail(MUON_ERR_INVALID_VALUE, "slots must be a 4-byte aligned device address");
  if (t->rows * jobs_per_token > kMaxWorkgroups * 4)
    return fail(MUON_ERR_UNSUPPORTED, "%lld x %lld is too large for one launch", (long long)t->rows,
                (long long)t->cols);
  return MUON_OK;
}

}  // namespace

extern "C" {

muon_status_t muon_block_quantize(const muon_batch_t* x, const int32_t* pairs, const float* weights, int64_t k,
                                  const muon_codes_t* q, const muon_codes_t* qt, void* stream) {
  muon_status_t st;
  muon_batch_t one;  // x without rows (every pair is behind them): nothing of it is read
  if (x && x->rows == 0 && pairs) {
    one = *x;
    one.rows = 1;
    one.base = const_cast<int32_t*>(pairs);
    if ((st = check_dense(&one, "x")) != MUON_OK) return st;
  } else if ((st = check_dense(x, "x")) != MUON_OK) {
    return st;
  }
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
  // (REDUCE numbers its tiles in chunks, up to four times as many)
  if (tiles > (product == MUON_PRODUCT_REDUCE ? kMaxWorkgroups / 4 : kMaxWorkgroups))
    return fail(MUON_ERR_UNSUPPORTED, "the product is too large for one launch");
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

int64_t muon_route_capacity(int64_t tokens, int64_t experts, int64_t k, int64_t align) {
  return route_sizes_ok(tokens, experts, k, align) && tokens <= MUON_MAX_ORDERED_TOKENS
             ? route_rows(tokens, experts, k, align)
             : 0;
}

size_t muon_route_workspace(int64_t tokens, int64_t experts) {
  if (!route_sizes_ok(tokens, experts, 1, 1)) return 0;
  // the counts of every 16 or 64 tokens, a byte each; never less than fewer tokens need
  const int64_t few = tokens < kMostInRunsOf16 ? tokens : kMostInRunsOf16;
  const int64_t runs = ceil_div(tokens, route_group(tokens, experts));
  const int64_t before = ceil_div(few, route_group(few, experts));
  const size_t bytes = static_cast<size_t>((runs > before ? runs : before) * (ceil_div(experts, 16) * 16));
  return bytes < 256 ? 256 : bytes;
}

muon_status_t muon_route(const muon_route_t* r, const float* bias, const uint8_t* mask, int32_t* chosen,
                         float* weights, int32_t* slots, int32_t* pairs, int32_t* offsets, int32_t* loads,
                         void* workspace, size_t ws_bytes, void* stream) {
  const muon_status_t st = check_route(r);
  if (st != MUON_OK) return st;
  if (!chosen || !weights) return fail(MUON_ERR_INVALID_VALUE, "chosen or weights are NULL");
  if ((slots != nullptr) != (pairs != nullptr) || (slots != nullptr) != (offsets != nullptr))
    return fail(MUON_ERR_INVALID_VALUE, "slots, pairs and offsets go together");
  if (!aligned(bias, 4) || !aligned(chosen, 4) || !aligned(weights, 4) || !aligned(slots, 4) || !aligned(pairs, 4) ||
      !aligned(offsets, 4) || !aligned(loads, 4))
    return fail(MUON_ERR_INVALID_VALUE, "every array must be 4-byte aligned");
  // the workgroup of every 256 tokens sums all counts: 137 GB out of L2 at this many of 128 experts
  if ((slots || loads) && r->tokens > MUON_MAX_ORDERED_TOKENS)
    return fail(MUON_ERR_UNSUPPORTED, "an order or loads of %lld tokens, more than %d", (long long)r->tokens,
                MUON_MAX_ORDERED_TOKENS);
  const int64_t rows = route_rows(r->tokens, r->experts, r->k, r->align);
  if (slots && rows == 0) return fail(MUON_ERR_UNSUPPORTED, "the order has more than 2^31-1 rows");
  const size_t need = muon_route_workspace(r->tokens, r->experts);
  if (!workspace || ws_bytes < need)
    return fail(MUON_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", ws_bytes, need);
  if (!aligned(workspace, 16)) return fail(MUON_ERR_WORKSPACE, "workspace must be 16-byte aligned");
  // 1024 lanes for 64 tokens
  if (ceil_div(r->tokens, 64) >= int64_t{1} << 22)
    return fail(MUON_ERR_UNSUPPORTED, "%lld tokens are too many for one launch", (long long)r->tokens);
  RouteArgs a{};
  a.logits = static_cast<const char*>(r->logits);
  a.ld = r->ld;
  a.bias = bias;
  a.mask = mask;
  a.chosen = chosen;
  a.weights = weights;
  a.slots = slots;
  a.pairs = pairs;
  a.offsets = offsets;
  a.loads = loads;
  a.counts = static_cast<uint8_t*>(workspace);
  a.capacity = rows;
  a.tokens = static_cast<int32_t>(r->tokens);
  a.experts = static_cast<int32_t>(r->experts);
  a.k = static_cast<int32_t>(r->k);
  a.dtype = r->dtype;
  a.sigmoid = r->score == MUON_SCORE_SIGMOID;
  a.renormalize = r->renormalize;
  a.groups = r->groups;
  a.top_groups = r->top_groups;
  a.group_best = r->group_best;
  a.align = r->align;
  a.scale = r->scale;
  const hipError_t e = launch_route(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return launch_status(e, "route");
  return done(static_cast<hipStream_t>(stream), "muon_route");
}

muon_status_t muon_route_backward(const muon_route_t* r, const int32_t* chosen, const float* weights,
                                  const float* grad_weights, void* grad_logits, int64_t ld_grad, void* stream) {
  const muon_status_t st = check_route(r);
  if (st != MUON_OK) return st;
  if (!chosen || !weights || !grad_weights || !grad_logits)
    return fail(MUON_ERR_INVALID_VALUE, "a required array is NULL");
  if (!aligned(chosen, 4) || !aligned(weights, 4) || !aligned(grad_weights, 4) ||
      !aligned(grad_logits, r->dtype == MUON_BF16 ? 2 : 4))
    return fail(MUON_ERR_INVALID_VALUE, "every array must be aligned to its element size");
  if (ld_grad < r->experts || ld_grad > kMaxExtent)
    return fail(MUON_ERR_INVALID_VALUE, "ld_grad %lld outside [experts, 2^31-128]", (long long)ld_grad);
  if (ceil_div(r->tokens, 16) >= int64_t{1} << 24)
    return fail(MUON_ERR_UNSUPPORTED, "%lld tokens are too many for one launch", (long long)r->tokens);
  RouteBackwardArgs a{};
  a.logits = static_cast<const char*>(r->logits);
  a.ld = r->ld;
  a.chosen = chosen;
  a.weights = weights;
  a.grad = grad_weights;
  a.out = static_cast<char*>(grad_logits);
  a.ld_out = ld_grad;
  a.tokens = static_cast<int32_t>(r->tokens);
  a.experts = static_cast<int32_t>(r->experts);
  a.k = static_cast<int32_t>(r->k);
  a.dtype = r->dtype;
  a.sigmoid = r->score == MUON_SCORE_SIGMOID;
  a.renormalize = r->renormalize;
  a.scale = r->scale;
  const hipError_t e = launch_route_backward(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return launch_status(e, "route backward");
  return done(static_cast<hipStream_t>(stream), "muon_route_backward");
}

muon_status_t muon_balance_update(float* bias, int32_t* loads, int64_t experts, float rate,
                                  const muon_step_control_t* control, void* stream) {
  if (!bias || !loads || !aligned(bias, 4) || !aligned(loads, 4))
    return fail(MUON_ERR_INVALID_VALUE, "bias and loads must be 4-byte aligned device addresses");
  if (experts < 1 || experts > MUON_MAX_EXPERTS)
    return fail(MUON_ERR_INVALID_VALUE, "experts %lld outside [1, %d]", (long long)experts, MUON_MAX_EXPERTS);
  if (!std::isfinite(rate) || rate < 0.0f) return fail(MUON_ERR_INVALID_VALUE, "rate must be finite and >= 0");
  if (control && !aligned(control, 16))
    return fail(MUON_ERR_INVALID_VALUE, "control must be a 16-byte aligned device address");
  BalanceArgs a{};
  a.bias = bias;
  a.loads = loads;
  a.experts = static_cast<int32_t>(experts);
  a.rate = rate;
  a.control = reinterpret_cast<const StepControl*>(control);
  const hipError_t e = launch_balance(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return launch_status(e, "balance");
  return done(static_cast<hipStream_t>(stream), "muon_balance_update");
}

muon_status_t muon_expert_sum(const muon_batch_t* y, const int32_t* slots, const float* weights, int64_t k,
                              const muon_batch_t* out, void* stream) {
  const muon_status_t st = check_sum(y, out, "out", slots, k, out ? ceil_div(out->cols, 512) : 1);
  if (st != MUON_OK) return st;
  if (!aligned(weights, 4)) return fail(MUON_ERR_INVALID_VALUE, "weights must be 4-byte aligned");
  ExpertSumArgs a{};
  a.y = to_mat(y);
  a.out = to_mat(out);
  a.slots = slots;
  a.weights = weights;
  a.tokens = out->rows;
  a.rows = static_cast<int32_t>(y->rows);
  a.cols = static_cast<int32_t>(y->cols);
  a.k = static_cast<int32_t>(k);
  const hipError_t e = launch_expert_sum(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return launch_status(e, "expert sum");
  return done(static_cast<hipStream_t>(stream), "muon_expert_sum");
}

muon_status_t muon_expert_dot(const muon_batch_t* grad, const muon_batch_t* y, const int32_t* slots, int64_t k,
                              float* dots, void* stream) {
  const muon_status_t st = check_sum(y, grad, "grad", slots, k, ceil_div(k, 4));
  if (st != MUON_OK) return st;
  if (!dots || !aligned(dots, 4)) return fail(MUON_ERR_INVALID_VALUE, "dots must be a 4-byte aligned device address");
  ExpertSumArgs a{};
  a.y = to_mat(y);
  a.out = to_mat(grad);
  a.slots = slots;
  a.dots = dots;
  a.tokens = grad->rows;
  a.rows = static_cast<int32_t>(y->rows);
  a.cols = static_cast<int32_t>(y->cols);
  a.k = static_cast<int32_t>(k);
  const hipError_t e = launch_expert_dot(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return launch_status(e, "expert dot");
  return done(static_cast<hipStream_t>(stream), "muon_expert_dot");
}

}  // extern "C"
