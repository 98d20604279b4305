// Drives the C-ABI layer of the expert operators with stand-in launchers that
// check every launch the layer builds: each operand of a kernel, over its whole
// extent, must lie inside what the caller described.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "block_internal.h"
#include "muon355.h"

static long checks = 0, launches = 0;
static void require(bool ok, const char* what) {
  ++checks;
  if (!ok) {
    std::fprintf(stderr, "launch: %s\n", what);
    std::abort();
  }
}

namespace muon {
hipError_t launch_quantize(const QuantizeArgs& a, int64_t count, hipStream_t) {
  ++launches;
  require(a.rows >= 1 && a.cols >= 1 && count >= 1 && a.k >= 1 && a.in_rows >= 1, "quantize: sizes");
  require(a.q.codes || a.qt.codes, "quantize: an output");
  const int64_t wide = (int64_t{a.cols} + 127) / 128 * 128, high = (int64_t{a.rows} + 127) / 128 * 128;
  if (a.q.codes) require(a.q.ld >= wide && a.q.scale_ld >= (a.square ? high / 128 : a.rows), "quantize: q");
  if (a.qt.codes) require(a.qt.ld >= high && a.qt.scale_ld >= (a.square ? wide / 128 : a.cols), "quantize: qt");
  require(a.pairs || a.in_rows == a.rows, "quantize: rows of x");
  require((int64_t{a.rows} + 15) / 16 * (wide / 128) < int64_t{1} << 23, "quantize: workgroups");
  return hipSuccess;
}
hipError_t launch_block_gemm(const BlockGemmArgs& a, hipStream_t) {
  ++launches;
  require(a.M >= 1 && a.N >= 1 && a.K >= 1 && a.count >= 1, "product: sizes");
  require(a.a.ld >= (int64_t{a.K} + 127) / 128 * 128 && a.b.ld >= a.a.ld / a.a.ld * ((int64_t{a.K} + 127) / 128 * 128),
          "product: rows");
  require(a.a.ld * 256 < int64_t{1} << 32 && a.b.ld * 256 < int64_t{1} << 32, "product: 256 rows within 32 bits");
  require((a.mode == GEMM_BATCH) == (a.offsets == nullptr), "product: offsets");
  require(!a.accumulate || a.c.dtype == 0, "product: accumulates in F32");
  const int64_t tiles = ((int64_t{a.M} + 63) / 64 + (a.mode == GEMM_ROWS ? a.count : 0)) * ((int64_t{a.N} + 63) / 64);
  // tiles of 64 are taken where there are few of 128: at most 128 of those
  require(tiles < (int64_t{1} << 25), "product: workgroups");
  return hipSuccess;
}
hipError_t launch_route(const RouteArgs& a, hipStream_t) {
  ++launches;
  require(a.tokens >= 1 && a.experts >= 1 && a.experts <= kMaxExperts && a.k >= 1 && a.k <= kMaxChosen, "route: sizes");
  require(a.groups <= kMaxExpertGroups && a.experts % a.groups == 0 && a.k <= a.experts / a.groups * a.top_groups,
          "route: groups");
  const int64_t most = int64_t{a.tokens} * a.k + int64_t{a.experts} * (a.align - 1);
  require(!a.slots || (a.capacity >= most && a.capacity % a.align == 0), "route: capacity");
  require(static_cast<size_t>((a.tokens + route_group(a.tokens, a.experts) - 1) / route_group(a.tokens, a.experts)) *
                  ((a.experts + 15) / 16 * 16) <=
              muon_route_workspace(a.tokens, a.experts),
          "route: workspace");
  return hipSuccess;
}
hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t) {
  ++launches;
  require(a.tokens >= 1 && a.experts <= kMaxExperts && a.k <= kMaxChosen && a.ld_out >= a.experts, "backward");
  return hipSuccess;
}
hipError_t launch_balance(const BalanceArgs& a, hipStream_t) {
  ++launches;
  require(a.experts >= 1 && a.experts <= kMaxExperts && a.rate >= 0, "balance");
  return hipSuccess;
}
hipError_t launch_expert_sum(const ExpertSumArgs& a, hipStream_t) {
  ++launches;
  require(a.tokens >= 1 && a.rows >= 1 && a.k >= 1 && a.k <= kMaxChosen, "sum");
  require(a.tokens * ((a.cols + 511) / 512) < int64_t{1} << 31, "sum: jobs");
  return hipSuccess;
}
hipError_t launch_expert_dot(const ExpertSumArgs& a, hipStream_t) {
  ++launches;
  require(a.dots && a.tokens >= 1 && a.k <= kMaxChosen, "dot");
  return hipSuccess;
}
}  // namespace muon

static void expect(muon_status_t got, muon_status_t want, const char* what) {
  ++checks;
  if (got != want || (got == MUON_OK) != (std::strlen(muon_last_error()) == 0)) {
    std::fprintf(stderr, "%s: status %d, expected %d (%s)\n", what, got, want, muon_last_error());
    std::abort();
  }
}

int main() {
  char* fake = reinterpret_cast<char*>(uintptr_t{1} << 40);  // device addresses, never dereferenced
  auto* scales = reinterpret_cast<float*>(fake + 4096);
  auto* ints = reinterpret_cast<int32_t*>(fake + 8192);
  auto up = [](int64_t n) { return (n + 127) / 128 * 128; };
  auto codes = [&](int64_t rows, int64_t cols, int32_t block, int64_t count) {
    const int64_t high = (rows + block - 1) / block;
    return muon_codes_t{fake, scales, rows * up(cols), up(cols) / 128 * high, count, rows, cols, up(cols), high, block, 0};
  };
  auto dense = [&](int64_t rows, int64_t cols, int32_t dtype, int64_t count) {
    return muon_batch_t{nullptr, fake, rows * cols, count, rows, cols, cols, dtype, 0};
  };
  const int64_t sizes[][2] = {{1, 1}, {127, 129}, {4096, 14336}, {131072, 2048}, {(int64_t{1} << 31) - 128, 1}, {16, 1 << 23}};
  for (auto& s : sizes)
    for (int32_t block : {1, 128})
      for (int64_t count : {1, 3}) {
        muon_batch_t x = dense(s[0], s[1], MUON_BF16, count);
        muon_codes_t q = codes(s[0], s[1], block, count), qt = codes(s[1], s[0], block, count);
        const bool fits = (s[0] + 15) / 16 * ((s[1] + 127) / 128) < int64_t{1} << 23;
        if (q.ld >= int64_t{1} << 31 || qt.ld >= int64_t{1} << 31) continue;
        expect(muon_block_quantize(&x, nullptr, nullptr, 1, &q, nullptr, nullptr), fits ? MUON_OK : MUON_ERR_UNSUPPORTED, "q");
        expect(muon_block_quantize(&x, nullptr, nullptr, 1, &q, &qt, nullptr), fits ? MUON_OK : MUON_ERR_UNSUPPORTED, "both");
      }
  {
    muon_batch_t x = dense(1000, 300, MUON_F32, 1);
    muon_codes_t q = codes(77, 300, 1, 1), qt = codes(300, 77, 1, 1);
    expect(muon_block_quantize(&x, ints, scales, 8, &q, &qt, nullptr), MUON_OK, "pairs");
    expect(muon_block_quantize(&x, ints, nullptr, 1, nullptr, &qt, nullptr), MUON_OK, "pairs, transposed");
  }
  const int64_t products[][3] = {{1, 1, 1}, {1, 4096, 4096}, {8192, 14336, 4096}, {1111, 1000, 2049}, {65536, 65536, 128}};
  for (auto& p : products)
    for (int32_t block : {1, 128})
      for (int32_t dtype : {MUON_F32, MUON_BF16}) {
        muon_codes_t a = codes(p[0], p[2], 1, 1), b = codes(p[1], p[2], block, 1), b3 = codes(p[1], p[2], block, 3);
        muon_batch_t c = dense(p[0], p[1], dtype, 1), c3 = dense(p[0], p[1], dtype, 3);
        expect(muon_block_matmul(&a, &b, &c, nullptr, MUON_PRODUCT_BATCH, 0, nullptr), MUON_OK, "batch");
        expect(muon_block_matmul(&a, &b3, &c, ints, MUON_PRODUCT_ROWS, dtype == MUON_F32, nullptr), MUON_OK, "rows");
        expect(muon_block_matmul(&a, &b, &c3, ints, MUON_PRODUCT_REDUCE, 0, nullptr), MUON_OK, "reduce");
      }
  for (int64_t tokens : {int64_t{1}, int64_t{64}, int64_t{65}, int64_t{16384}, int64_t{16385}, int64_t{1} << 26})
    for (int64_t experts : {1, 17, 256, 257, 512})
      for (int32_t align : {1, 128, 65536}) {
        const int64_t k = experts < 4 ? 1 : 4;
        muon_route_t r{fake, experts, tokens, experts, k, MUON_F32, MUON_SCORE_SIGMOID, 1, 1, 1, 2, align, 1.0f};
        const size_t need = muon_route_workspace(tokens, experts);
        const int64_t rows = muon_route_capacity(tokens, experts, k, align);
        if (rows == 0) continue;
        expect(muon_route(&r, scales, nullptr, ints, scales, ints, ints, ints, ints, fake, need, nullptr), MUON_OK, "route");
        expect(muon_route(&r, nullptr, nullptr, ints, scales, nullptr, nullptr, nullptr, nullptr, fake, need, nullptr), MUON_OK, "bare");
        expect(muon_route(&r, nullptr, nullptr, ints, scales, ints, ints, ints, nullptr, fake, need - 1, nullptr), MUON_ERR_WORKSPACE, "short");
        expect(muon_route_backward(&r, ints, scales, scales, fake, experts, nullptr), MUON_OK, "backward");
      }
  expect(muon_balance_update(scales, ints, 512, 0.0f, nullptr, nullptr), MUON_OK, "balance");
  for (int64_t tokens : {1, 32, 65536})
    for (int64_t cols : {1, 513, 8192}) {
      muon_batch_t y = dense(tokens * 8, cols, MUON_BF16, 1), out = dense(tokens, cols, MUON_F32, 1);
      expect(muon_expert_sum(&y, ints, scales, 8, &out, nullptr), MUON_OK, "sum");
      expect(muon_expert_sum(&y, ints, nullptr, 16, &out, nullptr), MUON_OK, "sum of ones");
      expect(muon_expert_dot(&out, &y, ints, 8, scales, nullptr), MUON_OK, "dot");
    }
  expect(muon_block_quantize(nullptr, nullptr, nullptr, 1, nullptr, nullptr, nullptr), MUON_ERR_INVALID_VALUE, "null");
  expect(muon_block_matmul(nullptr, nullptr, nullptr, nullptr, 0, 0, nullptr), MUON_ERR_INVALID_VALUE, "null");
  expect(muon_route(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr), MUON_ERR_INVALID_VALUE, "null");
  expect(muon_expert_sum(nullptr, ints, nullptr, 1, nullptr, nullptr), MUON_ERR_INVALID_VALUE, "null");
  std::printf("ok: %ld checks, %ld launches\n", checks, launches);
}
