// Drives the C-ABI layer of the many-tensor operators through valid and
// invalid arguments, with stand-in launchers (optim_stubs.cpp).
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <limits>

#include "muon355.h"

extern "C" void optim_stub_workspace(const void* base, size_t bytes);
extern "C" long optim_stub_launches();
extern "C" void stub_set_workspace(const void* base, size_t bytes);

static long checks = 0;
static void expect(muon_status_t got, muon_status_t want, const char* what) {
  ++checks;
  if (got != want) {
    std::fprintf(stderr, "%s: status %d, expected %d (%s)\n", what, got, want, muon_last_error());
    std::abort();
  }
  if ((got == MUON_OK) != (std::strlen(muon_last_error()) == 0)) {
    std::fprintf(stderr, "%s: error text '%s'\n", what, muon_last_error());
    std::abort();
  }
}

int main() {
  char* fake = reinterpret_cast<char*>(uintptr_t{1} << 40);  // device addresses, never dereferenced
  const float inf = std::numeric_limits<float>::infinity(), nan = std::numeric_limits<float>::quiet_NaN();
  auto* control = reinterpret_cast<muon_step_control_t*>(fake + 4096);

  for (int64_t chunks : {int64_t{0}, int64_t{1}, int64_t{511}, int64_t{512}, int64_t{1} << 20, (int64_t{1} << 31) - 1}) {
    muon_grad_list_t l{3, chunks, reinterpret_cast<const muon_grad_t*>(fake), reinterpret_cast<const int32_t*>(fake + 64)};
    const size_t need = muon_grad_norm_workspace(chunks);
    optim_stub_workspace(fake + 8192, need);
    expect(muon_grad_norm(&l, 1.0f, 0, control, fake + 8192, need, nullptr), MUON_OK, "norm");
    expect(muon_grad_norm(&l, inf, MUON_SKIP_NONFINITE, control, fake + 8192, need, nullptr), MUON_OK, "norm inf");
    expect(muon_grad_norm(&l, 1.0f, 0, control, fake + 8192, need - 1, nullptr), MUON_ERR_WORKSPACE, "norm short");
  }
  muon_grad_list_t l{3, 5, reinterpret_cast<const muon_grad_t*>(fake), reinterpret_cast<const int32_t*>(fake + 64)};
  const long before = optim_stub_launches();
  for (float bad : {0.0f, -1.0f, nan}) expect(muon_grad_norm(&l, bad, 0, control, fake, 256, nullptr), MUON_ERR_INVALID_VALUE, "max_norm");
  expect(muon_grad_norm(&l, 1.0f, 2, control, fake, 256, nullptr), MUON_ERR_INVALID_VALUE, "flags");
  expect(muon_grad_norm(&l, 1.0f, 0, nullptr, fake, 256, nullptr), MUON_ERR_INVALID_VALUE, "control");
  expect(muon_grad_norm(&l, 1.0f, 0, reinterpret_cast<muon_step_control_t*>(fake + 8), fake, 256, nullptr), MUON_ERR_INVALID_VALUE, "control alignment");
  expect(muon_grad_norm(&l, 1.0f, 0, control, nullptr, 256, nullptr), MUON_ERR_WORKSPACE, "workspace");
  expect(muon_grad_norm(&l, 1.0f, 0, control, fake + 4, 256, nullptr), MUON_ERR_WORKSPACE, "workspace alignment");
  expect(muon_grad_norm(nullptr, 1.0f, 0, control, fake, 256, nullptr), MUON_ERR_INVALID_VALUE, "list");
  for (int k = 0; k < 5; ++k) {
    muon_grad_list_t b = l;
    if (k == 0) b.count = 0;
    if (k == 1) b.total_chunks = -1;
    if (k == 2) b.total_chunks = int64_t{1} << 31;
    if (k == 3) b.grads = nullptr;
    if (k == 4) b.chunk_tensor = nullptr;
    expect(muon_grad_norm(&b, 1.0f, 0, control, fake, 1 << 20, nullptr), MUON_ERR_INVALID_VALUE, "list field");
  }
  if (muon_grad_norm_workspace(-1) != 0 || muon_grad_norm_workspace(int64_t{1} << 31) != 0) std::abort();

  muon_param_list_t p{3, 5, reinterpret_cast<const muon_param_t*>(fake), reinterpret_cast<const int32_t*>(fake + 64)};
  const muon_adamw_hyper_t h{1e-3, 0.9, 0.999, 1e-8, 7u, 0u};
  if (optim_stub_launches() != before) std::abort();
  for (int64_t step : {int64_t{1}, int64_t{1000}, int64_t{1} << 40})
    expect(muon_adamw_multi(&p, &h, step, nullptr, nullptr), MUON_OK, "adamw");
  expect(muon_adamw_multi(&p, &h, 0, control, nullptr), MUON_OK, "adamw with control");
  expect(muon_adamw_multi(&p, &h, 0, nullptr, nullptr), MUON_ERR_INVALID_VALUE, "step 0");
  expect(muon_adamw_multi(&p, nullptr, 1, nullptr, nullptr), MUON_ERR_INVALID_VALUE, "hyper");
  expect(muon_adamw_multi(nullptr, &h, 1, nullptr, nullptr), MUON_ERR_INVALID_VALUE, "list");
  expect(muon_adamw_multi(&p, &h, 1, reinterpret_cast<muon_step_control_t*>(fake + 4), nullptr), MUON_ERR_INVALID_VALUE, "control alignment");
  for (int k = 0; k < 9; ++k) {
    muon_adamw_hyper_t b = h;
    if (k == 0) b.beta1 = 1.0;
    if (k == 1) b.beta2 = -0.1;
    if (k == 2) b.beta1 = nan;
    if (k == 3) b.eps = -1e-9;
    if (k == 4) b.eps = inf;
    if (k == 5) b.lr = nan;
    if (k == 6) b.lr = inf;
    if (k == 7) b.reserved = 1;
    if (k == 8) b.beta2 = 1.0;
    expect(muon_adamw_multi(&p, &b, 1, nullptr, nullptr), MUON_ERR_INVALID_VALUE, "hyperparameter");
  }
  muon_adamw_hyper_t zero = h;
  zero.beta1 = zero.beta2 = 0.0;
  expect(muon_adamw_multi(&p, &zero, 1, control, nullptr), MUON_OK, "betas 0");
  muon_param_list_t empty{1, 0, reinterpret_cast<const muon_param_t*>(fake), nullptr};
  expect(muon_adamw_multi(&empty, &h, 1, nullptr, nullptr), MUON_OK, "no chunks");

  // Muon under a control block: the checks of the plain calls, and the block's own
  muon_batch_t g{nullptr, fake, 64 * 96, 2, 64, 96, 96, MUON_BF16, 0}, m = g, w = g;
  m.dtype = MUON_F32;
  const int64_t count = 2, rows = 64, cols = 96;
  const size_t need = muon_packed_grouped_workspace(1, &count, &rows, &cols, MUON_BF16);
  stub_set_workspace(fake, need);
  float* ss[1] = {reinterpret_cast<float*>(fake)};
  expect(muon_momentum_packed_grouped_controlled(1, &g, &m, ss, 0.9f, 1, MUON_BF16, fake, need, control, nullptr), MUON_OK, "momentum");
  expect(muon_momentum_packed_grouped_controlled(1, &g, &m, ss, 0.9f, 1, MUON_BF16, fake, need, nullptr, nullptr), MUON_ERR_INVALID_VALUE, "momentum control");
  expect(muon_momentum_packed_grouped_controlled(1, &g, &m, ss, 1.0f, 1, MUON_BF16, fake, need, control, nullptr), MUON_ERR_INVALID_VALUE, "momentum beta");
  expect(muon_momentum_packed_grouped_controlled(1, &g, &m, ss, 0.9f, 1, MUON_BF16, fake, need - 1, control, nullptr), MUON_ERR_WORKSPACE, "momentum workspace");
  expect(muon_apply_grouped_controlled(1, &w, &g, 0.1f, 0.1f, MUON_SCALE_MATCH_RMS, 0.2f, control, nullptr), MUON_OK, "apply");
  expect(muon_apply_grouped_controlled(1, &w, &g, 0.1f, 0.1f, MUON_SCALE_MATCH_RMS, 0.2f, nullptr, nullptr), MUON_ERR_INVALID_VALUE, "apply control");
  expect(muon_apply_grouped_controlled(1, &w, &g, nan, 0.1f, MUON_SCALE_MATCH_RMS, 0.2f, control, nullptr), MUON_ERR_INVALID_VALUE, "apply lr");
  std::printf("ok: %ld checks, %ld launches\n", checks, optim_stub_launches());
  return 0;
}
