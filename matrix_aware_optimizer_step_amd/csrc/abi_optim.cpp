// C-ABI layer of the many-tensor operators: the gradient norm with its step
// control block, and AdamW with 32-bit or 8-bit moments.  Contracts are in
// include/muon355.h.

#include "../../include/muon355.h"

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "abi_common.h"
#include "muon_internal.h"

namespace {

using namespace muon;

constexpr int64_t kMaxChunks = (int64_t{1} << 31) - 1;
// AdamW takes a workgroup of 256 for a chunk, and a launch has fewer than 2^32 work-items.
constexpr int64_t kMaxParamChunks = (int64_t{1} << 24) - 1;

static_assert(sizeof(StepControl) == sizeof(muon_step_control_t) && sizeof(StepControl) == 64, "control block");
static_assert(offsetof(StepControl, skip) == offsetof(muon_step_control_t, skip) &&
                  offsetof(StepControl, step) == offsetof(muon_step_control_t, step) &&
                  offsetof(StepControl, skipped) == offsetof(muon_step_control_t, skipped),
              "control block");
static_assert(sizeof(GradTensor) == sizeof(muon_grad_t) && offsetof(GradTensor, dtype) == offsetof(muon_grad_t, dtype),
              "gradient descriptor");
static_assert(sizeof(ParamTensor) == sizeof(muon_param_t) &&
                  offsetof(ParamTensor, numel) == offsetof(muon_param_t, numel) &&
                  offsetof(ParamTensor, weight_decay) == offsetof(muon_param_t, weight_decay) &&
                  offsetof(ParamTensor, state_bits) == offsetof(muon_param_t, state_bits),
              "parameter descriptor");
static_assert(kGradChunk == MUON_GRAD_CHUNK && kParamChunk == MUON_PARAM_CHUNK && kStateBlock == MUON_STATE_BLOCK,
              "chunk and block sizes");

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int32_t norm_blocks(int64_t total_chunks) {
  return static_cast<int32_t>(total_chunks < kGradMaxBlocks ? total_chunks : kGradMaxBlocks);
}

muon_status_t check_list(int64_t count, int64_t total_chunks, const void* tensors, const void* chunk_tensor) {
  if (count < 1 || count > kMaxChunks)
    return fail(MUON_ERR_INVALID_VALUE, "count %lld outside [1, 2^31-1]", (long long)count);
  if (total_chunks < 0 || total_chunks > kMaxChunks)
    return fail(MUON_ERR_INVALID_VALUE, "total_chunks %lld outside [0, 2^31-1]", (long long)total_chunks);
  if (!tensors || (total_chunks > 0 && !chunk_tensor))
    return fail(MUON_ERR_INVALID_VALUE, "a device array of the list is NULL");
  return MUON_OK;
}

}  // namespace

extern "C" {

size_t muon_grad_norm_workspace(int64_t total_chunks) {
  if (total_chunks < 0 || total_chunks > kMaxChunks) return 0;
  const size_t bytes = static_cast<size_t>(norm_blocks(total_chunks)) * sizeof(double);
  return bytes < 256 ? 256 : bytes;
}

muon_status_t muon_grad_norm(const muon_grad_list_t* l, float max_norm, int flags, muon_step_control_t* control,
                             void* workspace, size_t ws_bytes, void* stream) {
  if (!l) return fail(MUON_ERR_INVALID_VALUE, "gradient list is NULL");
  const muon_status_t st = check_list(l->count, l->total_chunks, l->grads, l->chunk_tensor);
  if (st != MUON_OK) return st;
  if (!(max_norm > 0.0f)) return fail(MUON_ERR_INVALID_VALUE, "max_norm must be > 0");
  if ((flags & ~MUON_SKIP_NONFINITE) != 0) return fail(MUON_ERR_INVALID_VALUE, "unknown flags 0x%x", flags);
  if (!control || !aligned16(control))
    return fail(MUON_ERR_INVALID_VALUE, "control must be a 16-byte aligned device address");
  const size_t need = muon_grad_norm_workspace(l->total_chunks);
  if (!workspace || ws_bytes < need)
    return fail(MUON_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", ws_bytes, need);
  if (!aligned16(workspace)) return fail(MUON_ERR_WORKSPACE, "workspace must be 16-byte aligned");
  GradNormArgs a{};
  a.count = l->count;
  a.total_chunks = l->total_chunks;
  a.grads = reinterpret_cast<const GradTensor*>(l->grads);
  a.chunk_tensor = l->chunk_tensor;
  a.partials = static_cast<double*>(workspace);
  a.blocks = norm_blocks(l->total_chunks);
  a.skip_nonfinite = (flags & MUON_SKIP_NONFINITE) != 0;
  a.max_norm = max_norm;
  a.control = reinterpret_cast<StepControl*>(control);
  const hipError_t e = launch_grad_norm(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return launch_status(e, "grad norm");
  return done(static_cast<hipStream_t>(stream), "muon_grad_norm");
}

muon_status_t muon_adamw_multi(const muon_param_list_t* l, const muon_adamw_hyper_t* h, int64_t step,
                               const muon_step_control_t* control, void* stream) {
  if (!l) return fail(MUON_ERR_INVALID_VALUE, "parameter list is NULL");
  const muon_status_t st = check_list(l->count, l->total_chunks, l->params, l->chunk_tensor);
  if (st != MUON_OK) return st;
  if (l->total_chunks > kMaxParamChunks)
    return fail(MUON_ERR_INVALID_VALUE, "total_chunks %lld outside [0, 2^24-1]", (long long)l->total_chunks);
  if (!h) return fail(MUON_ERR_INVALID_VALUE, "hyperparameters are NULL");
  if (h->reserved != 0) return fail(MUON_ERR_INVALID_VALUE, "reserved field must be 0");
  if (!(h->beta1 >= 0.0 && h->beta1 < 1.0) || !(h->beta2 >= 0.0 && h->beta2 < 1.0))
    return fail(MUON_ERR_INVALID_VALUE, "betas must lie in [0, 1)");
  // the kernel's reciprocal flushes what is below fp32's normal range, on either side
  if (h->eps != 0.0 && !(h->eps >= 0x1p-126 && h->eps <= 0x1p125))
    return fail(MUON_ERR_INVALID_VALUE, "eps must be 0 or lie in [2^-126, 2^125]");
  if (!std::isfinite(h->lr)) return fail(MUON_ERR_INVALID_VALUE, "lr must be finite");
  if (!control && step < 1) return fail(MUON_ERR_INVALID_VALUE, "step %lld < 1", (long long)step);
  if (control && !aligned16(control))
    return fail(MUON_ERR_INVALID_VALUE, "control must be a 16-byte aligned device address");
  AdamWMultiArgs a{};
  a.count = l->count;
  a.params = reinterpret_cast<const ParamTensor*>(l->params);
  a.chunk_tensor = l->chunk_tensor;
  a.control = reinterpret_cast<const StepControl*>(control);
  a.lr = h->lr;
  a.log_b1 = std::log(h->beta1);
  a.log_b2 = std::log(h->beta2);
  a.step = step;
  a.b1 = static_cast<float>(h->beta1);
  a.omb1 = static_cast<float>(1.0 - h->beta1);
  a.b2 = static_cast<float>(h->beta2);
  a.omb2 = static_cast<float>(1.0 - h->beta2);
  a.eps = static_cast<float>(h->eps);
  if (!control) {
    a.c1 = static_cast<float>(1.0 / (1.0 - std::pow(h->beta1, static_cast<double>(step))));
    a.c2 = static_cast<float>(1.0 / (1.0 - std::pow(h->beta2, static_cast<double>(step))));
  }
  a.seed = h->seed;
  const hipError_t e = launch_adamw_multi(a, l->total_chunks, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return launch_status(e, "adamw multi");
  return done(static_cast<hipStream_t>(stream), "muon_adamw_multi");
}

}  // extern "C"
