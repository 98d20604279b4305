// Host stand-ins for the launchers of the many-tensor operators (see
// stub_launchers.cpp): nothing is enqueued, every launch is checked.
#include <cstdio>
#include <cstdlib>

#include "muon_internal.h"

namespace {
const char* g_lo = nullptr;
size_t g_bytes = 0;
long g_launches = 0;
[[noreturn]] void die(const char* what) {
  std::fprintf(stderr, "launch check failed: %s\n", what);
  std::abort();
}
}  // namespace

extern "C" void optim_stub_workspace(const void* base, size_t bytes) {
  g_lo = static_cast<const char*>(base);
  g_bytes = bytes;
}
extern "C" long optim_stub_launches() { return g_launches; }

namespace muon {

hipError_t launch_grad_norm(const GradNormArgs& a, hipStream_t) {
  ++g_launches;
  if (a.count < 1 || a.total_chunks < 0 || a.blocks < 0 || a.blocks > kGradMaxBlocks) die("norm sizes");
  if (a.blocks > a.total_chunks || (a.total_chunks > 0 && a.blocks == 0)) die("norm grid");
  const char* p = reinterpret_cast<const char*>(a.partials);
  if (p < g_lo || static_cast<size_t>(p - g_lo) + static_cast<size_t>(a.blocks) * 8 > g_bytes) die("norm partials");
  if (!a.control || !(a.max_norm > 0.0f)) die("norm arguments");
  return hipSuccess;
}

hipError_t launch_adamw_multi(const AdamWMultiArgs& a, int64_t total_chunks, hipStream_t) {
  ++g_launches;
  if (a.count < 1 || total_chunks < 0 || !a.params) die("adamw multi sizes");
  if (a.b1 + a.omb1 < 0.999999f || a.b1 + a.omb1 > 1.000001f) die("beta1 and its complement");
  if (a.b2 + a.omb2 < 0.999999f || a.b2 + a.omb2 > 1.000001f) die("beta2 and its complement");
  if (!a.control && (a.step < 1 || !(a.c1 >= 1.0f) || !(a.c2 >= 1.0f))) die("bias corrections");
  return hipSuccess;
}

}  // namespace muon
