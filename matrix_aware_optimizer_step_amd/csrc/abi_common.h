// Status helpers shared by the C-ABI layer's source files (defined in
// abi.cpp, beside the thread-local error text that muon_last_error returns).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/muon355.h"

namespace muon {

// Records the error text and returns `st`.
muon_status_t fail(muon_status_t st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the error text.
muon_status_t ok();
muon_status_t launch_status(hipError_t e, const char* what);
// The end of an entry point: ok(), after a wait with MUON355_DEBUG_SYNC=1.
muon_status_t done(hipStream_t s, const char* what);

}  // namespace muon
