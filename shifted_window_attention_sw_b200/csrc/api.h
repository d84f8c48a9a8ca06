// What the translation units that hold C entry points share (vswin_api.cu
// defines the functions): error reporting, per-call context, scratch.
#pragma once

#include <cstddef>

#include <nvtx3/nvToolsExt.h>

#include "../../include/vswin.h"
#include "internal.h"

namespace vswin {

// Records a description for vswin_last_error and returns `status`.
int fail(int status, const char* fmt, ...);
int fail_cuda(cudaError_t e, const char* what);

// Error word and wait limit of a call; takes a pending injected CUDA failure.
int make_ctx(KernelCtx* ctx);

// Stream-ordered scratch from the library's pool (release with cudaFreeAsync).
int scratch_alloc(void** p, size_t bytes, cudaStream_t st);

bool aligned(const void* p, size_t a);
bool overlap(const void* a, size_t na, const void* b, size_t nb);

// Names every entry call on the NVTX timeline (a no-op unless a tool listens).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace vswin
