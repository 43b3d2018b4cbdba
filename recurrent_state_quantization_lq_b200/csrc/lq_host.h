// Host helpers that the files of C-ABI entry points share (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include <string>

#include "lq.h"

namespace lq {

// Record the calling thread's error text (lq_last_error_string) and return the status.
lq_status fail(lq_status code, const std::string &why);

inline lq_status cuda_fail(cudaError_t e, const char *what) {
    return fail(LQ_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// An NVTX range around a stream-ordered call, for timeline tools (nsys, ncu);
// nearly free when no tool is attached.
struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
    Range(const Range &) = delete;
    Range &operator=(const Range &) = delete;
};

}  // namespace lq
