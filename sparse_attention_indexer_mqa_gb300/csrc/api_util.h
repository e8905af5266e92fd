// api_util.h -- small helpers of the extern "C" entry points.
#pragma once

#include <nvtx3/nvToolsExt.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/idx.h"

namespace {

// One NVTX range per entry point call (visible in Nsight timelines; near free otherwise).
struct Range {
    explicit Range(const char* name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
    Range(const Range&) = delete;
    Range& operator=(const Range&) = delete;
};

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? IDX_OK : IDX_ECUDA; }

}  // namespace
