// zk_capi.h -- small host helpers shared by the C entry points.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "zero.h"

namespace zk {

// An NVTX range named after the entry point around each call that launches
// work, so that profilers (nsys, ncu --nvtx) group its kernels; with no tool
// attached it costs a branch.
struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};
#define ZK_CALL_RANGE() const zk::CallRange zk_call_range_(__func__)

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline zero_status from_cuda(cudaError_t e) { return e == cudaSuccess ? ZERO_OK : ZERO_ERR_CUDA; }

inline zero_status check_dev(const void* ptr, uintptr_t align = 16)
{
    if (ptr == nullptr) return ZERO_ERR_INVALID_ARG;
    return aligned(ptr, align) ? ZERO_OK : ZERO_ERR_MISALIGNED;
}

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

}  // namespace zk
