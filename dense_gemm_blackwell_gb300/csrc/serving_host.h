// serving_host.h -- host helpers of the serving operators (internal).
#pragma once

#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "gemm.h"

namespace dgb {

// Records the error for gemm_last_cuda_error.
gemm_status_t status_of(cudaError_t e);

// Zeroes device memory before it returns, whatever the legacy stream is busy with: cudaMemset waits in that stream's queue
// and returns at once, and non-blocking streams do not wait for it.
cudaError_t clear_now(void* mem, size_t bytes);

struct DeviceFacts {
    int device = 0;
    int sms = 0;
    int smem_optin = 0;    // shared memory a block may opt in to
};

// The current device's facts; GEMM_ERR_NO_DEVICE unless it is compute capability 10.3.
gemm_status_t device_facts(DeviceFacts* out);

// A plan's workspace lies on the device it was made on: GEMM_ERR_INVALID_ARG where another one is current.
inline gemm_status_t check_device(int made_on) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return status_of(e);
    return dev == made_on ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

inline bool all_aligned(uintptr_t bytes, std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) % bytes != 0) return false;
    return true;
}

inline bool all_multiples(int64_t of, std::initializer_list<int64_t> values) {
    for (int64_t v : values)
        if (v % of != 0) return false;
    return true;
}

// Launch with programmatic stream serialization: the kernel's set-up overlaps the previous kernel of the stream; it
// reads and writes memory only after griddep_wait().
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace dgb
