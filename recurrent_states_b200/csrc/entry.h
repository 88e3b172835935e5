// Host helpers of the entry points that check their arguments beside their
// kernels: alignment, status codes and the strides of strided operands.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/taylor_attn.h"

namespace ta {
namespace entry {

inline bool aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline int status(cudaError_t e) {
    if (e == cudaSuccess) return TAYLOR_OK;
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? TAYLOR_ERR_OUT_OF_MEMORY : TAYLOR_ERR_CUDA;
}

// Of the current device; asked for once on each.
inline int num_sms() {
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 148;
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

// Lets a kernel take up to `bytes` of dynamic shared memory, asked for once on
// each device; `done` is the kernel's own record of where that was.
template <typename K>
inline cudaError_t allow_smem(K* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Whether an output of these sizes and strides (elements) has every element
// at an address of its own: the sizes nest in the order of the strides.
// The innermost run of `row` elements is contiguous.
template <int K>
inline bool disjoint(const int64_t (&size)[K], const int64_t (&stride)[K], int64_t row) {
    int order[K];
    for (int i = 0; i < K; ++i) order[i] = i;
    for (int i = 1; i < K; ++i)
        for (int j = i; j > 0 && stride[order[j]] < stride[order[j - 1]]; --j) {
            const int t = order[j];
            order[j] = order[j - 1];
            order[j - 1] = t;
        }
    int64_t extent = row;
    for (int i = 0; i < K; ++i) {
        const int64_t n = size[order[i]], s = stride[order[i]];
        if (n <= 1) continue;
        if (s < extent) return false;
        extent = s * (n - 1) + extent;
    }
    return true;
}

}  // namespace entry
}  // namespace ta
