// api_util.h -- what the C-ABI sources share: argument checks and limits.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>
#include <set>
#include <utility>

#include "bimamba.h"

namespace {

constexpr int kMaxBatch = 65535;
constexpr int kSms = 148;
constexpr long long kWaitCycles = 4000000000LL;    // ~2 s at 1.965 GHz
constexpr long long kStarveWaitCycles = 200000LL;  // ~0.1 ms: the starved test gives up fast

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t elem_size(bimamba_dtype_t t) { return t == BIMAMBA_F32 ? 4 : 2; }

inline bool dtype_ok(int t) { return t == BIMAMBA_F32 || t == BIMAMBA_BF16; }

// Raise the dynamic shared-memory limit of a kernel once per device.
inline int ensure_smem(const void* fn, size_t bytes) {
    if (bytes <= 48 * 1024) return BIMAMBA_OK;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BIMAMBA_ERR_CUDA;
    static std::mutex mu;
    static std::set<std::pair<const void*, int>> done;
    std::lock_guard<std::mutex> lock(mu);
    if (done.count({fn, dev})) return BIMAMBA_OK;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return BIMAMBA_ERR_CUDA;
    done.insert({fn, dev});
    return BIMAMBA_OK;
}

inline int launch_status() { return cudaGetLastError() == cudaSuccess ? BIMAMBA_OK : BIMAMBA_ERR_CUDA; }

}  // namespace

namespace bimamba {

// glr_api.cu: the error word of the gated linear recurrence's kernels on the
// current device (read, and cleared if reset != 0).
int glr_error_word(int reset, unsigned int* word);

}  // namespace bimamba
