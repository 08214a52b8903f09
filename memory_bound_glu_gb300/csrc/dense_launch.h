// dense_launch.h -- launches of the gated block's kernels beyond the decode
// batch.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "api_internal.h"

namespace mbglu_host {

// The largest size these entry points take: the kernels' 32-bit indexes run up to
// the end of the last tile.
constexpr int kMostSize = INT32_MAX - 511;
inline bool bad_sizes(int a, int b, int c = 0) { return std::min({a, b, c}) < 0 || std::max({a, b, c}) > kMostSize; }

// An operand that tensor copies take: 16-byte aligned rows.
inline bool copyable(const void *p, int64_t ld, int elem) { return aligned(p, 16) && ld * elem % 16 == 0; }

// 2 when every row of elem-byte elements starts on 32 bytes, 1 on 16, else 0
inline int row_align(const void *p, int64_t ld, int elem)
{
    return aligned(p, 32) && ld * elem % 32 == 0 ? 2 : aligned(p, 16) && ld * elem % 16 == 0 ? 1 : 0;
}

// Places in workspaces are multiples of kAlign bytes.
constexpr int64_t kAlign = 256;
inline int64_t padded(int64_t bytes) { return (bytes + kAlign - 1) / kAlign * kAlign; }

// bytes from the first element of 16-bit [count][rows][cols] to the end of its last
inline int64_t extent3(int64_t count, int64_t rows, int64_t cols, int64_t stride, int64_t ld)
{
    return count <= 0 || rows <= 0 || cols <= 0 ? 0 : (count - 1) * stride * 2 + extent(rows, cols, ld, 2);
}

// The current device's SM count, after `setup` (attributes of the unit's
// kernels) has run once on it.
struct DeviceTable {
    std::mutex mu;
    int sms[64] = {};
    mbglu_status get(int *sm_count, cudaError_t (*setup)())
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return cuda_fail(e);
        if (dev < 0 || dev >= 64) return cuda_fail(cudaErrorInvalidDevice);
        std::lock_guard<std::mutex> lk(mu);
        if (sms[dev] == 0) {
            int n = 0;
            if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return cuda_fail(e);
            if ((e = setup()) != cudaSuccess) return cuda_fail(e);
            sms[dev] = n;
        }
        *sm_count = sms[dev];
        return MBGLU_OK;
    }
};

inline mbglu_status launched(cudaError_t e) { return e == cudaSuccess ? MBGLU_OK : cuda_fail(e); }

// Launch configuration with the process's launch policy: under PDL a kernel may
// be scheduled while its predecessor drains.  Every kernel launched here waits for the
// predecessor before it touches global memory, but for two:
//   fp8_tall_kernel and lora_pair_kernel copy their first weights before the wait under the
//     prefetch policy, so a kernel of the library that writes weights (quant_weight_kernel)
//     neither releases its dependents early nor leaves its stores to be performed later;
//   lora_pair_kernel behind a kernel that forms p reads the call's operands and releases its own
//     dependents while that one runs, which is sound because that one has waited for its
//     predecessor before it releases: lora_shrink_kernel and lora_shrink_tc_kernel keep
//     the release behind the wait.
struct Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    Launch(const Launch &) = delete;   // cfg points at attr
    Launch(dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster = 1)
    {
        cfg.gridDim = grid;
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        unsigned n = 0;
        if (launch_policy() != MBGLU_POLICY_SERIAL) {
            attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[n].val.programmaticStreamSerializationAllowed = 1;
            ++n;
        }
        if (cluster > 1) {
            attr[n].id = cudaLaunchAttributeClusterDimension;
            attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
            attr[n].val.clusterDim.y = 1;
            attr[n].val.clusterDim.z = 1;
            ++n;
        }
        cfg.attrs = attr;
        cfg.numAttrs = n;
    }
};

}  // namespace mbglu_host
