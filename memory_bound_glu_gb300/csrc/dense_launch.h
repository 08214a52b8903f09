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
// predecessor before it touches global memory, but for fp8_tall_kernel: under the
// prefetch policy it copies its first weights before the wait, so a kernel of the
// library that writes weights (quant_weight_kernel) neither releases its dependents
// early nor leaves its stores to be performed later.
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
