// api_internal.h -- what the library's translation units share on the host:
// status bookkeeping, pointer checks and tensor-map encoding (defined in
// mbglu_api.cu), and each unit's device error word.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "mbglu.h"
#include "ptx.cuh"

namespace mbglu_host {

// mbglu_last_variant codes of the operators outside mbglu_api.cu
enum DenseVariant {
    kPairGemm = 11,      // glu_gemm on a CTA-pair tcgen05 kernel
    kGemmGeneric = 12,   // glu_gemm on the kernel for any alignment
    kGemmBackward = 13,  // glu_gemm_backward
    kNormFp8 = 14,       // add_rmsnorm_fp8
    kFp8Pair = 15,       // an e4m3 product on the CTA-pair tcgen05 kernel
    kFp8Tall = 16,       // an e4m3 product of few rows
    kFp8Generic = 17,    // an e4m3 product on the kernel for any alignment
    kQuantWeight = 18    // quantize_weight_fp8
};

mbglu_status cuda_fail(cudaError_t e);   // records e for mbglu_last_cuda_error
void set_last_variant(int v);
void set_last_backward_path(int v);
int launch_policy();

// [rows][cols] of elem_bytes-wide elements (1 or 2), row stride ld elements,
// in 128-byte swizzled boxes; false where the driver takes no such map.
bool encode_tile_map(mbglu::TensorMap *out, const void *base, int64_t ld, int rows, int cols, int box_cols,
                     int box_rows, int elem_bytes);

// mbglu_block_plan's answer for the e4m3 products
void fp8_block_plan(bool dual, int M, int N, int K, int *plan);

// Reads and clears the unit's device error word; the device is idle.
cudaError_t take_gemm_error(int *w);
cudaError_t take_fp8_error(int *w);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// [p, p + bytes) and [q, q + bytes_q) intersect
inline bool overlaps(const void *p, int64_t bytes, const void *q, int64_t bytes_q)
{
    if (bytes <= 0 || bytes_q <= 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + static_cast<uintptr_t>(bytes_q) && b < a + static_cast<uintptr_t>(bytes);
}

// bytes from a matrix's first element to the end of its last
inline int64_t extent(int64_t rows, int64_t cols, int64_t ld, int64_t elem_bytes)
{
    return rows <= 0 || cols <= 0 ? 0 : ((rows - 1) * ld + cols) * elem_bytes;
}

inline int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

}  // namespace mbglu_host
