// stack_maps.cu -- descriptors of stacks of matrices (experts' weights, adapters) for
// tensor copies.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "api_internal.h"

namespace {

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime; null if
// unavailable.
PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
    }();
    return fn;
}

}  // namespace

namespace mbglu_host {

bool encode_stack_map(mbglu::TensorMap *out, const void *base, int64_t stride, int64_t ld, int count, int rows, int cols, int box_cols,
                      int box_rows)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
    if (!fn) return false;
    CUtensorMap m;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(count)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(count > 1 ? stride : rows * ld) * 2};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1u};
    const cuuint32_t elem_strides[3] = {1u, 1u, 1u};
    if (fn(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    std::memcpy(out, &m, sizeof m);
    return true;
}

}  // namespace mbglu_host
