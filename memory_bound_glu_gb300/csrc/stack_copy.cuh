// stack_copy.cuh -- inline-PTX wrappers for copies out of stacks of matrices (an expert's
// weights, an adapter's) and for what is asked for ahead of them.
#pragma once
#include "ptx.cuh"

namespace mbglu {

// tma_load_2d for a box of a stack of matrices (z: the matrix).
__device__ __forceinline__ void tma_load_3d(void *dst, const TensorMap *map, int x, int y, int z, uint64_t *bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

// Asks for a descriptor ahead of the copies that use it.
__device__ __forceinline__ void prefetch_tensor_map(const TensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Asks for `bytes` (a multiple of 16, the address 16-byte aligned) to be brought into L2.
__device__ __forceinline__ void bulk_prefetch_l2(const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

}  // namespace mbglu
