// lora_shrink_tc.cuh -- p = scale[a] x A[a]^T for many rows, on tcgen05.
//
// A cluster takes 128 rows, its blocks a range of the inner dimension each.  The rows are
// the MMA's M side; the columns are the A of up to kShrinkTcGroup adapters among the rows, both
// projections' one behind the other (256 columns at most), so that a tile with a border between
// two requests reads x once.  The block keeps of each adapter's columns the rows that use it,
// as a partial sum in global memory (which stays in L2); a row has one adapter, so no row is
// written twice, and one cluster barrier at the end lets the blocks add up 128 / split rows
// each, in order.
//
// What bounds it is x's way in: 4096 x 2560 are 21 MB.  Rows of one request lie together, so
// mostly there is one adapter, or two; a chunk of many short requests takes
// lora_shrink_kernel.
#pragma once
#include "lora_shrink.cuh"
#include "tc_pair.cuh"

namespace mbglu {

constexpr int kShrinkTcThreads = 192;
constexpr int kShrinkTcRows = 128;
constexpr uint32_t kShrinkTcX = kShrinkTcRows * 128;      // a chunk of 64 columns of x
constexpr int kShrinkTcMaxStages = 8;
constexpr uint32_t kShrinkTcHeader = 2048;                // barriers; the rows' scales and adapters

struct ShrinkTcMaps {
    TensorMap x;             // [M][K], boxes of 64 x 128
    TensorMap a[2];          // [adapters][R][K], 64 x R
};

struct ShrinkTcParams {
    LoraParams l;
    float *part;             // [split - 1][M][sides R]: a block's partial sums; the first block's lie in p
    int split, stages, nchunk;
    int group;               // adapters at a time
};

constexpr int kShrinkTcGroup = 4;
__host__ __device__ constexpr int shrink_tc_group(int width) { return 256 / width < kShrinkTcGroup ? 256 / width : kShrinkTcGroup; }
__host__ __device__ constexpr uint32_t shrink_tc_stage(int width)
{
    return kShrinkTcX + static_cast<uint32_t>((shrink_tc_group(width) * width + 15) / 16 * 16) * 128u;
}

// The adapters among 128 rows, each once; a warp walks them.
struct LoraDistinct {
    int id[4];
    uint32_t left[4];
    __device__ LoraDistinct(const LoraParams &p, int64_t m0)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            id[i] = lora_adapter(p, m0 + i * 32 + (threadIdx.x & 31));
            left[i] = __ballot_sync(0xffffffffu, id[i] >= 0);
        }
    }
    // up to `group` of them; how many
    __device__ int next(int (&a)[kShrinkTcGroup], int group)
    {
        int n = 0;
#pragma unroll
        for (int i = 0; i < kShrinkTcGroup; ++i) {
            a[i] = -1;
            if (n == i && i < group && one(a[i])) ++n;
        }
        return n;
    }
    __device__ bool one(int &a)
    {
        a = -1;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const int v = __shfl_sync(0xffffffffu, id[i], left[i] ? __ffs(left[i]) - 1 : 0);
            if (left[i]) a = v;
        }
        if (a < 0) return false;
#pragma unroll
        for (int i = 0; i < 4; ++i) left[i] &= ~__ballot_sync(0xffffffffu, id[i] == a);
        return true;
    }
};

// grid: (split, tiles of 128 rows), clusters of split
template <int SIDES>
__global__ void __launch_bounds__(kShrinkTcThreads, 1) lora_shrink_tc_kernel(const ShrinkTcParams p, const __grid_constant__ ShrinkTcMaps maps)
{
    extern __shared__ unsigned char shrink_raw[];
    unsigned char *base = shrink_raw + ((1024u - (smem_addr(shrink_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(base), *empty = full + kShrinkTcMaxStages;
    uint64_t *acc_full = empty + kShrinkTcMaxStages, *acc_empty = acc_full + 2, *done = acc_empty + 2;
    uint32_t *slot = reinterpret_cast<uint32_t *>(done + 1);
    float *scales = reinterpret_cast<float *>(base + 512);   // of the rows; 0 where none is used
    int *ids = reinterpret_cast<int *>(base + 1024);
    unsigned char *ring = base + kShrinkTcHeader;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int R = p.l.R, width = SIDES * R, rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const uint32_t stage = shrink_tc_stage(width);
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kShrinkTcRows;
    const int c0 = static_cast<int>(static_cast<int64_t>(p.nchunk) * rank / p.split), c1 = static_cast<int>(static_cast<int64_t>(p.nchunk) * (rank + 1) / p.split);

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    tc_fence_after();
    const uint32_t tmem = *slot;
    bool ok = true;
    grid_dependency_wait();
    grid_launch_dependents();   // behind the wait: lora_pair_kernel reads x then (LoraPairParams::early)

    if (warp == 0) {
        LoraDistinct adapters(p.l, m0);
        int st = 0, issued = 0, a[kShrinkTcGroup], n;
        uint32_t phase = 1;
        while (ok && (n = adapters.next(a, p.group)) > 0) {
            for (int c = c0; c < c1; ++c) {
                if (!pair_wait(&empty[st], phase, kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    unsigned char *d = ring + st * stage;
                    mbar_arrive_expect_tx(&full[st], kShrinkTcX + static_cast<uint32_t>(n * width) * 128u);
                    const uint64_t policy = l2_policy_evict_last();   // the shared product reads x again
                    tma_load_2d(d, &maps.x, c * 64, static_cast<int>(m0), &full[st], policy);
#pragma unroll
                    for (int j = 0; j < kShrinkTcGroup; ++j)
#pragma unroll
                        for (int i = 0; i < SIDES; ++i)
                            if (j < n) tma_load_3d(d + kShrinkTcX + (j * width + i * R) * 128, &maps.a[i], c * 64, 0, a[j], &full[st], policy);
                }
                __syncwarp();
                issued += issued < p.stages;
                if (++st == p.stages) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        for (int i = 0; i < issued; ++i) {   // no copy may be in flight when the block leaves
            int at = st - issued + i;
            const uint32_t ph = at < 0 ? phase : phase ^ 1;
            if (at < 0) at += p.stages;
            if (!pair_wait(&full[at], ph, kWaitLimitNs)) ok = false;
        }
    } else if (warp == 1) {
        LoraDistinct adapters(p.l, m0);
        int st = 0, a[kShrinkTcGroup], n;
        uint32_t phase = 0, buf = 0, acc_phase = 1;
        while (ok && (n = adapters.next(a, p.group)) > 0) {
            const uint32_t idesc = tc_idesc_bf16(kShrinkTcRows, 16) + (static_cast<uint32_t>((n * width + 15) / 16 * 16 - 16) >> 3 << 17);
            if (!pair_wait(&acc_empty[buf], acc_phase, kWaitLimitNs)) {
                ok = false;
                break;
            }
            for (int c = c0; c < c1; ++c) {
                if (!pair_wait(&full[st], phase, kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t x = smem_desc_sw128(ring + st * stage), w = smem_desc_sw128(ring + st * stage + kShrinkTcX);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) tc_mma_bf16(tmem + buf * 256u, x + 2 * kk, w + 2 * kk, idesc, c > c0 || kk > 0);
                    tc_commit(&empty[st]);
                }
                __syncwarp();
                if (++st == p.stages) {
                    st = 0;
                    phase ^= 1;
                }
            }
            if (elect_one() && ok) tc_commit(&acc_full[buf]);
            __syncwarp();
            buf ^= 1;
            if (buf == 0) acc_phase ^= 1;
        }
        if (elect_one()) tc_commit(done);
        __syncwarp();
        if (!pair_wait(done, 0, kWaitLimitNs)) ok = false;
    } else {
        LoraDistinct adapters(p.l, m0);
        const int q = warp & 3, row = q * 32 + lane;
        const int mine = lora_adapter(p.l, m0 + row);
        ids[row] = mine;
        scales[row] = mine >= 0 ? (p.l.scale ? p.l.scale[mine] : 1.0f) : 0.0f;
        if (p.l.blocks && rank == 0) {   // the table: a warp has 32 rows
            const uint32_t in = __ballot_sync(0xffffffffu, m0 + row < p.l.M);
            const int first = __shfl_sync(0xffffffffu, mine, 0);
            const uint32_t same = __ballot_sync(0xffffffffu, mine == first);
            if (lane == 0 && in) p.l.blocks[m0 / kLoraBlock + q] = (in & ~same) ? kMixed : first;
        }
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        float *dst = (rank == 0 ? p.l.p : p.part + static_cast<int64_t>(rank - 1) * p.l.M * width) + (m0 + row) * width;
        uint32_t buf = 0, acc_phase = 0;
        int a[kShrinkTcGroup];
        while (ok && adapters.next(a, p.group) > 0) {
            if (!__all_sync(0xffffffffu, pair_wait(&acc_full[buf], acc_phase, kWaitLimitNs))) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < kShrinkTcGroup; ++j) {
                if (a[j] < 0 || !__any_sync(0xffffffffu, mine == a[j])) continue;   // the whole warp
                for (int c = 0; c < width; c += 16) {
                    float v[16];
                    __syncwarp();
                    tmem_ld16(lanes + buf * 256u + static_cast<uint32_t>(j * width + c), v);
                    if (mine == a[j]) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (c + 4 * i < width) __stcg(reinterpret_cast<float4 *>(dst + c + 4 * i), make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
            buf ^= 1;
            if (buf == 0) acc_phase ^= 1;
        }
    }
    if (!ok) atomicExch(&g_dense_error, kErrTimeout);
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    if (p.split > 1) cluster_sync();   // the partial sums are there
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    // this block's rows of the tile; a thread has four columns of two rows at a time, whose parts
    // are on the way together
    const int rows = kShrinkTcRows / p.split, quads = width / 4;
    const int64_t stride = p.l.M * static_cast<int64_t>(width);
    for (int e0 = threadIdx.x; e0 < rows * quads; e0 += 2 * kShrinkTcThreads) {
        float4 v[2];
        int row[2];
        int64_t at[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = e0 + h * kShrinkTcThreads, r = rank * rows + e / quads;
            row[h] = e < rows * quads && ids[r] >= 0 ? r : -1;
            at[h] = (m0 + r) * width + e % quads * 4;
            v[h] = make_float4(0, 0, 0, 0);
        }
#pragma unroll 8
        for (int i = 0; i < p.split; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // of p a thread reads what it writes itself below
                const float *from = i == 0 ? p.l.p : p.part + (i - 1) * stride;
                const float4 x = row[h] >= 0 ? __ldcg(reinterpret_cast<const float4 *>(from + at[h])) : make_float4(0, 0, 0, 0);
                v[h] = make_float4(v[h].x + x.x, v[h].y + x.y, v[h].z + x.z, v[h].w + x.w);
            }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (row[h] < 0) continue;
            const float s = scales[row[h]];
            const float4 w = make_float4(v[h].x * s, v[h].y * s, v[h].z * s, v[h].w * s);
            *reinterpret_cast<float4 *>(p.l.p + at[h]) = w;
            uint2 hi, lo;
            split_bf16x2(w.x, w.y, hi.x, lo.x);
            split_bf16x2(w.z, w.w, hi.y, lo.y);
            *reinterpret_cast<uint2 *>(p.l.terms + at[h]) = hi;
            *reinterpret_cast<uint2 *>(p.l.terms + at[h] + stride) = lo;
        }
    }
}

}  // namespace mbglu
