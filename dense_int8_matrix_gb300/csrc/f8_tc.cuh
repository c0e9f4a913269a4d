// What the tensor-core kernels of the FP8 products share: the FP8 MMA, CTA
// pairs and clusters, groups, and the way a tile of D leaves registers.
#pragma once

#include <cuda.h>

#include "f8.cuh"
#include "ptx.cuh"

namespace gemm {

// Operands of the kernels: what is in F8Launch, as the device reads it.
struct F8Params {
    const float* a_scale;
    const float* b_scale;
    const int32_t* offsets;
    void* D;
    int* err;
    int64_t ldd, rows_a, rows_b;
    int m, n, groups, mode;
    int kb;               // blocks of 128 along K
    int nb;               // blocks of 128 along n
    int tiles_m, tiles_n; // tiles of one group's D (GEMM_GROUP_ROWS: tiles_n alone)
    int out_f32;
    int d_vec;            // rows of D are 16-byte aligned
    int pieces;           // row tiles that all groups together can have (GEMM_GROUP_ROWS)
};

// Instruction descriptor of tcgen05.mma kind::f8f6f4: D fp32 (bits 4-5 = 1),
// A and B format (bits 7-9, 10-12: 0 = e4m3, 1 = e5m2), both K-major, N >> 3
// in bits 17-22, M >> 4 in bits 24-28.
__host__ __device__ constexpr uint32_t idesc_f8(uint32_t a_type, uint32_t b_type, uint32_t M, uint32_t N) {
    return (1u << 4) | (a_type << 7) | (b_type << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

constexpr int kF8RowBytes = 128;   // one K block of a row: a 128-byte swizzle row
constexpr int kF8MmaK = 32;        // K of one FP8 MMA

// The groups' running sum in shared memory: pieces of `per` rows (ROWS: row
// tiles; K: blocks of 128 columns) of the groups before g, for g <= groups,
// never above `limit` (which a valid list does not reach past), so that any
// list of offsets gives tiles and blocks inside the operands.  One warp.
__device__ __forceinline__ void group_prefix(const int32_t* offsets, int groups, int rows, int per, int limit,
                                             int lane, int32_t* pre) {
    int before = 0;
    for (int g0 = 0; g0 < groups; g0 += 32) {
        int c = 0;
        if (g0 + lane < groups) {
            int lo, hi;
            group_rows(offsets, g0 + lane, rows, lo, hi);
            c = (hi - lo + per - 1) / per;
        }
        int sum = c;   // at most 32 * 2^30 / 128
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += t;
        }
        if (g0 + lane < groups) pre[g0 + lane] = min(before + sum - c, limit);
        before = min(before + __shfl_sync(0xffffffffu, sum, 31), limit);
    }
    if (lane == 0) pre[groups] = before;
}

// The group whose range of `pre` holds i (pre[0] = 0 <= i < pre[groups]).
__device__ __forceinline__ int group_of(const int32_t* pre, int groups, int i) {
    int lo = 0, hi = groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Four words of D to columns [c, c + 4 words) of a row; `out` is the row's
// address of column c, `left` the columns of D from c on.
template <bool F32>
__device__ __forceinline__ void store_d16(void* out, int left, bool vec, const uint4 v) {
    constexpr int N = F32 ? 4 : 8;
    if (vec && left >= N) {
        *static_cast<uint4*>(out) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (i >= left) break;
        if constexpr (F32)
            static_cast<uint32_t*>(out)[i] = w[i];
        else
            static_cast<uint16_t*>(out)[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// A warp's 32 rows (lane = row) x C columns of sums leave for D in slices of
// 128 bytes per row: through the warp's 4 KiB staging buffer (16-byte chunks
// swizzled by row & 7), so that eight lanes write one row's 128 bytes.  row0:
// D's row of lane 0; rows at or past row_end and columns at or past n are
// not written.
template <bool F32, int C>
__device__ __forceinline__ void store_rows(const float (&acc)[C], uint32_t stg, int lane, uint8_t* D, int64_t ldd,
                                           int64_t row0, int64_t row_end, int col0, int n, bool vec) {
    constexpr int W = F32 ? 32 : 64;   // columns per slice
    constexpr int ES = F32 ? 4 : 2;
    static_assert(C % W == 0, "whole slices");
#pragma unroll
    for (int s = 0; s < C / W; ++s) {
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 32; ++i)
            r[i] = F32 ? __float_as_uint(acc[s * W + i]) : bf16x2(acc[s * W + 2 * i], acc[s * W + 2 * i + 1]);
        __syncwarp();   // the slice before has been read out
        stage_rows32(stg, lane, r);
        __syncwarp();
        const int c = col0 + s * W + (lane & 7) * (16 / ES);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int rr = j * 4 + (lane >> 3);
            const uint4 v = ld_shared_v4(stg + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
            if (row0 + rr < row_end && c < n)
                store_d16<F32>(D + ((row0 + rr) * ldd + c) * ES, n - c, vec, v);
        }
    }
}

// ---- clusters ------------------------------------------------------------------
__device__ __forceinline__ uint32_t cta_rank_in_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t peer_address(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
// TMA load into this CTA's shared memory, completing on a barrier of the pair.
__device__ __forceinline__ void load_2d_pair(uint32_t dst, const void* desc, int32_t x, int32_t y, uint32_t bar,
                                             uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(desc)), "r"(x), "r"(y), "r"(bar), "l"(policy)
        : "memory");
}

// ---- the FP8 MMA ------------------------------------------------------------------
template <int CTAS>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    if constexpr (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}
// One arrival on `bar` in both CTAs of the pair once the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    const uint16_t mask = 0x3;
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            bar),
        "h"(mask)
        : "memory");
}
__device__ __forceinline__ void alloc_pair(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void free_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Host: the kernels' parameters for tiles of bm rows x bn columns of D.
F8Params f8_params(const F8Launch& a, int bm, int bn);
// Host: tensor map of an FP8 matrix (rows x k, row pitch ld), boxes of 128
// columns x box_rows, 128-byte swizzle; what lies outside reads as zero.
bool encode_f8(CUtensorMap* map, const void* ptr, int64_t k, int64_t rows, int64_t ld, int box_rows);

}  // namespace gemm
