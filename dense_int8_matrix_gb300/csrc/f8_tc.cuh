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
    int halves;           // two-SM kernel: every tile in halves of 128 columns (plans edited to bn = 128)
    int pieces;           // row tiles that all groups together can have (GEMM_GROUP_ROWS)
};

// wait_bounded() for a whole converged warp: all lanes probe, and the branches
// are uniform (a ready barrier costs about 30 cycles; with a loop that each
// lane leaves by itself it measured 170).  The clock that bounds the wait is
// slow to read, so it is asked only after some probes.
constexpr int kWaitProbes = 256;
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, int* err_word,
                                          int code) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
#pragma unroll 1
    for (int i = 0; i < kWaitProbes; ++i)
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, err_word, code));
}

// Both barriers at once: one round trip instead of two.
__device__ __forceinline__ bool wait_warp_both(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1,
                                               volatile uint32_t* abort_flag, int* err_word, int code) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
        "and.pred p, p, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar0), "r"(parity0), "r"(bar1), "r"(parity1)
        : "memory");
    if (__all_sync(0xffffffffu, ok != 0)) return true;
    return wait_warp(bar0, parity0, abort_flag, err_word, code) && wait_warp(bar1, parity1, abort_flag, err_word, code);
}

// One lane of a converged warp.  The loading and MMA warps run their loops
// whole, so that addresses and descriptors stay in uniform registers, and
// this lane issues (measured for one MMA issuer, see gemm_f8_tc2.cu).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A place in a ring of N and the parity of the round, stepped without division.
template <uint32_t N>
struct Turn {
    uint32_t i = 0, ph = 0;
    __device__ __forceinline__ void next(uint32_t by = 1) {
        i += by;
        if (i >= N) {
            i -= N;
            ph ^= 1u;
        }
    }
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
        // stays in 32 bits: of 32 clamped ranges in a row at most every other one can
        // start over, so they hold at most 16 times the rows (2^30), 2^30 / 16
        // pieces of the least size each time, and `before` is at most 2^26 + 1024
        int sum = c;
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

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// Waits for this thread's TMEM loads; r is not read before.
__device__ __forceinline__ void wait_tmem(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void wait_tmem(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void load_tmem(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld_32x32b_x32(taddr, r); }
__device__ __forceinline__ void load_tmem(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_32x32b_x16(taddr, r); }

// Two fp32 values in one 64-bit register pair, and a * b + c on both.
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float& lo, float& hi) {
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(d));
    lo = __uint_as_float(a);
    hi = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Adds N columns of a block's sums to the running sums: times s, or times s
// and the columns' scales c.
template <int N>
__device__ __forceinline__ void add_scaled(uint64_t* acc, const uint32_t (&v)[N], uint64_t s) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) acc[j] = fma2(pair_of(v[2 * j], v[2 * j + 1]), s, acc[j]);
}
template <int N>
__device__ __forceinline__ void add_scaled(uint64_t* acc, const uint32_t (&v)[N], uint64_t s, const uint4 (&c)[N / 4]) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
        acc[2 * j] = fma2(pair_of(v[4 * j], v[4 * j + 1]), mul2(s, pair_of(c[j].x, c[j].y)), acc[2 * j]);
        acc[2 * j + 1] = fma2(pair_of(v[4 * j + 2], v[4 * j + 3]), mul2(s, pair_of(c[j].z, c[j].w)), acc[2 * j + 1]);
    }
}

// The fragment form, for tiles whose columns have scales of their own.  With
// lane = row every lane would need every column's scale, and handing 128 of
// them to each lane of eight warps takes shared memory's way into the
// registers longer than the block's MMAs (1024 cycles of 128 bytes).
// tcgen05.ld's 16x128b shape gives a lane four rows (lane / 4 + 0, 8, 16, 24)
// and every fourth column (lane % 4), so it needs a quarter of them; it reads
// at half the rate of 32x32b (16x256b, with pairs of columns, at a quarter).
// v: 32 columns, [half of the rows][four columns][row + 0, 8].
__device__ __forceinline__ void load_tmem_frag(uint32_t taddr, uint32_t (&v)[32]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x128b.x8.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(v[16 * h]), "=r"(v[16 * h + 1]), "=r"(v[16 * h + 2]), "=r"(v[16 * h + 3]), "=r"(v[16 * h + 4]),
              "=r"(v[16 * h + 5]), "=r"(v[16 * h + 6]), "=r"(v[16 * h + 7]), "=r"(v[16 * h + 8]), "=r"(v[16 * h + 9]),
              "=r"(v[16 * h + 10]), "=r"(v[16 * h + 11]), "=r"(v[16 * h + 12]), "=r"(v[16 * h + 13]),
              "=r"(v[16 * h + 14]), "=r"(v[16 * h + 15])
            : "r"(taddr + (static_cast<uint32_t>(16 * h) << 16)));
}
// Column scales of a tile in shared memory are ordered so that a lane reads
// four of its columns at once: within sixteen columns, column c is at place
// frag_place(c).
__device__ __forceinline__ int frag_place(int c) { return (c & ~15) + (c & 3) * 4 + ((c >> 2) & 3); }
// s: the lane's row scales (rows + 0 and + 8, + 16 and + 24); c: the scales of
// its eight columns.  acc: [four columns][half of the rows].
__device__ __forceinline__ void add_scaled_frag(uint64_t* acc, const uint32_t (&v)[32], const uint64_t (&s)[2],
                                                const uint4 (&c)[2]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint4 x = c[j >> 2];
        const uint32_t y = (j & 3) == 0 ? x.x : (j & 3) == 1 ? x.y : (j & 3) == 2 ? x.z : x.w;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 16 * h + 2 * j;
            acc[2 * j + h] = fma2(pair_of(v[i], v[i + 1]), mul2(s[h], pair_of(y, y)), acc[2 * j + h]);
        }
    }
}

// Four bytes from global to shared memory without waiting (zero if !in).
__device__ __forceinline__ void copy4_async(uint32_t dst, const float* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)),
                 "r"(in ? 4 : 0)
                 : "memory");
}
// One arrival on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Waits for them (before the CTA ends).
__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) { return __uint_as_float(ld_shared_u32(addr)); }

// Registers of the calling warpgroup (all four warps call it).
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// A warp's 32 rows (lane = row) x `cols` of C columns of sums leave for D in slices of
// 128 bytes per row: through the warp's 4 KiB staging buffer (16-byte chunks
// swizzled by row & 7, free of bank conflicts both ways), so that eight lanes
// write one row's 128 bytes.  All of a slice is read back before the first
// store, as each would wait for its own read otherwise.  acc: pairs of columns
// of the lane's row, or (FRAG) the fragment form.  row0: D's row of the warp's
// first; rows at or past row_end and columns at or past n are not written.
constexpr int kStageRowsBytes = 32 * 128;
template <bool F32, bool FRAG, int C>
__device__ __forceinline__ void store_rows(const uint64_t (&acc)[C / 2], int cols, uint32_t stg, int lane, uint8_t* D, int64_t ldd,
                                           int64_t row0, int64_t row_end, int col0, int n, bool vec) {
    constexpr int W = F32 ? 32 : 64;   // columns per slice
    constexpr int ES = F32 ? 4 : 2;
    static_assert(C % W == 0, "whole slices");
    const int rows = static_cast<int>(row_end - row0 < 32 ? row_end - row0 : 32);
    const int r0 = lane >> 3, part = lane & 7;
    uint8_t* out = D + ((row0 + r0) * ldd + col0 + part * (16 / ES)) * ES;
    const int64_t step = 4 * ldd * ES;
    const bool whole = vec && n - col0 >= cols;   // the warp's columns are all D's, and 16-byte aligned
    const bool pairs = ldd % 2 == 0 && reinterpret_cast<uintptr_t>(D) % 4 == 0;
#pragma unroll
    for (int s = 0; s < C / W; ++s) {
        if (s * W >= cols) break;
        __syncwarp();   // the slice before has been read out
        if constexpr (FRAG) {
#pragma unroll
            for (int j = 0; j < W / 4; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[2];
                    unpair(acc[(s * (W / 4) + j) * 2 + h], x[0], x[1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int rr = (lane >> 2) + 16 * h + 8 * k;
                        const int at = (4 * j + (lane & 3)) * ES;   // byte in the row's 128
                        const uint32_t p = stg + rr * 128 + (((at >> 4) ^ (rr & 7)) << 4) + (at & 15);
                        if constexpr (F32)
                            st_shared_u32(p, __float_as_uint(x[k]));
                        else
                            asm volatile("st.shared.b16 [%0], %1;" ::"r"(p),
                                         "h"(__bfloat16_as_ushort(__float2bfloat16_rn(x[k])))
                                         : "memory");
                    }
                }
        } else {
            uint32_t r[32];
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                float a, b;
                unpair(acc[s * W / 2 + i], a, b);
                if constexpr (F32) {
                    r[2 * i] = __float_as_uint(a);
                    r[2 * i + 1] = __float_as_uint(b);
                } else {
                    r[i] = bf16x2(a, b);
                }
            }
            stage_rows32(stg, lane, r);
        }
        __syncwarp();
        uint4 v[8];
        if (whole)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = ld_shared_v4(stg + (4 * j + r0) * 128 + ((part ^ ((4 * j + r0) & 7)) << 4));
        if (whole) {   // predicated stores and no branch around any
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (4 * j + r0 < rows) *reinterpret_cast<uint4*>(out + j * step + s * W * ES) = v[j];
        } else {
            // ragged columns or unaligned rows: one row per store, so that each is
            // contiguous; four rows are read before the first is stored (4096^3
            // at n = 4095 74.7 -> 71.5 us; eight gain 1.3 more, but cost aligned
            // fp32 products with column scales a few per cent)
            const int c = col0 + s * W;
            uint8_t* to = D + (row0 * ldd + c) * ES;
#pragma unroll 1
            for (int r4 = 0; r4 < 32; r4 += 4) {
                uint32_t x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = ld_shared_u32(stg + (r4 + j) * 128 + (((lane >> 2) ^ ((r4 + j) & 7)) << 4) + (lane & 3) * 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int rr = r4 + j;
                    if (rr >= rows) continue;
                    if constexpr (F32) {
                        if (c + lane < n) reinterpret_cast<uint32_t*>(to)[rr * ldd + lane] = x[j];
                    } else if (pairs) {
                        if (c + 2 * lane + 1 < n)
                            reinterpret_cast<uint32_t*>(to + rr * ldd * 2)[lane] = x[j];
                        else if (c + 2 * lane < n)
                            reinterpret_cast<uint16_t*>(to)[rr * ldd + 2 * lane] = static_cast<uint16_t>(x[j]);
                    } else {
                        uint16_t* o = reinterpret_cast<uint16_t*>(to) + rr * ldd + 2 * lane;
                        if (c + 2 * lane < n) o[0] = static_cast<uint16_t>(x[j]);
                        if (c + 2 * lane + 1 < n) o[1] = static_cast<uint16_t>(x[j] >> 16);
                    }
                }
            }
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
// A float of another CTA of the cluster (behind a barrier).
__device__ __forceinline__ float load_in_cluster(uint32_t addr_cluster) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr_cluster));
    return v;
}
// Sums over the CTAs of a cluster of n floats that each has in shared memory at
// `at`, in rank order: put(i, sum) by one thread of one CTA for each i.  The
// whole cluster.
constexpr int kMostClusterCtas = 8;
template <typename F>
__device__ __forceinline__ void join_cluster(const float* at, int n, int ctas, F put) {
    if (ctas == 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += blockDim.x) put(i, at[i]);
        return;
    }
    const uint32_t base = smem_u32(at);
    cluster_barrier();
    for (int i = static_cast<int>(cta_rank_in_cluster()) + ctas * threadIdx.x; i < n; i += ctas * blockDim.x) {
        float v[kMostClusterCtas], sum = 0.f;   // (asked for together: a remote read takes its time)
#pragma unroll
        for (int r = 0; r < kMostClusterCtas; ++r) v[r] = r < ctas ? load_in_cluster(peer_address(base + 4 * i, r)) : 0.f;
#pragma unroll
        for (int r = 0; r < kMostClusterCtas; ++r) sum += v[r];
        put(i, sum);
    }
    cluster_barrier();   // the others' shared memory has been read
}

// Arrives on a barrier of a CTA of the cluster, releasing no memory beyond the
// CTA: for hand-offs whose data is in TMEM (tcgen05.fence orders it).  A
// release for the cluster waits for the thread's global accesses.
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
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

// launch_chained with clusters of x * y CTAs.
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kern)(P...), dim3 grid, dim3 cluster, unsigned threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster.x;
    attr[0].val.clusterDim.y = cluster.y;
    attr[0].val.clusterDim.z = cluster.z;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Host: the kernels' parameters for tiles of bm rows x bn columns of D.
F8Params f8_params(const F8Launch& a, int bm, int bn);
// Host: tensor map of an FP8 matrix (rows x k, row pitch ld), boxes of 128
// columns x box_rows, 128-byte swizzle; what lies outside reads as zero.
bool encode_f8(CUtensorMap* map, const void* ptr, int64_t k, int64_t rows, int64_t ld, int box_rows);

}  // namespace gemm
