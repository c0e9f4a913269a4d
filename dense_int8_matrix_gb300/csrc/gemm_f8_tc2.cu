// FP8 product with block scales on two-SM tiles (tcgen05 cta_group::2).
//
//   D[i][j] = sum_b (sa[b][i] * sb[..]) * (sum of block b of A[i] * Bt[j])
//
// A cluster of two CTAs computes a 256 x 256 tile (or a half, 256 x 128); each
// CTA loads 128 rows of A and of Bt per K block with TMA, and tcgen05.mma (M =
// 256, N = 256, K = 32, four per block) leaves its 128 rows in its own TMEM.  The
// scales change with every block of 128, so a block's sums are not added up
// in TMEM: the MMA of block b + 1 writes another TMEM buffer while the eight
// epilogue warps read block b's, multiply by the scales and add to fp32
// running sums in registers (128 per thread).
//
// Roles: warp 0 loads operands, warp 2 copies scales, warps 1 and 3 of the even
// CTA issue the MMAs of alternate blocks, warps 4-11 scale, add and store.
// Each role's loop is run by whole warps (one elected lane issues), so that its
// branches are uniform: together with the scales' own warp and one barrier
// round trip per block this took 8192^3 from 459 to 405 us.
// Grouped products read the group offsets on the device: warp 2 sums them into
// shared memory first, and every role walks the same list of tiles.
//
// What bounds it (GB300, bf16 output, 128 x 128 scales of Bt): 8192^3 takes
// 395 us, 2.79 PFLOP/s (450 on quantised data, under the power limit); without
// the epilogue's TMEM reads and multiply-adds 311 us (the MMAs, under the power
// limit), without the multiply-adds alone 350 us.  Per block and scheduler the
// epilogue's 256 cycles of multiply-adds and 140 of TMEM reads would fit beside
// the MMAs' 512, so it is not their number: at 4096^3 the tensor pipe is busy for
// 49 % of the time, a scheduler issues in 41 % of its cycles, and what warps wait
// for most is the TMEM read, whose latency each block's chain of reads pays.
// With column scales (1 x 128 for both) the multiply-adds double to the MMAs'
// own time: 8192^3 to fp32 580 us, which is longer than either; what the rest
// is has not been profiled.
#include <cuda_runtime.h>

#include <cstring>

#include "f8_tc.cuh"
#include "internal.h"

namespace gemm {

namespace {

constexpr int kHalfRows = 128;                       // rows of A per CTA
constexpr int kABytes = kHalfRows * kF8RowBytes;
constexpr int kPreBytes = (GEMM_F8_MAX_GROUPS + 1) * 4 + 12;
constexpr int kCtrlBytes = 512;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;

constexpr int kTileN = 256;                          // columns of a whole tile
constexpr int kCols = kTileN / 2;                    // columns of D per epilogue thread
constexpr int kBBytes = kTileN / 2 * kF8RowBytes;
constexpr int kStage = kABytes + kBBytes;
constexpr int kStages = 5;
constexpr int kBufs = 512 / kTileN;                  // TMEM accumulators
// Blocks whose scales are in shared memory.  Block i's are copied once block
// i - kAhead is multiplied: its accumulator was free then, so the block kBufs
// before it was read and the one before that added.  kAhead is small enough
// that the barrier it looks at cannot be a round further: block i - 1 + kBufs
// is the last that can be multiplied without i's scales.
constexpr int kAhead = kStages - kBufs;
constexpr int kSlots = kAhead + kBufs + 1;
template <bool BROWS>
struct Config {
    static constexpr int SLOT = kHalfRows * 4 + (BROWS ? kTileN * 4 : 16);
    static constexpr size_t SMEM = static_cast<size_t>(kStages) * kStage + kEpiWarps * kStageRowsBytes + kSlots * SLOT +
                                   kPreBytes + kCtrlBytes + 1024;
    static_assert(SMEM <= 232448, "shared memory");
};

struct Unit {
    int arow;      // first row of A of the pair's tile
    int drow;      // its row of D
    int dend;      // rows of D at or past this are not the tile's
    int brow;      // first row of Bt
    int col;       // first column of D
    int sblock;    // block-scale row: group * nb + col / 128
    int kb_lo, kb_hi;
    bool half;     // 128 columns instead of 256
};

// The list of units that the pairs take in turn: whole tiles, and the tiles of
// a last round that would leave half of the pairs idle as two halves of 128
// columns each.  Half a tile takes 0.77 of a whole one's time, so this pays
// where both halves run at once: 4096^3 (256 tiles on 76 pairs) 64.8 -> 61.3
// us, 512 x 4096 x 4096 (32 tiles) 18.9 -> 15.8 us.
struct Units {
    int whole, count;   // units [0, whole) are tiles, the rest halves
};
__device__ __forceinline__ Units list_units(const F8Params& p, const int32_t* pre, int npairs) {
    const int tiles = p.mode == GEMM_GROUP_ROWS ? pre[p.groups] * p.tiles_n : p.groups * p.tiles_m * p.tiles_n;
    Units x;
    x.whole = p.halves ? 0 : tiles / npairs * npairs;
    if (!p.halves && 2 * (tiles - x.whole) > npairs) x.whole = tiles;
    x.count = x.whole + 2 * (tiles - x.whole);
    return x;
}

__device__ __forceinline__ Unit unit_at(int u, const Units& list, const F8Params& p, const int32_t* pre) {
    const bool half = u >= list.whole;
    const int part = half ? (u - list.whole) & 1 : 0;
    if (half) u = list.whole + ((u - list.whole) >> 1);
    Unit x;
    int g = 0, tm, tn, lo = 0, hi = p.m;
    if (p.mode == GEMM_GROUP_ROWS) {
        g = group_of(pre, p.groups, u / p.tiles_n);
        group_rows(p.offsets, g, p.m, lo, hi);
        tc_tile_coords(u - pre[g] * p.tiles_n, pre[g + 1] - pre[g], p.tiles_n, tm, tn);
    } else {
        const int per = p.tiles_m * p.tiles_n;
        g = u / per;
        tc_tile_coords(u - g * per, p.tiles_m, p.tiles_n, tm, tn);
    }
    x.arow = lo + tm * 256;
    x.drow = x.arow;
    x.dend = hi;
    x.half = half;
    x.col = tn * kTileN + part * kF8Block;
    x.brow = x.col;
    x.sblock = x.col / kF8Block;
    x.kb_lo = 0;
    x.kb_hi = p.kb;
    if (p.mode == GEMM_GROUP_ROWS) {
        x.brow += g * p.n;
        x.sblock += g * p.nb;
    } else if (p.mode == GEMM_GROUP_K) {
        x.drow += g * p.m;
        x.dend += g * p.m;
        x.kb_lo = min(pre[g], p.kb);
        x.kb_hi = min(pre[g + 1], p.kb);
    }
    if (x.col >= p.n) x.kb_hi = x.kb_lo;   // a half past D's last column
    return x;
}

template <bool BROWS>
__global__ void __launch_bounds__(kThreads, 1)
    f8_tc2_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const F8Params p,
                  const uint32_t idesc, const uint32_t idesc_half) {
    using R = Config<BROWS>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t sA = base;
    const uint32_t sB = base + kStages * kABytes;
    const uint32_t sEpi = base + kStages * kStage;
    const uint32_t sScale = sEpi + kEpiWarps * kStageRowsBytes;
    uint8_t* ctrl = smem_raw + (sScale - raw) + kSlots * R::SLOT;
    int32_t* pre = reinterpret_cast<int32_t*>(ctrl + kCtrlBytes);
    const uint32_t bar0 = smem_u32(ctrl);
    const uint32_t full0 = bar0;                      // used in the even CTA
    const uint32_t done0 = full0 + 8u * kStages;      // a stage's block is multiplied
    const uint32_t acce0 = done0 + 8u * kStages;      // used in the even CTA: an accumulator has been read
    const uint32_t scale0 = acce0 + 8u * kBufs;       // a block's scales have landed
    const uint32_t last0 = scale0 + 8u * kSlots;
    static_assert(8 * (2 * kStages + kBufs + kSlots + 2) + 8 <= kCtrlBytes, "barriers fit");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * (2 * kStages + kBufs + kSlots + 2));
    volatile uint32_t* abort_flag = tmem_slot + 1;

    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank_in_cluster();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (warp == 0) {   // one barrier per lane: full, done, acce, scale, last
        constexpr int kBars = 2 * kStages + kBufs + kSlots + 2;
        for (int i = lane; i < kBars; i += 32) {
            const bool acce = i >= 2 * kStages && i < 2 * kStages + kBufs, scale = !acce && i >= 2 * kStages && i < kBars - 2;
            mbar_init(full0 + 8u * i, acce ? 2 * kEpiWarps : scale ? 32 : 1);
        }
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmB);
            *abort_flag = 0u;
        }
        fence_barrier_init();
    }
    if (warp == 1) alloc_pair(smem_u32(tmem_slot), 512);
    if (warp == 2 && p.mode != GEMM_GROUP_NONE) {
        pdl_wait();   // the offsets may come from the kernel before
        if (p.mode == GEMM_GROUP_ROWS)
            group_prefix(p.offsets, p.groups, p.m, 256, p.pieces, lane, pre);
        else
            group_prefix(p.offsets, p.groups, p.kb * kF8Block, kF8Block, p.kb, lane, pre);
    }
    tc_fence_before();
    __syncthreads();
    cluster_barrier();   // barriers and TMEM of both CTAs are ready
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Units list = list_units(p, pre, npairs);
    const int units = list.count;

    // the epilogue's running sums need more registers than an even share: of
    // 384 threads with 168, 128 keep 40 each and 256 take 232
    if (warp < 4) {
        fewer_registers<40>();
        if (warp == 0) {
            // ------------------------------------------------ operand loads --
            pdl_wait();
            const uint64_t pol = policy_evict_normal();
            const uint32_t full_leader = peer_address(full0, 0);
            Turn<kStages> at;
            uint32_t issued = 0;
            bool ok = true;
            for (int u = pair; ok && u < units; u += npairs) {
                const Unit w = unit_at(u, list, p, pre);
                const int ya = w.arow + static_cast<int>(rank) * kHalfRows;
                // (a half's box brings 64 rows more than are multiplied)
                const int yb = w.brow + static_cast<int>(rank) * (w.half ? kF8Block / 2 : kF8Block);
                for (int kb = w.kb_lo; kb < w.kb_hi; ++kb, ++issued) {
                    // the stage is free once the block that was in it has been multiplied
                    if (!wait_warp(done0 + 8u * at.i, at.ph ^ 1u, abort_flag, p.err, kDevErrTimeoutProducer)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t fb = full_leader + 8u * at.i;
                        if (leader) mbar_arrive_expect_tx(full0 + 8u * at.i, 2 * kStage);
                        load_2d_pair(sA + at.i * kABytes, &tmA, kb * kF8Block, ya, fb, pol);
                        load_2d_pair(sB + at.i * kBBytes, &tmB, kb * kF8Block, yb, fb, pol);
                    }
                    __syncwarp();
                    at.next();
                }
            }
            // after a time-out the copies still in flight land before the pair ends
            if (!ok && leader)
                for (uint32_t j = issued > kStages ? issued - kStages : 0u; j < issued; ++j)
                    wait_bounded(full0 + 8u * (j % kStages), (j / kStages) & 1u, nullptr, p.err, kDevErrTimeoutTeardown);
        }
        if (warp == 2) {
            // -------------------------------------------------------- scales --
            // The CTA's 128 row scales of each block, and the block scales of
            // the tile's column blocks (or its columns' scales).
            pdl_wait();
            Turn<kStages> at;   // block i - AHEAD, from i = AHEAD on
            Turn<kSlots> slot;
            uint32_t n = 0;
            bool ok = true;
            for (int u = pair; ok && u < units; u += npairs) {
                const Unit w = unit_at(u, list, p, pre);
                const int row0 = w.arow + static_cast<int>(rank) * kHalfRows + lane;
                const float* sa = p.a_scale + static_cast<int64_t>(w.kb_lo) * p.rows_a;
                const float* sb = BROWS ? p.b_scale + static_cast<int64_t>(w.kb_lo) * p.rows_b + w.brow + lane
                                        : p.b_scale + static_cast<int64_t>(w.sblock + (lane & 1)) * p.kb + w.kb_lo;
                const bool sb_in = w.col / kF8Block + (lane & 1) < p.nb;
                for (int kb = w.kb_lo; kb < w.kb_hi; ++kb) {
                    if (n >= kAhead) {
                        if (!wait_warp(done0 + 8u * at.i, at.ph, abort_flag, p.err, kDevErrTimeoutProducer)) {
                            ok = false;
                            break;
                        }
                        at.next();
                    }
                    ++n;
                    const uint32_t slot_at = sScale + slot.i * R::SLOT, dst = slot_at + 4 * lane;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool in = row0 + 32 * i < p.rows_a;
                        copy4_async(dst + 128 * i, in ? sa + row0 + 32 * i : p.a_scale, in);
                    }
                    if constexpr (BROWS) {
#pragma unroll
                        for (int i = 0; i < kTileN / 32; ++i) {
                            const bool in = w.col + lane + 32 * i < p.n;
                            copy4_async(slot_at + 512 + 4 * frag_place(lane + 32 * i), in ? sb + 32 * i : p.b_scale, in);
                        }
                        sb += p.rows_b;
                    } else {
                        if (lane < 2) copy4_async(dst + 512, sb_in ? sb : p.b_scale, sb_in);
                        sb += 1;
                    }
                    sa += p.rows_a;
                    copies_arrive(scale0 + 8u * slot.i);
                    slot.next();
                }
            }
            copies_wait_all();
        }
        if ((warp == 1 || warp == 3) && leader) {
            // ------------ MMAs: warps 1 and 3 take the K blocks in turn --
            const uint32_t turn = warp >> 1;
            Turn<kStages> st;
            Turn<kBufs> buf;
            st.i = buf.i = turn;
            uint32_t skip = turn;   // blocks until this warp's next one
            bool ok = true;
            for (int u = pair; ok && u < units; u += npairs) {
                const Unit w = unit_at(u, list, p, pre);
                const uint32_t blocks = static_cast<uint32_t>(w.kb_hi - w.kb_lo);
                const uint32_t desc = w.half ? idesc_half : idesc;
                uint32_t j = skip;
                for (; j < blocks; j += 2) {
                    if (!wait_warp(acce0 + 8u * buf.i, buf.ph ^ 1u, abort_flag, p.err, kDevErrTimeoutMma) ||
                        !wait_warp(full0 + 8u * st.i, st.ph, abort_flag, p.err, kDevErrTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = smem_desc_sw128_kmajor(sA + st.i * kABytes);
                    const uint64_t bd = smem_desc_sw128_kmajor(sB + st.i * kBBytes);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kF8Block / kF8MmaK; ++kk)
                            mma_f8<2>(tmem + buf.i * kTileN, ad + 2u * kk, bd + 2u * kk, desc, kk > 0 ? 1u : 0u);
                        commit_pair(done0 + 8u * st.i);
                    }
                    __syncwarp();
                    st.next(2);
                    buf.next(2);
                }
                skip = j - blocks;
            }
            if (elect_one()) commit_pair(last0 + 8u * turn);
            __syncwarp();
            wait_bounded(last0 + 8u * turn, 0u, nullptr, p.err, kDevErrTimeoutTeardown);
        }
    } else {
        // ------------------------------------------- scale, add and store --
        more_registers<232>();
        pdl_wait();
        const int e = warp - 4, q = warp & 3, h = e >> 2;
        const uint32_t stg = sEpi + e * kStageRowsBytes;
        const uint32_t acce = peer_address(acce0, 0);
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        // the lane's row, or the first of its four (eight rows apart)
        const uint32_t row_scale = sScale + 4 * (q * 32 + (BROWS ? lane >> 2 : lane));
        Turn<kStages> st;
        Turn<kBufs> buf;
        Turn<kSlots> slot;
        bool ok = true;
        for (int u = pair; ok && u < units; u += npairs) {
            const Unit w = unit_at(u, list, p, pre);
            const bool full = !w.half;
            const int in_tile = static_cast<int>(rank) * kHalfRows + q * 32;   // the warp's first row
            const int my = h * (full ? kCols : kCols / 2);                     // the thread's first column of the tile
            const uint32_t t0 = lanes + my;
            const uint32_t col_scale = sScale + 512 + (BROWS ? my * 4 : (my / kF8Block) * 4);
            uint64_t acc[kCols / 2];   // pairs of columns, or of rows (fragment form); the first half of them for a half
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) acc[j] = 0;
            // One chunk of 32 columns is added while the next is on its way,
            // the first of the next block included.  Order matters: what goes
            // through the shared-memory queue behind a TMEM load waits for it,
            // so scales are asked for first.
            uint32_t v[2][32];
            uint4 sc[2][2];
            float sa[BROWS ? 4 : 1], sb = 1.f;
            uint64_t s2[2] = {0, 0};
            auto chunk = [&](int c, uint32_t cols, uint32_t taddr) {
                if constexpr (BROWS) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) sc[c & 1][i] = ld_shared_v4(cols + (c * 32 + i * 16 + (lane & 3) * 4) * 4);
                    load_tmem_frag(taddr + c * 32, v[c & 1]);
                } else {
                    tmem_ld_32x32b_x32(taddr + c * 32, v[c & 1]);
                }
            };
            auto add = [&](int c) {
                if constexpr (BROWS)
                    add_scaled_frag(acc + c * 16, v[c & 1], s2, sc[c & 1]);
                else
                    add_scaled<32>(acc + c * 16, v[c & 1], s2[0]);
            };
            auto first_chunk = [&] {   // of the block that st, buf and slot point to
                tc_fence_after();
                const uint32_t cols = col_scale + slot.i * R::SLOT;
#pragma unroll
                for (int k = 0; k < (BROWS ? 4 : 1); ++k) sa[k] = ld_shared_f32(row_scale + slot.i * R::SLOT + 32 * k);
                if constexpr (!BROWS) sb = ld_shared_f32(cols);
                chunk(0, cols, t0 + buf.i * kTileN);
            };
            if (w.kb_lo < w.kb_hi) {
                ok = wait_warp_both(done0 + 8u * st.i, st.ph, scale0 + 8u * slot.i, slot.ph, abort_flag, p.err,
                                    kDevErrTimeoutEpilogue);
                if (!ok) break;
                first_chunk();
            }
            for (int left = w.kb_hi - w.kb_lo; left > 0; --left) {
                const uint32_t tb = t0 + buf.i * kTileN, free_bar = acce + 8u * buf.i, cols = col_scale + slot.i * R::SLOT;
                st.next();
                buf.next();
                slot.next();
                wait_tmem(v[0]);
                if constexpr (BROWS) {
                    s2[0] = pair_of(__float_as_uint(sa[0]), __float_as_uint(sa[1]));
                    s2[1] = pair_of(__float_as_uint(sa[2]), __float_as_uint(sa[3]));
                } else {
                    const uint32_t s = __float_as_uint(sa[0] * sb);
                    s2[0] = pair_of(s, s);
                }
                chunk(1, cols, tb);
                add(0);
                wait_tmem(v[1]);
                if (full) {
                    chunk(2, cols, tb);
                    add(1);
                    wait_tmem(v[0]);
                    chunk(3, cols, tb);
                    add(2);
                    wait_tmem(v[1]);
                }
                // all columns are in registers: the accumulator is free
                tc_fence_before();
                if (lane == 0) arrive_in_cluster(free_bar);
                if (left > 1) {
                    ok = wait_warp_both(done0 + 8u * st.i, st.ph, scale0 + 8u * slot.i, slot.ph, abort_flag, p.err,
                                        kDevErrTimeoutEpilogue);
                    if (!ok) break;
                    first_chunk();
                }
                if (full)
                    add(3);
                else
                    add(1);
            }
            if (!ok) break;
            uint8_t* D = static_cast<uint8_t*>(p.D);
            const int col = w.col + my, cols = full ? kCols : kCols / 2;
            if (p.out_f32)
                store_rows<true, BROWS, kCols>(acc, cols, stg, lane, D, p.ldd, w.drow + in_tile, w.dend, col, p.n, p.d_vec != 0);
            else
                store_rows<false, BROWS, kCols>(acc, cols, stg, lane, D, p.ldd, w.drow + in_tile, w.dend, col, p.n, p.d_vec != 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_barrier();   // the peer may still use this CTA's shared memory or barriers until here
    tc_fence_after();
    if (warp == 1) free_pair(tmem, 512);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

template <bool BROWS>
cudaError_t launch(const F8Launch& a, cudaStream_t stream) {
    using R = Config<BROWS>;
    CUtensorMap mA, mB;
    if (!encode_f8(&mA, a.A, a.k, a.rows_a, a.lda, kHalfRows) || !encode_f8(&mB, a.Bt, a.k, a.rows_b, a.ldb, kTileN / 2))
        return cudaErrorInvalidValue;
    F8Params p = f8_params(a, 256, kTileN);
    p.halves = a.bn == kF8Block ? 1 : 0;
    const int64_t tiles = a.group_mode == GEMM_GROUP_ROWS ? static_cast<int64_t>(p.pieces) * p.tiles_n
                                                          : static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.groups;
    if (2 * tiles > INT32_MAX) return cudaErrorInvalidValue;
    int64_t pairs = a.pairs > 0 ? a.pairs : a.num_sms / 2;
    if (pairs < 1) pairs = 1;
    // (grouped by rows, `tiles` is only the most there can be)
    const int64_t use = p.halves || 2 * tiles <= pairs || a.group_mode == GEMM_GROUP_ROWS ? 2 * tiles : tiles;
    if (pairs > use) pairs = use;
    const void* kern = reinterpret_cast<const void*>(f8_tc2_kernel<BROWS>);
    const cudaError_t e = kernel_attrs_once(kern, static_cast<int>(R::SMEM), true);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = R::SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    uint32_t idesc = idesc_f8(a.a_type, a.b_type, 256, kTileN), idesc_half = idesc_f8(a.a_type, a.b_type, 256, kTileN / 2);
    void* args[] = {&mA, &mB, &p, &idesc, &idesc_half};
    const cudaError_t r = cudaLaunchKernelExC(&cfg, kern, args);
    return r != cudaSuccess ? r : cudaGetLastError();
}

}  // namespace

bool encode_f8(CUtensorMap* map, const void* ptr, int64_t k, int64_t rows, int64_t ld, int box_rows) {
    auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!enc) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(kF8RowBytes), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

F8Params f8_params(const F8Launch& a, int bm, int bn) {
    F8Params p;
    p.a_scale = a.a_scale;
    p.b_scale = a.b_scale;
    p.offsets = a.offsets;
    p.D = a.D;
    p.err = a.err;
    p.ldd = a.ldd;
    p.rows_a = a.rows_a;
    p.rows_b = a.rows_b;
    p.m = static_cast<int>(a.m);
    p.n = static_cast<int>(a.n);
    p.groups = a.groups;
    p.mode = a.group_mode;
    p.kb = static_cast<int>((a.k + kF8Block - 1) / kF8Block);
    p.nb = static_cast<int>((a.n + kF8Block - 1) / kF8Block);
    p.tiles_m = static_cast<int>((a.m + bm - 1) / bm);
    p.tiles_n = static_cast<int>((a.n + bn - 1) / bn);
    p.halves = 0;
    p.pieces = static_cast<int>(a.m / bm + (a.groups < a.m ? a.groups : a.m));   // each group may end in a part of a tile
    p.out_f32 = a.out_f32 ? 1 : 0;
    p.d_vec = reinterpret_cast<uintptr_t>(a.D) % 16 == 0 && (a.ldd * (a.out_f32 ? 4 : 2)) % 16 == 0;
    return p;
}

cudaError_t launch_f8_tc2(const F8Launch& a, cudaStream_t stream) {
    return a.b_scale_mode == GEMM_SCALE_ROWS ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace gemm
