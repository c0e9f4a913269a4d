// FP8 product with block scales for few rows (decode batches, experts with a
// few rows each).  Bt dwarfs A and D, so the work is to stream Bt once.
//
// Computed as D^T = Bt x A^T: a CTA's tile is 128 rows of Bt (the MMA's M
// side) by NT rows of A (its N side, NT in {16, 32, 64, 128}).  Per K block
// one 16 KiB box of Bt and NT * 128 bytes of A go through a shared-memory
// ring, four MMAs (K = 32) leave the block's sums in one of two TMEM buffers,
// and the epilogue thread that owns a row of Bt multiplies them by the row's
// and the columns' scales and adds them to fp32 sums in registers.
//
// With few tiles, a cluster of split_k CTAs shares a tile along K.  Each sends
// its sums to the CTAs that finish them (one share of the rows of A each)
// through distributed shared memory, and these add them up in rank order: no
// scratch, no second launch, and the same bits every time.  Sent, not fetched:
// a remote store needs no answer.
//
// Grouped by rows: the tiles of all groups are numbered on the device from the
// offsets; the grid is as large as any split of the rows could need, and
// clusters without a tile leave at once.
#include <cuda_runtime.h>

#include <cstring>

#include "f8_tc.cuh"
#include "internal.h"

namespace gemm {

namespace {

constexpr int kTileRows = 128;                          // rows of Bt per tile
constexpr int kWBytes = kTileRows * kF8RowBytes;
constexpr int kPreBytes = (GEMM_F8_MAX_GROUPS + 1) * 4 + 12;
constexpr int kCtrlBytes = 512;

template <int NT, bool BROWS>
struct Config {
    // epilogue warps per lane quarter and rows of A per thread: at most 32, so
    // that several warps share a scheduler and hide each other's waits
    static constexpr int PARTS = NT == 16 ? 1 : NT == 128 ? 4 : 2;
    static constexpr int EPI_WARPS = 4 * PARTS;
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int COLS = NT / PARTS;
    // 32 columns per thread and more: TMEM read as fragments, so that a lane
    // needs the scales of eight columns instead of 32 (f8_tc.cuh)
    static constexpr bool FRAG = COLS == 32;
    static constexpr int A_BYTES = NT * kF8RowBytes;
    static constexpr int STAGE = kWBytes + A_BYTES;
    // The ring covers the latency of Bt: two CTAs per SM with five stages each,
    // or one with 192 KiB (NT = 64, 64 x 8192 x 8192 on GB300: two CTAs with
    // four stages 19.8 us, one with eight 16.2 us)
    static constexpr int STAGES = NT <= 32 ? 5 : NT == 64 ? 8 : 6;
    static constexpr int BUFS = 4;                     // TMEM accumulators: the epilogue's latency spans several blocks
    static constexpr int TMEM = NT * BUFS < 32 ? 32 : NT * BUFS;
    static constexpr int SLOTS = 8;                     // blocks whose scales are in shared memory
    static constexpr int SLOT = NT * 4 + (BROWS ? kTileRows * 4 : 16);
    static constexpr int PER_SM = NT >= 64 ? 1 : 2;   // for the registers
    static constexpr size_t SMEM = static_cast<size_t>(STAGES) * STAGE + SLOTS * SLOT + kPreBytes + kCtrlBytes + 1024;
    static_assert(STAGES * STAGE >= NT * kTileRows * 4, "the sums of a split tile fit in the ring");
    static_assert(SMEM <= (PER_SM == 1 ? 227 : 113) * 1024 && SMEM > 24 * 1024, "one or two CTAs per SM");
};

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

template <int NT, bool BROWS>
__global__ void __launch_bounds__(Config<NT, BROWS>::THREADS, Config<NT, BROWS>::PER_SM)
    f8_skinny_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, const F8Params p,
                     const uint32_t idesc, const int split) {
    using R = Config<NT, BROWS>;
    constexpr int kStages = R::STAGES, kBufs = R::BUFS, kSlots = R::SLOTS, kCols = R::COLS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t sW = base;
    const uint32_t sA = base + kStages * kWBytes;
    const uint32_t sScale = base + kStages * R::STAGE;
    uint8_t* ctrl = smem_raw + (sScale - raw) + kSlots * R::SLOT;
    int32_t* pre = reinterpret_cast<int32_t*>(ctrl + kCtrlBytes);
    const uint32_t full0 = smem_u32(ctrl);
    const uint32_t done0 = full0 + 8u * kStages;
    const uint32_t acce0 = done0 + 8u * kStages;
    const uint32_t scale0 = acce0 + 8u * kBufs;
    const uint32_t used0 = scale0 + 8u * kSlots;
    static_assert(8 * (2 * kStages + kBufs + 2 * kSlots) + 8 <= kCtrlBytes, "barriers fit");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * (2 * kStages + kBufs + 2 * kSlots));
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmA);
    }
    const int rank = static_cast<int>(blockIdx.x) % split;
    const int id = static_cast<int>(blockIdx.x) / split;

    if (warp == 0) {   // one barrier per lane: full, done, acce, scale, used
        constexpr int kBars = 2 * kStages + kBufs + 2 * kSlots;
        for (int i = lane; i < kBars; i += 32) {
            const bool scale = i >= 2 * kStages + kBufs && i < kBars - kSlots;
            mbar_init(full0 + 8u * i, i < 2 * kStages ? 1 : scale ? 32 : R::EPI_WARPS);
        }
        if (lane == 0) *abort_flag = 0u;
        fence_barrier_init();
    }
    // TMEM is taken only once the kernel before has ended, so that neither
    // waits for the other's.
    pdl_wait();
    if (warp == 1 && p.mode != GEMM_GROUP_NONE) {
        if (p.mode == GEMM_GROUP_ROWS)
            group_prefix(p.offsets, p.groups, p.m, NT, p.pieces, lane, pre);
        else
            group_prefix(p.offsets, p.groups, p.kb * kF8Block, kF8Block, p.kb, lane, pre);
    }
    __syncthreads();

    // the cluster's tile: NT rows of A from arow (those before arow_end are
    // D's), 128 rows of Bt from brow, columns of D from col
    int arow, arow_end, drow, brow, col, sblock, kb_lo = 0, kb_hi = p.kb;
    if (p.mode == GEMM_GROUP_ROWS) {
        const int piece = id % p.pieces;
        if (piece >= pre[p.groups]) return;   // the whole cluster alike
        const int g = group_of(pre, p.groups, piece);
        int lo, hi;
        group_rows(p.offsets, g, p.m, lo, hi);
        arow = lo + (piece - pre[g]) * NT;
        arow_end = hi;
        drow = arow;
        col = id / p.pieces * kTileRows;
        brow = g * p.n + col;
        sblock = g * p.nb + col / kF8Block;
    } else {
        const int tm = id % p.tiles_m, r = id / p.tiles_m;
        const int g = r / p.tiles_n;
        arow = tm * NT;
        arow_end = p.m;
        drow = arow;
        col = (r - g * p.tiles_n) * kTileRows;
        brow = col;
        sblock = col / kF8Block;
        if (p.mode == GEMM_GROUP_K) {
            drow += g * p.m;
            kb_lo = min(pre[g], p.kb);
            kb_hi = min(pre[g + 1], p.kb);
        }
    }
    {   // this CTA's share of the K blocks
        const int len = kb_hi - kb_lo, at = kb_lo;
        kb_lo = at + static_cast<int>(static_cast<int64_t>(len) * rank / split);
        kb_hi = at + static_cast<int>(static_cast<int64_t>(len) * (rank + 1) / split);
    }
    const int blocks = kb_hi - kb_lo;

    // TMEM: the MMA warps and the epilogue wait for its address; the loads
    // start without it
    const auto tmem_ready = [] { asm volatile("bar.sync 1, %0;" ::"n"(64 + 32 * R::EPI_WARPS) : "memory"); };
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), R::TMEM);
        tmem_relinquish();
        pdl_launch_dependents();   // with this CTA's TMEM taken
        tc_fence_before();
    }
    if (warp == 1 || warp >= 3) {
        tmem_ready();
        tc_fence_after();
    }
    const uint32_t tmem = *tmem_slot;   // (the loading warps do not use it)

    uint64_t acc[kCols / 2];
#pragma unroll
    for (int j = 0; j < kCols / 2; ++j) acc[j] = 0;

    if (warp == 0) {
        // ---------------------------------------------------- operand loads --
        const uint64_t polw = p.tiles_m == 1 ? policy_evict_first() : policy_evict_normal();
        const uint64_t pola = policy_evict_last();
        Turn<kStages> at;
        int issued = 0;
        for (; issued < blocks; ++issued) {
            if (!wait_warp(done0 + 8u * at.i, at.ph ^ 1u, abort_flag, p.err, kDevErrTimeoutProducer)) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(full0 + 8u * at.i, R::STAGE);
                tma_load_2d(sW + at.i * kWBytes, &tmW, (kb_lo + issued) * kF8Block, brow, full0 + 8u * at.i, polw);
                tma_load_2d(sA + at.i * R::A_BYTES, &tmA, (kb_lo + issued) * kF8Block, arow, full0 + 8u * at.i, pola);
            }
            __syncwarp();
            at.next();
        }
        if (issued < blocks)   // after a time-out the copies still in flight land before the CTA ends
            for (int j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
                wait_bounded(full0 + 8u * (j % kStages), (j / kStages) & 1u, nullptr, p.err, kDevErrTimeoutTeardown);
    } else if (warp == 1 || warp == 3) {
        // ---------------- MMAs: warps 1 and 3 take the K blocks in turn, as
        // waiting and issuing take one warp longer than a block's loads
        Turn<kStages> st;
        Turn<kBufs> buf;
        st.i = buf.i = warp >> 1;
        int n = warp >> 1;
        for (; n < blocks; n += 2) {
            if (!wait_warp(acce0 + 8u * buf.i, buf.ph ^ 1u, abort_flag, p.err, kDevErrTimeoutMma) ||
                !wait_warp(full0 + 8u * st.i, st.ph, abort_flag, p.err, kDevErrTimeoutMma))
                break;
            tc_fence_after();
            const uint64_t wd = smem_desc_sw128_kmajor(sW + st.i * kWBytes);
            const uint64_t ad = smem_desc_sw128_kmajor(sA + st.i * R::A_BYTES);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kF8Block / kF8MmaK; ++kk)
                    mma_f8<1>(tmem + buf.i * NT, wd + 2u * kk, ad + 2u * kk, idesc, kk > 0 ? 1u : 0u);
                mma_commit(done0 + 8u * st.i);
            }
            __syncwarp();
            st.next(2);
            buf.next(2);
        }
        // the epilogue sees the last block done; after a time-out wait here for
        // the MMAs that were issued
        if (n < blocks && n > 1)
            wait_bounded(done0 + 8u * ((n - 2) % kStages), ((n - 2) / kStages) & 1u, nullptr, p.err, kDevErrTimeoutTeardown);
    } else if (warp == 2) {
        // ----------------------------------------------------------- scales --
        Turn<kSlots> slot;
        for (int n = 0; n < blocks; ++n) {
            if (!wait_warp(used0 + 8u * slot.i, slot.ph ^ 1u, abort_flag, p.err, kDevErrTimeoutProducer)) break;
            const int64_t kb = kb_lo + n;
            const uint32_t slot_at = sScale + slot.i * R::SLOT, dst = slot_at + 4 * lane;
#pragma unroll
            for (int i = 0; i < (NT + 31) / 32; ++i) {
                const int r = arow + lane + 32 * i;
                const bool in = r < p.rows_a;
                const int c = lane + 32 * i;
                if (NT >= 32 || lane < NT)
                    copy4_async(slot_at + 4 * (R::FRAG ? frag_place(c) : c), in ? p.a_scale + kb * p.rows_a + r : p.a_scale, in);
            }
            if constexpr (BROWS) {
#pragma unroll
                for (int i = 0; i < kTileRows / 32; ++i) {
                    const bool in = col + lane + 32 * i < p.n;
                    copy4_async(dst + NT * 4 + 128 * i, in ? p.b_scale + kb * p.rows_b + brow + lane + 32 * i : p.b_scale, in);
                }
            } else if (lane == 0) {
                copy4_async(slot_at + NT * 4, p.b_scale + static_cast<int64_t>(sblock) * p.kb + kb, true);
            }
            copies_arrive(scale0 + 8u * slot.i);
            slot.next();
        }
        copies_wait_all();
    } else if (warp >= 4) {
        // --------------------------------------------------- scale and add --
        const int q = warp & 3, h = (warp - 4) >> 2;   // lane quarter, part of the columns
        const uint32_t t0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * kCols;
        Turn<kStages> st;
        Turn<kBufs> buf;
        Turn<kSlots> slot;
        for (int n = 0; n < blocks; ++n) {
            if (!wait_warp_both(done0 + 8u * st.i, st.ph, scale0 + 8u * slot.i, slot.ph, abort_flag, p.err,
                                kDevErrTimeoutEpilogue))
                break;
            tc_fence_after();
            const uint32_t at = sScale + slot.i * R::SLOT;
            uint32_t v[kCols];
            if constexpr (R::FRAG) {
                float s[4];
                uint4 sc[2];
#pragma unroll
                for (int k = 0; k < (BROWS ? 4 : 1); ++k)
                    s[k] = ld_shared_f32(at + NT * 4 + (BROWS ? 4 * (q * 32 + (lane >> 2) + 8 * k) : 0));
#pragma unroll
                for (int i = 0; i < 2; ++i) sc[i] = ld_shared_v4(at + (h * kCols + i * 16 + (lane & 3) * 4) * 4);
                load_tmem_frag(t0 + buf.i * NT, v);
                wait_tmem(v);
                tc_fence_before();
                if (lane == 0) mbar_arrive(acce0 + 8u * buf.i);
                uint64_t s2[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    s2[i] = pair_of(__float_as_uint(s[BROWS ? 2 * i : 0]), __float_as_uint(s[BROWS ? 2 * i + 1 : 0]));
                add_scaled_frag(acc, v, s2, sc);
            } else {
                const float s = ld_shared_f32(at + NT * 4 + (BROWS ? 4 * (q * 32 + lane) : 0));
                uint4 sc[kCols / 4];
#pragma unroll
                for (int i = 0; i < kCols / 4; ++i) sc[i] = ld_shared_v4(at + (h * kCols + 4 * i) * 4);
                load_tmem(t0 + buf.i * NT, v);
                wait_tmem(v);
                tc_fence_before();
                if (lane == 0) mbar_arrive(acce0 + 8u * buf.i);
                add_scaled<kCols>(acc, v, pair_of(__float_as_uint(s), __float_as_uint(s)), sc);
            }
            __syncwarp();   // every lane has read the block's scales
            if (lane == 0) mbar_arrive(used0 + 8u * slot.i);
            st.next();
            buf.next();
            slot.next();
        }
    }

    // ------------------------------------------------------------ join, store --
    // The ring is idle: every block has been multiplied (or the call has failed).
    // put(r, c, v): row r of A, row c of Bt.  each(f): f(r, c, v) of this thread's sums.
    auto put = [&](int r, int c, float v) {
        if (r < arow_end - arow && col + c < p.n) {
            const int64_t at = (static_cast<int64_t>(drow) + r) * p.ldd + col + c;
            if (p.out_f32)
                static_cast<float*>(p.D)[at] = v;
            else
                static_cast<__nv_bfloat16*>(p.D)[at] = __float2bfloat16_rn(v);
        }
    };
    const int q = warp & 3, h = (warp - 4) >> 2;
    auto each = [&](auto f) {
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
            float x, y;
            unpair(acc[j], x, y);
            if constexpr (R::FRAG) {
                const int r = h * kCols + 4 * (j >> 1) + (lane & 3), c = q * 32 + (lane >> 2) + 16 * (j & 1);
                f(r, c, x);
                f(r, c + 8, y);
            } else {
                f(h * kCols + 2 * j, q * 32 + lane, x);
                f(h * kCols + 2 * j + 1, q * 32 + lane, y);
            }
        }
    };
    if (split == 1) {
        if (warp >= 4) each(put);
    } else {
        // Row r of A is finished by CTA r / share, whose ring (idle in every
        // CTA after the first barrier) holds sums[sender][row][row of Bt].
        const int share = NT / split, shift = 31 - __clz(share);   // a power of two
        cluster_barrier();
        if (warp >= 4)
            each([&](int r, int c, float v) {
                const int owner = r >> shift;
                st_cluster_f32(peer_address(base + ((rank * share + r - owner * share) * kTileRows + c) * 4, owner), v);
            });
        cluster_barrier();
        if (warp >= 4) {
            const int c = threadIdx.x & 127;
            for (int r = h; r < share; r += R::EPI_WARPS / 4) {
                float v = 0.f;
                for (int s = 0; s < split; ++s) v += ld_shared_f32(base + ((s * share + r) * kTileRows + c) * 4);
                put(share * rank + r, c, v);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, R::TMEM);
}

template <int NT, bool BROWS>
cudaError_t launch(const F8Launch& a, cudaStream_t stream) {
    using R = Config<NT, BROWS>;
    CUtensorMap mW, mA;
    if (!encode_f8(&mW, a.Bt, a.k, a.rows_b, a.ldb, kTileRows) || !encode_f8(&mA, a.A, a.k, a.rows_a, a.lda, NT))
        return cudaErrorInvalidValue;
    F8Params p = f8_params(a, NT, kTileRows);
    const int64_t tiles = a.group_mode == GEMM_GROUP_ROWS ? static_cast<int64_t>(p.pieces) * p.tiles_n
                                                          : static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.groups;
    if (tiles * a.split_k > INT32_MAX) return cudaErrorInvalidValue;
    const void* kern = reinterpret_cast<const void*>(f8_skinny_kernel<NT, BROWS>);
    const cudaError_t e = kernel_attrs_once(kern, static_cast<int>(R::SMEM), true);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.split_k);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.split_k), 1, 1);
    cfg.blockDim = dim3(R::THREADS, 1, 1);
    cfg.dynamicSmemBytes = R::SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    uint32_t idesc = idesc_f8(a.b_type, a.a_type, kTileRows, NT);
    int split = a.split_k;
    void* args[] = {&mW, &mA, &p, &idesc, &split};
    const cudaError_t r = cudaLaunchKernelExC(&cfg, kern, args);
    return r != cudaSuccess ? r : cudaGetLastError();
}

template <int NT>
cudaError_t launch_nt(const F8Launch& a, cudaStream_t stream) {
    return a.b_scale_mode == GEMM_SCALE_ROWS ? launch<NT, true>(a, stream) : launch<NT, false>(a, stream);
}

}  // namespace

cudaError_t launch_f8_skinny(const F8Launch& a, cudaStream_t stream) {
    switch (a.bm) {
        case 16: return launch_nt<16>(a, stream);
        case 32: return launch_nt<32>(a, stream);
        case 64: return launch_nt<64>(a, stream);
        default: return launch_nt<128>(a, stream);
    }
}

}  // namespace gemm
