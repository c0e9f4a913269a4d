// FP8 product with block scales on two-SM tiles (tcgen05 cta_group::2).
//
//   D[i][j] = sum_b (sa[b][i] * sb[..]) * (sum of block b of A[i] * Bt[j])
//
// A cluster of two CTAs computes a 256 x BN tile; each CTA loads 128 rows of
// A and BN / 2 rows of Bt per K block with TMA, and one tcgen05.mma (M = 256,
// N = BN, K = 32, four per block) leaves its 128 rows in its own TMEM.  The
// scales change with every block of 128, so a block's sums are not added up
// in TMEM: the MMA of block b + 1 writes another TMEM buffer while the eight
// epilogue warps read block b's, multiply by the scales and add to fp32
// running sums in registers (BN / 2 per thread).  The tensor pipe needs
// 2 * BN cycles per block; reading BN columns of TMEM and the BN multiply-adds
// per lane quarter fit beside it.
//
// Roles as in the library's other two-SM kernel: warp 0 loads, warp 1 of the
// even CTA issues MMAs, warps 4-11 scale, add and store.  Grouped products
// read the group offsets on the device: warp 2 sums them into shared memory
// first, and every role walks the same list of tiles.
#include <cuda_runtime.h>

#include <cstring>

#include "f8_tc.cuh"
#include "internal.h"

namespace gemm {

namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kHalfRows = 128;                       // rows of A per CTA
constexpr int kABytes = kHalfRows * kF8RowBytes;
constexpr int kEpiBytes = kEpiWarps * 4096;
constexpr int kPreBytes = (GEMM_F8_MAX_GROUPS + 1) * 4 + 12;
constexpr int kCtrlBytes = 512;

template <int BN>
struct Ring {
    static constexpr int B_BYTES = BN / 2 * kF8RowBytes;
    static constexpr int STAGE = kABytes + B_BYTES;
    static constexpr int STAGES = BN == 256 ? 5 : 7;
    static constexpr int BUFS = 512 / BN;            // TMEM accumulators
    static constexpr int SCALES = 2 * (BN / 2) * 4;  // column scales of two blocks, per epilogue warp
    static constexpr size_t SMEM = static_cast<size_t>(STAGES) * STAGE + kEpiBytes + kEpiWarps * SCALES + kPreBytes + kCtrlBytes + 1024;
};
static_assert(Ring<256>::SMEM <= 232448 && Ring<128>::SMEM <= 232448, "shared memory");

struct Unit {
    int arow;      // first row of A of the pair's tile
    int drow;      // its row of D
    int dend;      // rows of D at or past this are not the tile's
    int brow;      // first row of Bt
    int col;       // first column of D
    int sblock;    // block-scale row: group * nb + col / 128
    int kb_lo, kb_hi;
};

__device__ __forceinline__ int unit_count(const F8Params& p, const int32_t* pre) {
    if (p.mode == GEMM_GROUP_ROWS) return pre[p.groups] * p.tiles_n;
    return p.groups * p.tiles_m * p.tiles_n;
}

template <int BN>
__device__ __forceinline__ Unit unit_at(int u, const F8Params& p, const int32_t* pre) {
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
    x.col = tn * BN;
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
    return x;
}

template <int BN, bool BROWS>
__global__ void __launch_bounds__(kThreads, 1)
    f8_tc2_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const F8Params p,
                  const uint32_t idesc) {
    using R = Ring<BN>;
    constexpr int kStages = R::STAGES, kBufs = R::BUFS;
    constexpr int kCols = BN / 2;   // columns per epilogue thread
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t sA = base;
    const uint32_t sB = base + kStages * kABytes;
    const uint32_t sEpi = base + kStages * R::STAGE;
    const uint32_t sScale = sEpi + kEpiBytes;
    uint8_t* ctrl = smem_raw + (sScale - raw) + kEpiWarps * R::SCALES;
    int32_t* pre = reinterpret_cast<int32_t*>(ctrl + kCtrlBytes);
    const uint32_t bar0 = smem_u32(ctrl);
    const uint32_t full0 = bar0;                      // used in the even CTA
    const uint32_t done0 = full0 + 8u * kStages;      // a stage's block is multiplied
    const uint32_t acce0 = done0 + 8u * kStages;      // used in the even CTA: an accumulator has been read
    const uint32_t last0 = acce0 + 8u * kBufs;
    static_assert(8 * (2 * kStages + kBufs + 2) + 8 <= kCtrlBytes, "barriers fit");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * (2 * kStages + kBufs + 2));
    volatile uint32_t* abort_flag = tmem_slot + 1;

    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank_in_cluster();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8u * s, 2);   // the arrivals that announce A's and Bt's bytes
            mbar_init(done0 + 8u * s, 1);
        }
        for (int b = 0; b < kBufs; ++b) mbar_init(acce0 + 8u * b, 2 * kEpiWarps);
        mbar_init(last0, 1);
        mbar_init(last0 + 8u, 1);
        *abort_flag = 0u;
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
    const int units = unit_count(p, pre);

    // the epilogue's running sums need more registers than an even share: 128
    // threads keep 40 each, 256 take 232, as many as were launched (384 * 168)
    if (warp < 4) {
        fewer_registers<40>();
        if ((warp == 0 || warp == 2) && lane == 0) {
            // ------------------------------- loads: warp 0 A, warp 2 Bt --
            pdl_wait();
            const bool isA = warp == 0;
            const uint64_t pol = policy_evict_normal();
            const uint32_t dst = isA ? sA : sB, step = isA ? kABytes : R::B_BYTES;
            const void* map = isA ? &tmA : &tmB;
            const int off = static_cast<int>(rank) * (isA ? kHalfRows : BN / 2);
            const uint32_t full_leader = peer_address(full0, 0);
            Turn<kStages> at;
            uint32_t issued = 0;
            bool ok = true;
            for (int u = pair; ok && u < units; u += npairs) {
                const Unit w = unit_at<BN>(u, p, pre);
                const int y = (isA ? w.arow : w.brow) + off;
                for (int kb = w.kb_lo; kb < w.kb_hi; ++kb, ++issued) {
                    // the stage is free once the block that was in it has been multiplied
                    if (!wait_step(done0 + 8u * at.i, at.ph ^ 1u, abort_flag, p.err, kDevErrTimeoutProducer)) {
                        ok = false;
                        break;
                    }
                    if (leader) mbar_arrive_expect_tx(full0 + 8u * at.i, 2 * step);
                    load_2d_pair(dst + at.i * step, map, kb * kF8Block, y, full_leader + 8u * at.i, pol);
                    at.next();
                }
            }
            // after a time-out the copies still in flight land before the pair ends
            if (!ok && leader)
                for (uint32_t j = issued > kStages ? issued - kStages : 0u; j < issued; ++j)
                    wait_bounded(full0 + 8u * (j % kStages), (j / kStages) & 1u, nullptr, p.err, kDevErrTimeoutTeardown);
        }
        if ((warp == 1 || warp == 3) && lane == 0 && leader) {
            // ------------ MMAs: warps 1 and 3 take the K blocks in turn --
            const uint32_t turn = warp >> 1;
            Turn<kStages> st;
            Turn<kBufs> buf;
            st.i = buf.i = turn;
            uint32_t skip = turn;   // blocks until this warp's next one
            bool ok = true;
            for (int u = pair; ok && u < units; u += npairs) {
                const Unit w = unit_at<BN>(u, p, pre);
                const uint32_t blocks = static_cast<uint32_t>(w.kb_hi - w.kb_lo);
                uint32_t j = skip;
                for (; j < blocks; j += 2) {
                    if (!wait_step(acce0 + 8u * buf.i, buf.ph ^ 1u, abort_flag, p.err, kDevErrTimeoutMma) ||
                        !wait_step(full0 + 8u * st.i, st.ph, abort_flag, p.err, kDevErrTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = smem_desc_sw128_kmajor(sA + st.i * kABytes);
                    const uint64_t bd = smem_desc_sw128_kmajor(sB + st.i * R::B_BYTES);
#pragma unroll
                    for (int kk = 0; kk < kF8Block / kF8MmaK; ++kk)
                        mma_f8<2>(tmem + buf.i * BN, ad + 2u * kk, bd + 2u * kk, idesc, kk > 0 ? 1u : 0u);
                    commit_pair(done0 + 8u * st.i);
                    st.next(2);
                    buf.next(2);
                }
                skip = j - blocks;
            }
            commit_pair(last0 + 8u * turn);
            wait_bounded(last0 + 8u * turn, 0u, nullptr, p.err, kDevErrTimeoutTeardown);
        }
    } else {
        more_registers<232>();
        pdl_wait();
        const int e = warp - 4, q = warp & 3, h = e >> 2;
        const uint32_t stg = sEpi + e * 4096, scl = sScale + e * R::SCALES;
        const uint32_t acce = peer_address(acce0, 0);
        Turn<kStages> st;
        Turn<kBufs> buf;
        bool ok = true;
        for (int u = pair; ok && u < units; u += npairs) {
            const Unit w = unit_at<BN>(u, p, pre);
            const int in_tile = static_cast<int>(rank) * kHalfRows + q * 32;   // the warp's first row
            const int arow = min(w.arow + in_tile + lane, static_cast<int>(p.rows_a) - 1);
            const int col = w.col + h * kCols;
            const float* sa = p.a_scale + arow;
            // column scales: one per block of 128 columns, or one per column
            const float* sb = BROWS ? p.b_scale + (w.brow - w.col) + col
                                    : p.b_scale + static_cast<int64_t>(w.sblock + (BN == 256 ? h : 0)) * p.kb;
            const bool col_in = BROWS || col / kF8Block < p.nb;
            uint64_t acc[kCols / 2];   // pairs of columns
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) acc[j] = 0;
            // The scales of four blocks are loaded while the four before are
            // added: a load takes longer than a block.  Loads past the last
            // block repeat it.
            float cur[4], sa_next[4], sb_next[4];
            const int last = max(w.kb_hi - 1, w.kb_lo);
            auto load_scales = [&](int kb) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t x = min(kb + i, last);
                    sa_next[i] = __ldg(sa + x * p.rows_a);
                    if constexpr (!BROWS) sb_next[i] = col_in ? __ldg(sb + x) : 0.f;
                }
            };
            auto take_scales = [&] {
#pragma unroll
                for (int i = 0; i < 4; ++i) cur[i] = BROWS ? sa_next[i] : sa_next[i] * sb_next[i];
            };
            // column scales: through the warp's shared memory, two blocks deep
            float sc_next[BROWS ? kCols / 32 : 1];
            auto load_cols = [&](int kb) {
                const float* x = sb + static_cast<int64_t>(min(kb, last)) * p.rows_b + lane;
#pragma unroll
                for (int i = 0; i < (BROWS ? kCols / 32 : 0); ++i) sc_next[i] = col + lane + 32 * i < p.n ? __ldg(x + 32 * i) : 0.f;
            };
            constexpr int kChunks = kCols / 32;
            const uint32_t t0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * kCols;
            // 32 columns are added while the next 32 are on their way, the
            // first of the next block included
            uint32_t v[2][32];
            if (w.kb_lo < w.kb_hi) {
                load_scales(w.kb_lo);
                if constexpr (BROWS) load_cols(w.kb_lo);
                take_scales();
                load_scales(w.kb_lo + 4);
                ok = wait_step(done0 + 8u * st.i, st.ph, abort_flag, p.err, kDevErrTimeoutEpilogue);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                tmem_ld_32x32b_x32(t0 + buf.i * BN, v[0]);
            }
            int left = w.kb_hi - w.kb_lo;   // blocks
            for (int i = 0; left > 0; ++i, --left) {
                const bool more = left > 1;
                float s = i & 2 ? (i & 1 ? cur[3] : cur[2]) : (i & 1 ? cur[1] : cur[0]);
                const uint32_t cols = scl + (i & 1) * (kCols * 4);
                if constexpr (BROWS) {
#pragma unroll
                    for (int x = 0; x < kCols / 32; ++x) st_shared_u32(cols + 4 * (lane + 32 * x), __float_as_uint(sc_next[x]));
                    __syncwarp();
                    load_cols(w.kb_lo + i + 1);
                }
                if ((i & 3) == 3) {
                    take_scales();
                    load_scales(w.kb_lo + i + 5);
                }
                const uint64_t s2 = pair_of(__float_as_uint(s), __float_as_uint(s));
                const uint32_t tb = t0 + buf.i * BN, free_bar = acce + 8u * buf.i;
                st.next();
                buf.next();
                bool ready = true;
                wait_tmem(v[0]);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    if (c + 1 < kChunks) {
                        tmem_ld_32x32b_x32(tb + (c + 1) * 32, v[(c + 1) & 1]);
                        if (c + 2 == kChunks && more) ready = mbar_try_wait(done0 + 8u * st.i, st.ph);   // asked early
                        add_scaled<BROWS>(acc + c * 16, v[c & 1], s2, cols + c * 128);
                        wait_tmem(v[(c + 1) & 1]);
                    } else {
                        // all columns are in registers: the accumulator is free
                        tc_fence_before();
                        if (lane == 0) arrive_in_cluster(free_bar);
                        if (more) {
                            if (!__all_sync(0xffffffffu, ready)) {
                                ok = wait_step(done0 + 8u * st.i, st.ph, abort_flag, p.err, kDevErrTimeoutEpilogue);
                                ok = __all_sync(0xffffffffu, ok);
                                if (!ok) break;
                            }
                            tc_fence_after();
                            tmem_ld_32x32b_x32(t0 + buf.i * BN, v[0]);
                        }
                        add_scaled<BROWS>(acc + c * 16, v[c & 1], s2, cols + c * 128);
                    }
                }
                if (!ok) break;
            }
            if (!ok) break;
            if (p.out_f32)
                store_rows<true, kCols>(acc, stg, lane, static_cast<uint8_t*>(p.D), p.ldd, w.drow + in_tile, w.dend, col, p.n,
                                 p.d_vec != 0);
            else
                store_rows<false, kCols>(acc, stg, lane, static_cast<uint8_t*>(p.D), p.ldd, w.drow + in_tile, w.dend, col, p.n,
                                  p.d_vec != 0);
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

template <int BN, bool BROWS>
cudaError_t launch(const F8Launch& a, cudaStream_t stream) {
    using R = Ring<BN>;
    CUtensorMap mA, mB;
    if (!encode_f8(&mA, a.A, a.k, a.rows_a, a.lda, kHalfRows) || !encode_f8(&mB, a.Bt, a.k, a.rows_b, a.ldb, BN / 2))
        return cudaErrorInvalidValue;
    F8Params p = f8_params(a, 256, BN);
    const int64_t units = a.group_mode == GEMM_GROUP_ROWS ? static_cast<int64_t>(p.pieces) * p.tiles_n
                                                          : static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.groups;
    if (units > INT32_MAX) return cudaErrorInvalidValue;
    int64_t pairs = a.pairs > 0 ? a.pairs : a.num_sms / 2;
    if (pairs > units) pairs = units;
    if (pairs < 1) pairs = 1;
    const void* kern = reinterpret_cast<const void*>(f8_tc2_kernel<BN, BROWS>);
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
    uint32_t idesc = idesc_f8(a.a_type, a.b_type, 256, BN);
    void* args[] = {&mA, &mB, &p, &idesc};
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
    p.pieces = static_cast<int>(a.m / bm + (a.groups < a.m ? a.groups : a.m));   // each group may end in a part of a tile
    p.out_f32 = a.out_f32 ? 1 : 0;
    p.d_vec = reinterpret_cast<uintptr_t>(a.D) % 16 == 0 && (a.ldd * (a.out_f32 ? 4 : 2)) % 16 == 0;
    return p;
}

cudaError_t launch_f8_tc2(const F8Launch& a, cudaStream_t stream) {
    const bool rows = a.b_scale_mode == GEMM_SCALE_ROWS;
    if (a.bn == 128) return rows ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
    return rows ? launch<256, true>(a, stream) : launch<256, false>(a, stream);
}

}  // namespace gemm
