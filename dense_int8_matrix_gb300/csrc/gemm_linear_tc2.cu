// bfloat16 product with bias, activation and residual on two-SM tiles
// (tcgen05 cta_group::2).
//
//   v = sum_kk A[i][kk] B[kk][j] + bias[j],  D = act(v) + residual, or v act'(Z) + residual
//
// A cluster of two CTAs computes a 256 x 256 tile (or a half, 256 x 128); each
// CTA loads its 128 rows of A and its half of the columns of B per K step with
// TMA, and tcgen05.mma (M = 256, N = 256, K = 16, four per step) adds them up in
// TMEM, in 32 bits.  The MMA truncates what it adds to an accumulator, an error
// that grows with K and always points to zero, so that a chunk of K at a time
// is added up there and the chunks in registers, rounded to nearest (set_chunks).  The two
// accumulators of 256 columns alternate: one is read while the next chunk, or
// the next tile, is multiplied.
//
// An operand whose rows lie along K (GEMM_FORM_NT) comes in boxes of 64 K
// elements by 128 rows.  The backward pass reads the same tensors along their
// other dimension: their boxes are 64 rows by 64 K elements, and the MMA takes
// them MN-major, so that nothing is ever transposed in memory.
//
// Bound by the tensor cores where K is long: 4096^3 81 us (1.70 PFLOP/s; 256 tiles on
// 76 pairs are 3.5 rounds), 8192^3 563 to 575 us (1.93 PFLOP/s, power limited), fp32
// output of 4096^3 87 us.  By the epilogue where K is short: about 4.3 us for a tile
// beside the next one's products, 9 with GELU (8192 x 1024 x 8192 80 us, 114 with GELU).
// GELU and its gradient spill 16 and 28 bytes.
//
// Roles: warp 0 loads operands, warp 1 of the even CTA issues the MMAs, warps 4
// to 11 take the sums through shared memory (so that rows leave in contiguous
// pieces, and residual and Z come in the same way) and finish them.
#include <cuda_runtime.h>

#include <cstring>

#include "internal.h"
#include "linear.cuh"

namespace gemm {

namespace {

constexpr int kThreads = 384;
constexpr int kStages = 6;
constexpr int kHalfRows = 128;                      // rows of A, and of B, per CTA and step
constexpr int kHalfBytes = kHalfRows * 128;
constexpr int kStage = 2 * kHalfBytes;
constexpr int kTileN = 256;
constexpr int kEpiWarps = 8;
constexpr int kCtrlBytes = 512;
constexpr size_t kSmem = static_cast<size_t>(kStages) * kStage + kEpiWarps * kStageRowsBytes + kCtrlBytes + 1024;
static_assert(kSmem <= 232448, "shared memory");

struct Unit {
    int row, col;   // first row and column of D
    bool half;      // 128 columns instead of 256
};

// The list of units that the pairs take in turn: whole tiles, and the tiles of
// a last round that would leave half of the pairs idle as two halves of 128
// columns each.
struct Units {
    int whole, count;   // units [0, whole) are tiles, the rest halves
};
__device__ __forceinline__ Units list_units(const LinearParams& p, int npairs) {
    const int tiles = p.tiles_m * p.tiles_n;
    Units x;
    x.whole = p.halves ? 0 : tiles / npairs * npairs;
    if (!p.halves && 2 * (tiles - x.whole) > npairs) x.whole = tiles;
    x.count = x.whole + 2 * (tiles - x.whole);
    return x;
}
__device__ __forceinline__ Unit unit_at(int u, const Units& list, const LinearParams& p) {
    Unit x;
    x.half = u >= list.whole;
    const int part = x.half ? (u - list.whole) & 1 : 0;
    if (x.half) u = list.whole + ((u - list.whole) >> 1);
    int tm, tn;
    tc_tile_coords(u, p.tiles_m, p.tiles_n, tm, tn);
    x.row = tm * 256;
    x.col = tn * kTileN + part * (kTileN / 2);
    return x;
}
// A half past D's last column has no steps.
__device__ __forceinline__ int steps_of(const Unit& w, const LinearParams& p) { return w.col < p.n ? p.num_kb : 0; }

// One operand's box of a step: `row` its first row, `kb` the step.
__device__ __forceinline__ void load_operand(uint32_t dst, const void* map, bool mn, int row, int kb, uint32_t bar,
                                             uint64_t policy) {
    if (mn) {
        load_2d_pair(dst, map, row, kb * kLinBK, bar, policy);
        load_2d_pair(dst + kLinBoxBytes, map, row + 64, kb * kLinBK, bar, policy);
    } else {
        load_2d_pair(dst, map, kb * kLinBK, row, bar, policy);
    }
}

// Adds 32 columns of a chunk to the running sums.
__device__ __forceinline__ void add_block(uint64_t* acc, const uint32_t (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = add2(acc[j], pair_of(v[2 * j], v[2 * j + 1]));
}
// 32 columns of running sums into the warp's staging buffer.
__device__ __forceinline__ void stage_block(uint32_t stg, int lane, const uint64_t* acc) {
    uint32_t r[32];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float a, b;
        unpair(acc[j], a, b);
        r[2 * j] = __float_as_uint(a);
        r[2 * j + 1] = __float_as_uint(b);
    }
    stage_rows32(stg, lane, r);
}

template <int ACT>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tc2_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const LinearParams p, const uint32_t idesc, const uint32_t idesc_half) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t sA = base;
    const uint32_t sB = base + kStages * kHalfBytes;
    const uint32_t sEpi = base + kStages * kStage;
    uint8_t* ctrl = smem_raw + (sEpi - raw) + kEpiWarps * kStageRowsBytes;
    const uint32_t full0 = smem_u32(ctrl);            // used in the even CTA
    const uint32_t done0 = full0 + 8u * kStages;      // a stage has been multiplied
    const uint32_t accf0 = done0 + 8u * kStages;      // an accumulator is complete
    const uint32_t acce0 = accf0 + 16u;               // used in the even CTA: an accumulator has been read
    const uint32_t last = acce0 + 16u;
    constexpr int kBars = 2 * kStages + 5;
    static_assert(8 * kBars + 8 <= kCtrlBytes, "barriers fit");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * kBars);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank_in_cluster();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (warp == 0) {
        if (lane < kBars) mbar_init(full0 + 8u * lane, lane == 2 * kStages + 2 || lane == 2 * kStages + 3 ? 2 * kEpiWarps : 1);
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmB);
            *abort_flag = 0u;
        }
        fence_barrier_init();
    }
    static_assert(kBars <= 32, "a barrier per lane");
    if (warp == 1) alloc_pair(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    cluster_barrier();   // barriers and TMEM of both CTAs are ready
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Units list = list_units(p, npairs);

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
            for (int u = pair; ok && u < list.count; u += npairs) {
                const Unit w = unit_at(u, list, p);
                const int steps = steps_of(w, p);
                const int ya = w.row + static_cast<int>(rank) * kHalfRows;
                // (a half's boxes bring 64 columns more than are multiplied)
                const int yb = w.col + static_cast<int>(rank) * (w.half ? kTileN / 4 : kTileN / 2);
                for (int kb = 0; kb < steps; ++kb, ++issued) {
                    // the stage is free once the step that was in it has been multiplied
                    if (!wait_warp(done0 + 8u * at.i, at.ph ^ 1u, abort_flag, p.err, kDevErrTimeoutProducer)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t fb = full_leader + 8u * at.i;
                        if (leader) mbar_arrive_expect_tx(full0 + 8u * at.i, 2 * kStage);
                        load_operand(sA + at.i * kHalfBytes, &tmA, p.mn_a, ya, kb, fb, pol);
                        load_operand(sB + at.i * kHalfBytes, &tmB, p.mn_b, yb, kb, fb, pol);
                    }
                    __syncwarp();
                    at.next();
                }
            }
            // after a time-out the copies still in flight land before the pair ends
            if (!ok && leader)
                for (uint32_t j = issued > kStages ? issued - kStages : 0u; j < issued; ++j)
                    wait_bounded(full0 + 8u * (j % kStages), (j / kStages) & 1u, nullptr, p.err, kDevErrTimeoutTeardown);
        } else if (warp == 1 && leader) {
            // ---------------------------------------------------------- MMAs --
            Turn<kStages> st;
            Turn<2> buf;
            bool ok = true;
            const uint32_t step_a = desc_step(p.mn_a), step_b = desc_step(p.mn_b);
            for (int u = pair; ok && u < list.count; u += npairs) {
                const Unit w = unit_at(u, list, p);
                const int steps = steps_of(w, p);
                const uint32_t desc = w.half ? idesc_half : idesc;
                int left = 0;   // steps of the running chunk that remain
                for (int kb = 0; kb < steps; ++kb) {
                    const bool fresh = left == 0;
                    if (fresh) {
                        left = min(kb == 0 ? p.first : p.chunk, steps - kb);
                        ok = wait_warp(acce0 + 8u * buf.i, buf.ph ^ 1u, abort_flag, p.err, kDevErrTimeoutMma);
                    }
                    ok = ok && wait_warp(full0 + 8u * st.i, st.ph, abort_flag, p.err, kDevErrTimeoutMma);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = smem_desc_linear(sA + st.i * kHalfBytes, p.mn_a);
                    const uint64_t bd = smem_desc_linear(sB + st.i * kHalfBytes, p.mn_b);
                    --left;
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t kk = 0; kk < kLinBK / kLinMmaK; ++kk)
                            mma_bf16<2>(tmem + buf.i * kTileN, ad + kk * step_a, bd + kk * step_b, desc, fresh && kk == 0 ? 0u : 1u);
                        commit_pair(done0 + 8u * st.i);
                        if (left == 0) commit_pair(accf0 + 8u * buf.i);
                    }
                    __syncwarp();
                    st.next();
                    if (left == 0) buf.next();
                }
            }
            if (elect_one()) commit_pair(last);
            __syncwarp();
            wait_bounded(last, 0u, nullptr, p.err, kDevErrTimeoutTeardown);
        }
    } else {
        // ---------------------------------------------------------- epilogue --
        more_registers<232>();
        pdl_wait();
        const int e = warp - 4, q = warp & 3, h = e >> 2;
        const uint32_t stg = sEpi + e * kStageRowsBytes;
        const uint32_t acce = peer_address(acce0, 0);
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        Turn<2> buf;
        bool ok = true;
        auto prefetch = [&](int u) {
            if (u >= list.count || !((ACT & GEMM_ACT_GRADIENT) != 0 || p.R)) return;
            const Unit w = unit_at(u, list, p);
            const int cols = w.half ? kTileN / 4 : kTileN / 2;
            prefetch_rows<(ACT & GEMM_ACT_GRADIENT) != 0>(p, lane, w.row + static_cast<int>(rank) * kHalfRows + q * 32,
                                                          w.col + h * cols, cols);
        };
        prefetch(pair);
        for (int u = pair; ok && u < list.count; u += npairs) {
            const Unit w = unit_at(u, list, p);
            const int steps = steps_of(w, p);
            if (steps == 0) continue;
            const int cols = w.half ? kTileN / 4 : kTileN / 2;   // of this warp
            const int row0 = w.row + static_cast<int>(rank) * kHalfRows + q * 32, col0 = w.col + h * cols;
            uint64_t acc[kTileN / 4];   // pairs of columns; the first half of them for a half
#pragma unroll
            for (int j = 0; j < kTileN / 4; ++j) acc[j] = 0;
            for (int kb = 0; kb < steps; kb += kb == 0 ? p.first : p.chunk) {
                ok = wait_warp(accf0 + 8u * buf.i, buf.ph, abort_flag, p.err, kDevErrTimeoutEpilogue);
                if (!ok) break;
                tc_fence_after();
                const uint32_t t0 = lanes + buf.i * kTileN + h * cols, free_bar = acce + 8u * buf.i;
                buf.next();
                // one block of 32 columns is added while the next is on its way
                uint32_t v[2][32];
                tmem_ld_32x32b_x32(t0, v[0]);
                wait_tmem(v[0]);
                tmem_ld_32x32b_x32(t0 + 32, v[1]);
                add_block(acc, v[0]);
                wait_tmem(v[1]);
                if (!w.half) {
                    tmem_ld_32x32b_x32(t0 + 64, v[0]);
                    add_block(acc + 16, v[1]);
                    wait_tmem(v[0]);
                    tmem_ld_32x32b_x32(t0 + 96, v[1]);
                    add_block(acc + 32, v[0]);
                    wait_tmem(v[1]);
                }
                // all columns are in registers: the accumulator is free
                tc_fence_before();
                if (lane == 0) arrive_in_cluster(free_bar);
                if (w.half)
                    add_block(acc + 16, v[1]);
                else
                    add_block(acc + 48, v[1]);
            }
            if (!ok) break;
            prefetch(u + npairs);
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
                if (row0 >= p.m || col0 + c >= p.n) break;   // (the whole warp alike)
                __syncwarp();   // the block before has been read out
                switch (c) {
                    case 0: stage_block(stg, lane, acc); break;
                    case 32: stage_block(stg, lane, acc + 16); break;
                    case 64: stage_block(stg, lane, acc + 32); break;
                    default: stage_block(stg, lane, acc + 48); break;
                }
                __syncwarp();
                finish<ACT>(p, stg, lane, row0, p.m, col0 + c);
            }
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

bool aligned_to(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

}  // namespace

bool encode_bf16(CUtensorMap* map, const void* ptr, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
    auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!enc) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(kLinBK), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_operand(CUtensorMap* map, const LinearLaunch& a, bool is_b, int box_rows) {
    const bool mn = is_b ? a.form != GEMM_FORM_NT : a.form == GEMM_FORM_TN;
    const void* ptr = is_b ? a.B : a.A;
    const int64_t rows = is_b ? a.n : a.m, ld = is_b ? a.ldb : a.lda;
    return mn ? encode_bf16(map, ptr, rows, a.k, ld, kLinBK) : encode_bf16(map, ptr, a.k, rows, ld, box_rows);
}

// K steps that are added up in TMEM.  Relative error of sums of products of normal
// values, fp32 output, against 64 bits: 4096 products in one chunk 4.4e-6 (a
// plain fp32 matrix product 6e-7), 131072 1.5e-4, and 8e-4 if all are positive;
// chunks of 512 keep it near 6e-7, and small tiles take them whatever the output
// (at most 2 % longer).  The two-SM tiles take 1024 for bfloat16 outputs, whose
// rounding is 2e-3: 8192^3 601 us with Z and GELU_TANH as with 2048, 639 with 512, as
// reading an accumulator holds the MMAs up.  A tile's first chunk is 1536: the
// one before it is finished in the time of its first two (4096^3 with GELU and
// residual 91 us, 95 with 1024).  Positive sums are short by 2.4e-6, one
// output in 1300 differs from the rounded exact sum (chunks of 2048: 5.7e-6, one in 800).
void set_chunks(const LinearLaunch& a, LinearParams* p) {
    const bool fine = a.out_f32 || a.bm < 256;
    p->chunk = (fine ? 512 : 1024) / kLinBK;
    p->first = (fine ? 512 : 1536) / kLinBK;
}

LinearParams linear_params(const LinearLaunch& a, int bm, int bn) {
    LinearParams p;
    p.bias = a.bias;
    p.R = a.R;
    p.Z = static_cast<__nv_bfloat16*>(a.Z);
    p.D = a.D;
    p.err = a.err;
    p.ldd = a.ldd;
    p.ldr = a.ldr;
    p.ldz = a.ldz;
    p.m = static_cast<int>(a.m);
    p.n = static_cast<int>(a.n);
    p.num_kb = static_cast<int>((a.k + kLinBK - 1) / kLinBK);
    p.tiles_m = static_cast<int>((a.m + bm - 1) / bm);
    p.tiles_n = static_cast<int>((a.n + bn - 1) / bn);
    p.out_f32 = a.out_f32;
    p.mn_a = a.form == GEMM_FORM_TN;
    p.mn_b = a.form != GEMM_FORM_NT;
    const int64_t es = a.out_f32 ? 4 : 2;
    p.vec = aligned_to(a.D, 16) && a.ldd * es % 16 == 0 && (!a.R || (aligned_to(a.R, 16) && a.ldr * es % 16 == 0)) &&
            (!a.Z || (aligned_to(a.Z, 16) && a.ldz % 8 == 0)) && aligned_to(a.bias, 16);
    p.pairs = aligned_to(a.D, 4) && a.ldd % 2 == 0 && (!a.R || (aligned_to(a.R, 4) && a.ldr % 2 == 0)) &&
              (!a.Z || (aligned_to(a.Z, 4) && a.ldz % 2 == 0));
    p.halves = false;
    set_chunks(a, &p);
    return p;
}

cudaError_t launch_linear_tc2(const LinearLaunch& a, cudaStream_t stream) {
    CUtensorMap mA, mB;
    if (!encode_operand(&mA, a, false, kHalfRows) || !encode_operand(&mB, a, true, kTileN / 2)) return cudaErrorInvalidValue;
    LinearParams p = linear_params(a, 256, kTileN);
    p.halves = a.bn == kTileN / 2;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    if (2 * tiles > INT32_MAX) return cudaErrorInvalidValue;
    int64_t pairs = a.pairs > 0 ? a.pairs : a.num_sms / 2;
    if (pairs < 1) pairs = 1;
    const int64_t use = p.halves || 2 * tiles <= pairs ? 2 * tiles : tiles;
    if (pairs > use) pairs = use;
    return by_activation(a, [&](auto act) -> cudaError_t {
        const void* kern = reinterpret_cast<const void*>(linear_tc2_kernel<decltype(act)::value>);
        const cudaError_t e = kernel_attrs_once(kern, static_cast<int>(kSmem), true);
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
        cfg.dynamicSmemBytes = kSmem;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        uint32_t idesc = idesc_linear(p.mn_a, p.mn_b, 256, kTileN), idesc_half = idesc_linear(p.mn_a, p.mn_b, 256, kTileN / 2);
        void* args[] = {&mA, &mB, &p, &idesc, &idesc_half};
        const cudaError_t r = cudaLaunchKernelExC(&cfg, kern, args);
        return r != cudaSuccess ? r : cudaGetLastError();
    });
}

}  // namespace gemm
