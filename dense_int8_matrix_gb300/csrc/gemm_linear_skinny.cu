// bfloat16 product with bias, activation and residual on small tiles: few rows
// (decode batches), and products with too few 256 x 256 tiles for the GPU.
//
// Computed as D^T: a CTA's tile is 128 columns of D (the MMA's M side, from B,
// the weights) by NT rows (its N side, from A; NT in {16, 32, 64, 128}).  Per K
// step of 64 a 16 KiB box of B and NT * 128 bytes of A go through a
// shared-memory ring, and four MMAs (K = 16) add them up in TMEM; chunks of K
// join fp32 sums in registers (see set_chunks in gemm_linear_tc2.cu).
//
// With few tiles a cluster of split_k CTAs shares a tile along K.  Each sends
// its sums to the CTAs that finish them (one share of the rows each) through
// distributed shared memory, and these add them up in rank order: no scratch,
// no second launch, and the same bits every time.  Then bias, activation and
// residual are applied once, to the joined sums.
//
// Bound by DRAM for few rows: 1 x 8192 x 8192 25.4 us, 5.3 TB/s, 64 rows 28; without
// the split 223 us.  Otherwise by a fixed part of 4 to 8 us around few K steps
// (1024^3 8.6 us).
//
// Operands that lie across K (GEMM_FORM_NN, GEMM_FORM_TN) are multiplied
// MN-major, as in gemm_linear_tc2.cu.  (Tiles of 32 rows spill 56 bytes, of 128 rows 8.)
#include <cuda_runtime.h>

#include <cstring>

#include "internal.h"
#include "linear.cuh"

namespace gemm {

namespace {

constexpr int kTileCols = 128;                         // columns of D per tile
constexpr int kWBytes = kTileCols * 128;
constexpr int kCtrlBytes = 512;

template <int NT>
struct Config {
    // epilogue warps per lane quarter and rows of A per thread: at most 32, so
    // that several warps share a scheduler and hide each other's waits
    static constexpr int PARTS = NT == 16 ? 1 : NT == 128 ? 4 : 2;
    static constexpr int EPI_WARPS = 4 * PARTS;
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int ROWS = NT / PARTS;
    static constexpr int A_BYTES = NT * 128;
    static constexpr int STAGE = kWBytes + A_BYTES;
    static constexpr int STAGES = NT == 16 ? 6 : NT == 32 ? 5 : NT == 64 ? 8 : 6;
    static constexpr int TMEM = 2 * NT;                // two accumulators
    static constexpr int PER_SM = NT >= 64 ? 1 : 2;
    static constexpr size_t SMEM = static_cast<size_t>(STAGES) * STAGE + kCtrlBytes + 1024;
    // after the products the ring holds the sums of a split tile and, for tiles
    // that leave in blocks, the warps' staging buffers
    static constexpr int SUMS = NT * kTileCols * 4;
    static constexpr bool BLOCKS = NT >= 64;
    static_assert(STAGES * STAGE >= SUMS + (BLOCKS ? EPI_WARPS * kStageRowsBytes : 0), "the sums fit in the ring");
    static_assert(SMEM <= (PER_SM == 1 ? 227 : 113) * 1024 && SMEM > 24 * 1024, "one or two CTAs per SM");
};

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// One operand's boxes of a step: `row` its first row, `rows` of them.
__device__ __forceinline__ void load_operand(uint32_t dst, const void* map, bool mn, int row, int rows, int kb, uint32_t bar,
                                             uint64_t policy) {
    if (mn) {
        tma_load_2d(dst, map, row, kb * kLinBK, bar, policy);
        if (rows > 64) tma_load_2d(dst + kLinBoxBytes, map, row + 64, kb * kLinBK, bar, policy);
    } else {
        tma_load_2d(dst, map, kb * kLinBK, row, bar, policy);
    }
}

// f(integral constant of the call's GEMM_ACT_*): the kernels are as many as
// there are tiles, the epilogue branches once.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F f) {
#define GEMM_ACT_CASE(ACT) case ACT: f(std::integral_constant<int, ACT>{}); break;
    switch (act) {
        GEMM_ACT_CASE(GEMM_ACT_RELU)
        GEMM_ACT_CASE(GEMM_ACT_GELU)
        GEMM_ACT_CASE(GEMM_ACT_GELU_TANH)
        GEMM_ACT_CASE(GEMM_ACT_SILU)
        GEMM_ACT_CASE(GEMM_ACT_RELU | GEMM_ACT_GRADIENT)
        GEMM_ACT_CASE(GEMM_ACT_GELU | GEMM_ACT_GRADIENT)
        GEMM_ACT_CASE(GEMM_ACT_GELU_TANH | GEMM_ACT_GRADIENT)
        GEMM_ACT_CASE(GEMM_ACT_SILU | GEMM_ACT_GRADIENT)
        default: f(std::integral_constant<int, GEMM_ACT_NONE>{}); break;
    }
#undef GEMM_ACT_CASE
}

template <int NT>
__global__ void __launch_bounds__(Config<NT>::THREADS, Config<NT>::PER_SM)
    linear_skinny_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, const LinearParams p,
                         const uint32_t idesc, const int split, const int act) {
    using R = Config<NT>;
    constexpr int kStages = R::STAGES, kRows = R::ROWS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t sW = base;
    const uint32_t sA = base + kStages * kWBytes;
    uint8_t* ctrl = smem_raw + (base - raw) + kStages * R::STAGE;
    const uint32_t full0 = smem_u32(ctrl);
    const uint32_t done0 = full0 + 8u * kStages;      // a stage has been multiplied
    const uint32_t accf0 = done0 + 8u * kStages;      // an accumulator is complete
    const uint32_t acce0 = accf0 + 16u;               // an accumulator has been read
    constexpr int kBars = 2 * kStages + 4;
    static_assert(8 * kBars + 8 <= kCtrlBytes && kBars <= 32, "barriers fit, one per lane");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * kBars);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        if (lane < kBars) mbar_init(full0 + 8u * lane, lane >= 2 * kStages + 2 ? R::EPI_WARPS : 1);
        if (lane == 0) {
            tma_prefetch_desc(&tmW);
            tma_prefetch_desc(&tmA);
            *abort_flag = 0u;
        }
        fence_barrier_init();
    }
    const int rank = static_cast<int>(blockIdx.x) % split;
    const int id = static_cast<int>(blockIdx.x) / split;
    const int row0 = id % p.tiles_m * NT, col0 = id / p.tiles_m * kTileCols;
    const int kb_lo = static_cast<int>(static_cast<int64_t>(p.num_kb) * rank / split);
    const int steps = static_cast<int>(static_cast<int64_t>(p.num_kb) * (rank + 1) / split) - kb_lo;
    // TMEM is taken only once the kernel before has ended, so that neither
    // waits for the other's.
    pdl_wait();
    __syncthreads();
    // the MMA warp and the epilogue wait for TMEM's address; the loads start
    // without it
    const auto tmem_ready = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 + 32 * R::EPI_WARPS) : "memory"); };
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), R::TMEM);
        tmem_relinquish();
        pdl_launch_dependents();   // with this CTA's TMEM taken
        tc_fence_before();
    }
    if (warp == 1 || warp >= 4) {
        tmem_ready();
        tc_fence_after();
    }
    const uint32_t tmem = *tmem_slot;   // (the loading warp does not use it)

    uint64_t acc[kRows / 2];   // pairs of rows of A, of column lane of the warp's 32
#pragma unroll
    for (int j = 0; j < kRows / 2; ++j) acc[j] = 0;

    if (warp == 0) {
        // ---------------------------------------------------- operand loads --
        const uint64_t polw = p.tiles_m == 1 ? policy_evict_first() : policy_evict_normal();
        const uint64_t pola = policy_evict_last();
        Turn<kStages> at;
        int issued = 0;
        for (; issued < steps; ++issued) {
            if (!wait_warp(done0 + 8u * at.i, at.ph ^ 1u, abort_flag, p.err, kDevErrTimeoutProducer)) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(full0 + 8u * at.i, R::STAGE);
                load_operand(sW + at.i * kWBytes, &tmW, p.mn_b, col0, kTileCols, kb_lo + issued, full0 + 8u * at.i, polw);
                load_operand(sA + at.i * R::A_BYTES, &tmA, p.mn_a, row0, NT, kb_lo + issued, full0 + 8u * at.i, pola);
            }
            __syncwarp();
            at.next();
        }
        if (issued < steps)   // after a time-out the copies still in flight land before the CTA ends
            for (int j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
                wait_bounded(full0 + 8u * (j % kStages), (j / kStages) & 1u, nullptr, p.err, kDevErrTimeoutTeardown);
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMAs --
        Turn<kStages> st;
        Turn<2> buf;
        const uint32_t step_w = desc_step(p.mn_b), step_a = desc_step(p.mn_a);
        int left = 0, kb = 0;   // steps of the running chunk that remain
        for (; kb < steps; ++kb) {
            const bool fresh = left == 0;
            if (fresh) {
                left = min(p.chunk, steps - kb);
                if (!wait_warp(acce0 + 8u * buf.i, buf.ph ^ 1u, abort_flag, p.err, kDevErrTimeoutMma)) break;
            }
            if (!wait_warp(full0 + 8u * st.i, st.ph, abort_flag, p.err, kDevErrTimeoutMma)) break;
            tc_fence_after();
            const uint64_t wd = smem_desc_linear(sW + st.i * kWBytes, p.mn_b);
            const uint64_t ad = smem_desc_linear(sA + st.i * R::A_BYTES, p.mn_a);
            --left;
            if (elect_one()) {
#pragma unroll
                for (uint32_t kk = 0; kk < kLinBK / kLinMmaK; ++kk)
                    mma_bf16<1>(tmem + buf.i * NT, wd + kk * step_w, ad + kk * step_a, idesc, fresh && kk == 0 ? 0u : 1u);
                mma_commit(done0 + 8u * st.i);
                if (left == 0) mma_commit(accf0 + 8u * buf.i);
            }
            __syncwarp();
            st.next();
            if (left == 0) buf.next();
        }
        // the epilogue sees the last chunk complete; after a time-out wait here
        // for the MMAs that were issued
        if (kb < steps && kb > 0)
            wait_bounded(done0 + 8u * ((kb - 1) % kStages), ((kb - 1) / kStages) & 1u, nullptr, p.err, kDevErrTimeoutTeardown);
    } else if (warp >= 4) {
        // --------------------------------------------------- add the chunks --
        const int q = warp & 3, h = (warp - 4) >> 2;   // lane quarter, part of the rows
        const uint32_t t0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * kRows;
        Turn<2> buf;
        if (rank == 0) {   // (rows of this part of the tile, whichever CTA finishes them)
            if (act >= GEMM_ACT_GRADIENT)
                prefetch_rows<true>(p, lane, row0 + h * kRows, col0 + q * 32, 32);
            else
                prefetch_rows<false>(p, lane, row0 + h * kRows, col0 + q * 32, 32);
        }
        for (int kb = 0; kb < steps; kb += p.chunk) {
            if (!wait_warp(accf0 + 8u * buf.i, buf.ph, abort_flag, p.err, kDevErrTimeoutEpilogue)) break;
            tc_fence_after();
            uint32_t v[kRows];
            load_tmem(t0 + buf.i * NT, v);
            wait_tmem(v);
            tc_fence_before();
            if (lane == 0) mbar_arrive(acce0 + 8u * buf.i);
#pragma unroll
            for (int j = 0; j < kRows / 2; ++j) acc[j] = add2(acc[j], pair_of(v[2 * j], v[2 * j + 1]));
            buf.next();
        }
    }

    // ----------------------------------------------------------- join, finish --
    // The ring is idle: every step has been multiplied (or the call has failed).
    const int q = warp & 3, h = (warp - 4) >> 2;
    float v[kRows];
#pragma unroll
    for (int j = 0; j < kRows / 2; ++j) unpair(acc[j], v[2 * j], v[2 * j + 1]);
    int first = h * kRows, count = kRows;   // this thread's rows of the tile
    if (split > 1) {
        // Row r of A is finished by CTA r / share, whose ring (idle in every
        // CTA after the first barrier) holds sums[sender][row][column].
        const int share = NT / split, shift = 31 - __clz(share);   // a power of two
        cluster_barrier();
        if (warp >= 4) {
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int r = first + j, owner = r >> shift;
                st_cluster_f32(peer_address(base + ((rank * share + r - owner * share) * kTileCols + q * 32 + lane) * 4, owner), v[j]);
            }
        }
        cluster_barrier();
        count = share / R::PARTS;
        first = rank * share + h * count;
        if (warp >= 4) {
#pragma unroll
            for (int j = 0; j < kRows / 2; ++j)   // (a split leaves half of a thread's rows at most)
                if (j < count) {
                    v[j] = 0.f;
                    for (int s = 0; s < split; ++s)
                        v[j] += ld_shared_f32(base + ((s * share + h * count + j) * kTileCols + q * 32 + lane) * 4);
                }
        }
    }
    if (warp >= 4) {
        const int row = row0 + first, rows = min(count, p.m - row), col = col0 + q * 32;
        if constexpr (R::BLOCKS) {
            // lane = column: the block is turned on its way through the staging buffer
            const uint32_t stg = base + R::SUMS + (warp - 4) * kStageRowsBytes;
#pragma unroll
            for (int j = 0; j < kRows; ++j)
                if (j < count) st_shared_u32(stg + j * 128 + (((lane >> 2) ^ (j & 7)) << 4) + (lane & 3) * 4, __float_as_uint(v[j]));
            __syncwarp();
            if (rows > 0 && col < p.n)
                with_activation(act, [&](auto a) { finish<decltype(a)::value>(p, stg, lane, row, row + rows, col); });
        } else if (rows > 0) {
            with_activation(act, [&](auto a) {
                if (p.out_f32)
                    finish_column<true, decltype(a)::value, kRows>(p, row, rows, col + lane, v);
                else
                    finish_column<false, decltype(a)::value, kRows>(p, row, rows, col + lane, v);
            });
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, R::TMEM);
}

template <int NT>
cudaError_t launch(const LinearLaunch& a, cudaStream_t stream) {
    using R = Config<NT>;
    if (a.form == GEMM_FORM_TN && NT < 64) return cudaErrorInvalidValue;   // (MN-major boxes of A hold 64 rows)
    CUtensorMap mW, mA;
    if (!encode_operand(&mW, a, true, kTileCols) || !encode_operand(&mA, a, false, NT)) return cudaErrorInvalidValue;
    LinearParams p = linear_params(a, NT, kTileCols);
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    if (tiles * a.split_k > INT32_MAX) return cudaErrorInvalidValue;
    const void* kern = reinterpret_cast<const void*>(linear_skinny_kernel<NT>);
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
    uint32_t idesc = idesc_linear(p.mn_b, p.mn_a, kTileCols, NT);
    int split = a.split_k, act = a.act | (a.grad ? GEMM_ACT_GRADIENT : 0);
    void* args[] = {&mW, &mA, &p, &idesc, &split, &act};
    const cudaError_t r = cudaLaunchKernelExC(&cfg, kern, args);
    return r != cudaSuccess ? r : cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_skinny(const LinearLaunch& a, cudaStream_t stream) {
    switch (a.bm) {
        case 16: return launch<16>(a, stream);
        case 32: return launch<32>(a, stream);
        case 64: return launch<64>(a, stream);
        default: return launch<128>(a, stream);
    }
}

}  // namespace gemm
