// Quantisation to FP8 with a scale for each block of 128.
#include "f8.cuh"
#include "ptx.cuh"

namespace gemm {

namespace {

// 1 x 128 blocks: half a warp takes one block of one row, eight values per
// lane.  Reads rows * cols elements, writes as many bytes: bound by DRAM.
template <typename T, int F8>
__global__ void __launch_bounds__(256) quant_rows_kernel(const F8Quant p, bool vec, bool qvec) {
    const int64_t kb = (p.cols + kF8Block - 1) / kF8Block;
    const int64_t items = p.rows * kb;
    constexpr float M = F8 == GEMM_F8_E4M3 ? kE4M3Max : kE5M2Max;
    const int sub = threadIdx.x & 15;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (blockDim.x / 16);
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 16); i0 < items; i0 += stride) {
        const int64_t i = i0 + threadIdx.x / 16;
        const bool on = i < items;   // uniform in each half warp; every lane takes part in the shuffles
        const int64_t row = on ? i / kb : 0, b = on ? i - row * kb : 0;
        const int64_t c = on ? b * kF8Block + sub * 8 : p.cols;
        float f[8];
        load8(static_cast<const T*>(p.X) + row * p.ldx, c, p.cols, vec).get(f);
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(f[j]));
        const float s = block_scale(half_warp_max(a), M);
        const float inv = __frcp_rn(s);
        if (!on) continue;
        store8_bytes(p.Q + row * p.ldq, c, p.cols, qvec, f8x4<F8>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                     f8x4<F8>(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
        if (sub == 0) p.scale[b * p.rows + row] = s;
    }
}

// 128 x 128 blocks: one CTA per block; sixteen lanes cover 128 columns, a
// thread takes eight rows.
template <typename T, int F8>
__global__ void __launch_bounds__(256) quant_blocks_kernel(const F8Quant p, bool vec, bool qvec) {
    __shared__ float red[8];
    constexpr float M = F8 == GEMM_F8_E4M3 ? kE4M3Max : kE5M2Max;
    const int64_t kb = (p.cols + kF8Block - 1) / kF8Block;
    const int64_t rb = blockIdx.x / kb, b = blockIdx.x - rb * kb;
    const int64_t c = b * kF8Block + (threadIdx.x & 15) * 8;
    Vec8<T> v[8];
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = rb * kF8Block + (threadIdx.x >> 4) + 16 * i;
        if (row < p.rows)
            v[i] = load8(static_cast<const T*>(p.X) + row * p.ldx, c, p.cols, vec);
        else
            v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        v[i].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(f[j]));
    }
    a = warp_max(a);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, red[i]);
    const float s = block_scale(a, M);
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = rb * kF8Block + (threadIdx.x >> 4) + 16 * i;
        if (row >= p.rows) continue;
        float f[8];
        v[i].get(f);
        store8_bytes(p.Q + row * p.ldq, c, p.cols, qvec, f8x4<F8>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                     f8x4<F8>(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
    }
    if (threadIdx.x == 0) p.scale[blockIdx.x] = s;
}

// Which rows the padded block `pb` of 128 columns of Q covers: [row, row + n),
// n <= 128; n < 0 when the block lies behind the last group.  The groups'
// padded sizes are summed by one warp, 32 groups at a time.
__device__ void find_block_rows(const F8Quant& p, int pb, int lane, int& row, int& n) {
    const int rows = static_cast<int>(p.rows);
    if (p.offsets == nullptr) {
        row = pb * kF8Block;
        n = row < rows ? min(kF8Block, rows - row) : -1;
        return;
    }
    int before = 0;   // padded blocks of the groups before this round
    row = 0;
    n = -1;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
        int lo = 0, hi = 0;
        if (g0 + lane < p.groups) group_rows(p.offsets, g0 + lane, rows, lo, hi);
        const int nb = (hi - lo + kF8Block - 1) / kF8Block;
        int sum = nb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += t;
        }
        const int first = before + sum - nb;
        const unsigned hit = __ballot_sync(0xffffffffu, pb >= first && pb < first + nb);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int r = lo + (pb - first) * kF8Block;
            row = __shfl_sync(0xffffffffu, r, src);
            n = __shfl_sync(0xffffffffu, min(kF8Block, hi - r), src);
            return;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
        if (before > pb) return;
    }
}

// Transposed 1 x 128 blocks: one CTA turns 128 rows x 128 columns of X into
// 128 rows of 128 bytes of Q.  A thread holds eight rows of eight columns, so
// that a column's eight values pack into two words of shared memory; the
// bytes leave as 128-byte rows.
constexpr int kColsPitch = 144;   // bytes per column in shared memory (16-byte aligned, spreads the banks)
template <typename T, int F8>
__global__ void __launch_bounds__(256) quant_cols_kernel(const F8Quant p, bool vec) {
    __shared__ __align__(16) uint8_t tile[kF8Block * kColsPitch];
    __shared__ float red[8][kF8Block];
    constexpr float M = F8 == GEMM_F8_E4M3 ? kE4M3Max : kE5M2Max;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kF8Block;
    for (int pb = blockIdx.y; pb < p.kp / kF8Block; pb += gridDim.y) {
        int row, n;
        find_block_rows(p, pb, lane, row, n);
        if (n < 0) return;   // behind the last group, as every later block is
        const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
        const int64_t c = c0 + cg * 8;
        Vec8<T> v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = rg * 8 + i;
            if (r < n)
                v[i] = load8(static_cast<const T*>(p.X) + (row + r) * p.ldx, c, p.cols, vec);
            else
                v[i].zero();
        }
        float am[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) am[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[8];
            v[i].get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) am[j] = fmaxf(am[j], fabsf(f[j]));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) am[j] = fmaxf(am[j], __shfl_xor_sync(0xffffffffu, am[j], 16));
        if (lane < 16)
#pragma unroll
            for (int j = 0; j < 8; ++j) red[warp][cg * 8 + j] = am[j];
        __syncthreads();
        float s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) a = fmaxf(a, red[w][cg * 8 + j]);
            s[j] = block_scale(a, M);
        }
        if (rg == 0)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < p.cols) p.scale[static_cast<int64_t>(pb) * p.cols + c + j] = s[j];
        uint32_t w0[8], w1[8];
        float f[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i].get(f[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float inv = __frcp_rn(s[j]);
            w0[j] = f8x4<F8>(f[0][j] * inv, f[1][j] * inv, f[2][j] * inv, f[3][j] * inv);
            w1[j] = f8x4<F8>(f[4][j] * inv, f[5][j] * inv, f[6][j] * inv, f[7][j] * inv);
            *reinterpret_cast<uint2*>(tile + (cg * 8 + j) * kColsPitch + rg * 8) = make_uint2(w0[j], w1[j]);
        }
        __syncthreads();
        // eight lanes write one column's 128 bytes
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = (threadIdx.x >> 3) + 32 * i, part = threadIdx.x & 7;
            if (c0 + col < p.cols)
                *reinterpret_cast<uint4*>(p.Q + (c0 + col) * p.ldq + static_cast<int64_t>(pb) * kF8Block + part * 16) =
                    *reinterpret_cast<const uint4*>(tile + col * kColsPitch + part * 16);
        }
        __syncthreads();   // the tile and the column maxima are reused
    }
}

template <typename T>
bool vec_ok(const void* p, int64_t pitch) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (pitch * sizeof(T)) % 16 == 0;
}

template <typename T, int F8>
cudaError_t rows_launch(const F8Quant& q, cudaStream_t stream) {
    const int64_t items = q.rows * ((q.cols + kF8Block - 1) / kF8Block);
    const int64_t grid = (items + 15) / 16, cap = static_cast<int64_t>(q.num_sms) * 64;
    quant_rows_kernel<T, F8><<<static_cast<unsigned>(grid < cap ? grid : cap), 256, 0, stream>>>(
        q, vec_ok<T>(q.X, q.ldx), reinterpret_cast<uintptr_t>(q.Q) % 8 == 0 && q.ldq % 8 == 0);
    return cudaGetLastError();
}

template <typename T, int F8>
cudaError_t blocks_launch(const F8Quant& q, cudaStream_t stream) {
    const int64_t grid = ((q.rows + kF8Block - 1) / kF8Block) * ((q.cols + kF8Block - 1) / kF8Block);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    quant_blocks_kernel<T, F8><<<static_cast<unsigned>(grid), 256, 0, stream>>>(
        q, vec_ok<T>(q.X, q.ldx), reinterpret_cast<uintptr_t>(q.Q) % 8 == 0 && q.ldq % 8 == 0);
    return cudaGetLastError();
}

template <typename T, int F8>
cudaError_t cols_launch(const F8Quant& q, cudaStream_t stream) {
    const int64_t gx = (q.cols + kF8Block - 1) / kF8Block, gy = q.kp / kF8Block;
    quant_cols_kernel<T, F8><<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy < 65535 ? gy : 65535)), 256, 0,
                               stream>>>(q, vec_ok<T>(q.X, q.ldx));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_f8_quant_rows(const F8Quant& q, cudaStream_t stream) {
    const bool bf = q.x_type == GEMM_DTYPE_BF16, e4 = q.f8_type == GEMM_F8_E4M3;
    return bf ? (e4 ? rows_launch<__nv_bfloat16, GEMM_F8_E4M3>(q, stream) : rows_launch<__nv_bfloat16, GEMM_F8_E5M2>(q, stream))
              : (e4 ? rows_launch<float, GEMM_F8_E4M3>(q, stream) : rows_launch<float, GEMM_F8_E5M2>(q, stream));
}

cudaError_t launch_f8_quant_blocks(const F8Quant& q, cudaStream_t stream) {
    const bool bf = q.x_type == GEMM_DTYPE_BF16, e4 = q.f8_type == GEMM_F8_E4M3;
    return bf ? (e4 ? blocks_launch<__nv_bfloat16, GEMM_F8_E4M3>(q, stream) : blocks_launch<__nv_bfloat16, GEMM_F8_E5M2>(q, stream))
              : (e4 ? blocks_launch<float, GEMM_F8_E4M3>(q, stream) : blocks_launch<float, GEMM_F8_E5M2>(q, stream));
}

cudaError_t launch_f8_quant_cols(const F8Quant& q, cudaStream_t stream) {
    const bool bf = q.x_type == GEMM_DTYPE_BF16, e4 = q.f8_type == GEMM_F8_E4M3;
    return bf ? (e4 ? cols_launch<__nv_bfloat16, GEMM_F8_E4M3>(q, stream) : cols_launch<__nv_bfloat16, GEMM_F8_E5M2>(q, stream))
              : (e4 ? cols_launch<float, GEMM_F8_E4M3>(q, stream) : cols_launch<float, GEMM_F8_E5M2>(q, stream));
}

}  // namespace gemm
