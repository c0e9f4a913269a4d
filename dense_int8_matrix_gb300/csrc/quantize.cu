// Quantisation to FP8 with a scale for each block of 128.  GB300, 8192 x 8192
// bfloat16: rows 39 us (78 % of the measured copy rate), 128 x 128 blocks 45
// (67 %), transposed columns 46 (65 %); fp32 54, 57 and 56 us (88 to 92 %).  Rows
// of 8191: 65, 106 and 105 us (fp32 73, 109 and 109); of 1001 and 5003 elements
// rows 34 to 38 %, blocks 20 to 23 %, columns 22 to 24 %.
#include "f8.cuh"
#include "ptx.cuh"

namespace gemm {

namespace {

// 1 x 128 blocks: half a warp takes one block of one row, eight values per
// lane; a warp takes eight neighbouring blocks of a row, all loads first.
// Reads every element once and writes a byte for it: bound by DRAM.
constexpr int kRowBlocks = 8;   // blocks of a row per warp
template <typename T, int F8, bool VEC>
__global__ void __launch_bounds__(256) quant_rows_kernel(const F8Quant p, bool qvec) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr float kStep = F8 == GEMM_F8_E4M3 ? kE4M3Step : kE5M2Step;
    constexpr int kLoads = kRowBlocks / 2;
    const int64_t kb = (p.cols + kF8Block - 1) / kF8Block;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= p.rows) return;   // whole warps
    const T* x = static_cast<const T*>(p.X) + row * p.ldx;
    uint8_t* q = p.Q + row * p.ldq;
    const int half = (threadIdx.x >> 4) & 1, sub = threadIdx.x & 15;
    for (int64_t b0 = static_cast<int64_t>(blockIdx.y) * kRowBlocks; b0 < kb; b0 += static_cast<int64_t>(gridDim.y) * kRowBlocks) {
        Vec8<T> v[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) v[i] = load8<VEC>(x, (b0 + 2 * i + half) * kF8Block + sub * 8, p.cols);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int64_t b = b0 + 2 * i + half, c = b * kF8Block + sub * 8;
            float f[8];
            v[i].get(f);
            float a = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(f[j]));
            const float s = block_scale(half_warp_max(a), kStep);   // every lane takes part in the shuffles
            const float inv = __frcp_rn(s);
            if (b < kb) {
                store8_bytes(q, c, p.cols, qvec, f8x4<F8>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                             f8x4<F8>(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
                if (sub == 0) p.scale[b * p.rows + row] = s;
            }
        }
    }
}

// 128 x 128 blocks: one CTA per block; sixteen lanes cover 128 columns, a
// thread takes eight rows.
template <typename T, int F8, bool VEC>
__global__ void __launch_bounds__(256) quant_blocks_kernel(const F8Quant p, bool qvec) {
    __shared__ float red[8];
    pdl_launch_dependents();
    pdl_wait();
    constexpr float kStep = F8 == GEMM_F8_E4M3 ? kE4M3Step : kE5M2Step;
    const int64_t kb = (p.cols + kF8Block - 1) / kF8Block;
    const int64_t rb = blockIdx.x / kb, b = blockIdx.x - rb * kb;
    const int64_t c = b * kF8Block + (threadIdx.x & 15) * 8;
    Vec8<T> v[8];
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = rb * kF8Block + (threadIdx.x >> 4) + 16 * i;
        if (row < p.rows)
            v[i] = load8<VEC>(static_cast<const T*>(p.X) + row * p.ldx, c, p.cols);
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
    const float s = block_scale(a, kStep);
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
    int before = 0;   // padded blocks of the groups before these 32
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
// that a column's eight values pack into eight bytes of shared memory; the
// bytes leave as 128-byte rows.  The tile's 8-byte pieces are swizzled by the
// column group, so that neither side has bank conflicts beyond its width.
template <typename T, int F8, bool VEC>
__global__ void __launch_bounds__(256) quant_cols_kernel(const F8Quant p) {
    __shared__ __align__(16) uint8_t tile[kF8Block * kF8Block];
    __shared__ __align__(16) float red[8][kF8Block];
    __shared__ __align__(16) float inverse[kF8Block];
    pdl_launch_dependents();
    pdl_wait();
    constexpr float kStep = F8 == GEMM_F8_E4M3 ? kE4M3Step : kE5M2Step;
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
                v[i] = load8<VEC>(static_cast<const T*>(p.X) + (row + r) * p.ldx, c, p.cols);
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
        if (lane < 16) {
            *reinterpret_cast<float4*>(&red[warp][cg * 8]) = make_float4(am[0], am[1], am[2], am[3]);
            *reinterpret_cast<float4*>(&red[warp][cg * 8 + 4]) = make_float4(am[4], am[5], am[6], am[7]);
        }
        __syncthreads();
        if (threadIdx.x < kF8Block) {   // one thread per column
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) a = fmaxf(a, red[w][threadIdx.x]);
            const float s = block_scale(a, kStep);
            inverse[threadIdx.x] = __frcp_rn(s);
            if (c0 + threadIdx.x < p.cols) p.scale[static_cast<int64_t>(pb) * p.cols + c0 + threadIdx.x] = s;
        }
        __syncthreads();
        float f[8][8], inv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i].get(f[i]);
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const float4 x = *reinterpret_cast<const float4*>(&inverse[cg * 8 + j]);
            inv[j] = x.x; inv[j + 1] = x.y; inv[j + 2] = x.z; inv[j + 3] = x.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint2*>(tile + (cg * 8 + j) * kF8Block + ((rg ^ cg) << 3)) =
                make_uint2(f8x4<F8>(f[0][j] * inv[j], f[1][j] * inv[j], f[2][j] * inv[j], f[3][j] * inv[j]),
                           f8x4<F8>(f[4][j] * inv[j], f[5][j] * inv[j], f[6][j] * inv[j], f[7][j] * inv[j]));
        __syncthreads();
        // eight lanes write one column's 128 bytes
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = (threadIdx.x >> 3) + 32 * i, part = threadIdx.x & 7, g = col >> 3;
            uint4 x = *reinterpret_cast<const uint4*>(tile + col * kF8Block + (((2 * part) ^ (g & ~1)) << 3));
            if (g & 1) x = make_uint4(x.z, x.w, x.x, x.y);
            if (c0 + col < p.cols)
                *reinterpret_cast<uint4*>(p.Q + (c0 + col) * p.ldq + static_cast<int64_t>(pb) * kF8Block + part * 16) = x;
        }
        __syncthreads();   // the tile and the column maxima are reused
    }
}

template <typename T>
bool vec_ok(const void* p, int64_t pitch) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (pitch * sizeof(T)) % 16 == 0;
}

bool q_vec(const F8Quant& q) { return reinterpret_cast<uintptr_t>(q.Q) % 8 == 0 && q.ldq % 8 == 0; }

struct RowsForm {
    template <typename T, int F8, bool VEC>
    static cudaError_t launch(const F8Quant& q, cudaStream_t stream) {
        const int64_t gx = (q.rows + 7) / 8, gy = (q.cols + kF8Block * kRowBlocks - 1) / (kF8Block * kRowBlocks);
        return launch_chained(quant_rows_kernel<T, F8, VEC>,
                              dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy < 65535 ? gy : 65535)), 256, 0, stream, q,
                              q_vec(q));
    }
};

struct BlocksForm {
    template <typename T, int F8, bool VEC>
    static cudaError_t launch(const F8Quant& q, cudaStream_t stream) {
        const int64_t grid = ((q.rows + kF8Block - 1) / kF8Block) * ((q.cols + kF8Block - 1) / kF8Block);
        if (grid > INT32_MAX) return cudaErrorInvalidValue;
        return launch_chained(quant_blocks_kernel<T, F8, VEC>, dim3(static_cast<unsigned>(grid)), 256, 0, stream, q, q_vec(q));
    }
};

struct ColsForm {
    template <typename T, int F8, bool VEC>
    static cudaError_t launch(const F8Quant& q, cudaStream_t stream) {
        const int64_t gx = (q.cols + kF8Block - 1) / kF8Block, gy = q.kp / kF8Block;
        return launch_chained(quant_cols_kernel<T, F8, VEC>,
                              dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy < 65535 ? gy : 65535)), 256, 0, stream, q);
    }
};

template <typename Form, typename T, int F8>
cudaError_t by_alignment(const F8Quant& q, cudaStream_t stream) {
    return vec_ok<T>(q.X, q.ldx) ? Form::template launch<T, F8, true>(q, stream) : Form::template launch<T, F8, false>(q, stream);
}

template <typename Form>
cudaError_t quantise(const F8Quant& q, cudaStream_t stream) {
    const bool e4 = q.f8_type == GEMM_F8_E4M3;
    if (q.x_type == GEMM_DTYPE_BF16)
        return e4 ? by_alignment<Form, __nv_bfloat16, GEMM_F8_E4M3>(q, stream)
                  : by_alignment<Form, __nv_bfloat16, GEMM_F8_E5M2>(q, stream);
    return e4 ? by_alignment<Form, float, GEMM_F8_E4M3>(q, stream) : by_alignment<Form, float, GEMM_F8_E5M2>(q, stream);
}

}  // namespace

cudaError_t launch_f8_quant_rows(const F8Quant& q, cudaStream_t stream) { return quantise<RowsForm>(q, stream); }
cudaError_t launch_f8_quant_blocks(const F8Quant& q, cudaStream_t stream) { return quantise<BlocksForm>(q, stream); }
cudaError_t launch_f8_quant_cols(const F8Quant& q, cudaStream_t stream) { return quantise<ColsForm>(q, stream); }

}  // namespace gemm
