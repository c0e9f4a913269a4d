// RMS norm with the residual's addition and an 8-bit output, and its
// gradient.
//
//   h = x + r,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * w
//   dx = dr + rstd * (g - xhat * mean(g * xhat)),  g = dy * w, xhat = h * rstd
//   dw = sum over rows of dy * xhat
//
// Both are bound by DRAM: every element is read and written once.
#include "f8.cuh"
#include "ptx.cuh"

namespace gemm {

namespace {

// Sum (or largest) over the CTA; `red` is used by this call alone.
template <bool MAX>
__device__ __forceinline__ float cta_reduce(float v, float* red) {
    v = MAX ? warp_max(v) : warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
    return MAX ? warp_max(v) : warp_sum(v);
}

// One CTA per row; the row stays in registers (V vectors of eight values per
// thread, vector v of thread t at column 8 * (v * blockDim + t), so sixteen
// neighbouring lanes hold one block of 128 columns).  The mean square is
// taken of h as it is stored.
template <typename T, int V, bool I8>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormFwd p, bool vec, bool qvec, bool wvec) {
    __shared__ float red[2][32];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.X) + row * p.ldx;
    const T* r = p.R ? static_cast<const T*>(p.R) + row * p.ldr : nullptr;
    Vec8<T> h[V];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = 8 * (static_cast<int64_t>(v) * blockDim.x + threadIdx.x);
        h[v] = load8(x, c, p.d, vec);
        if (r) {
            float a[8], b[8];
            h[v].get(a);
            load8(r, c, p.d, vec).get(b);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] += b[i];
            h[v].set(a);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = 8 * (static_cast<int64_t>(v) * blockDim.x + threadIdx.x);
        if (p.H) store8(static_cast<T*>(p.H) + row * p.ldh, c, p.d, vec, h[v]);
        float a[8];
        h[v].get(a);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += a[i] * a[i];
    }
    ss = cta_reduce<false>(ss, red[0]);
    const float mean = ss / static_cast<float>(p.d) + p.eps;
    const float rstd = 1.f / sqrtf(mean);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
    float y[V][8];
    float amax = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = 8 * (static_cast<int64_t>(v) * blockDim.x + threadIdx.x);
        float w[8];
        load8_f32(p.W, c, p.d, wvec, w);
        h[v].get(y[v]);
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[v][i] = y[v][i] * rstd * w[i];
            a = fmaxf(a, fabsf(y[v][i]));
        }
        if constexpr (I8) {
            amax = fmaxf(amax, a);
        } else {
            const float s = block_scale(half_warp_max(a), kE4M3Max);
            const float inv = __frcp_rn(s);
            if (c < p.d) {
                store8_bytes(static_cast<uint8_t*>(p.Q) + row * p.ldq, c, p.d, qvec,
                             f8x4<GEMM_F8_E4M3>(y[v][0] * inv, y[v][1] * inv, y[v][2] * inv, y[v][3] * inv),
                             f8x4<GEMM_F8_E4M3>(y[v][4] * inv, y[v][5] * inv, y[v][6] * inv, y[v][7] * inv));
                if ((threadIdx.x & 15) == 0) p.scale[(c / kF8Block) * p.rows + row] = s;
            }
        }
    }
    if constexpr (I8) {
        amax = cta_reduce<true>(amax, red[1]);
        const float s = block_scale(amax, 127.f);
        const float inv = __frcp_rn(s);
        // int8 holds no NaN: the row's scale carries it
        if (threadIdx.x == 0) p.scale[row] = isfinite(mean) ? s : __int_as_float(0x7fc00000);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = 8 * (static_cast<int64_t>(v) * blockDim.x + threadIdx.x);
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int q = max(-127, min(127, __float2int_rn(y[v][i] * inv)));
                w[i >> 2] |= (static_cast<uint32_t>(q) & 0xffu) << (8 * (i & 3));
            }
            if (c < p.d) store8_bytes(static_cast<uint8_t*>(p.Q) + row * p.ldq, c, p.d, qvec, w[0], w[1]);
        }
    }
}

// Persistent CTAs over the rows; dw's running sums of the CTA's rows stay in
// shared memory (each thread owns its columns), and go to `partial`, which
// dw_reduce_kernel adds up in CTA order.
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const NormBwd p, bool vec, bool wvec) {
    extern __shared__ float dw[];
    __shared__ float red[2][32];
    if (p.dW)
        for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) dw[c] = 0.f;
    __syncthreads();
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        Vec8<T> dy[V], h[V];
        const float rstd = __ldg(p.rstd + row);
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = 8 * (static_cast<int64_t>(v) * blockDim.x + threadIdx.x);
            dy[v] = load8(static_cast<const T*>(p.dY) + row * p.lddy, c, p.d, vec);
            h[v] = load8(static_cast<const T*>(p.H) + row * p.ldh, c, p.d, vec);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = 8 * (static_cast<int64_t>(v) * blockDim.x + threadIdx.x);
            float w[8], a[8], b[8];
            load8_f32(p.W, c, p.d, wvec, w);
            dy[v].get(a);
            h[v].get(b);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot += a[i] * w[i] * (b[i] * rstd);
        }
        const float mean = cta_reduce<false>(dot, red[turn]) / static_cast<float>(p.d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = 8 * (static_cast<int64_t>(v) * blockDim.x + threadIdx.x);
            float w[8], a[8], b[8], o[8];
            load8_f32(p.W, c, p.d, wvec, w);
            dy[v].get(a);
            h[v].get(b);
            if (p.dR) {
                load8(static_cast<const T*>(p.dR) + row * p.lddr, c, p.d, vec).get(o);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // written out so that dX has the same bits with and without dW
                const float xhat = __fmul_rn(b[i], rstd);
                o[i] = __fmaf_rn(rstd, __fmaf_rn(a[i], w[i], -__fmul_rn(xhat, mean)), o[i]);
                if (p.dW && c + i < p.d) dw[c + i] = __fmaf_rn(a[i], xhat, dw[c + i]);
            }
            Vec8<T> out;
            out.set(o);
            store8(static_cast<T*>(p.dX) + row * p.lddx, c, p.d, vec, out);
        }
    }
    if (p.dW) {
        float* out = gridDim.x > 1 ? p.partial + static_cast<int64_t>(blockIdx.x) * p.d : p.dW;
        __syncthreads();
        for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) out[c] = dw[c];
    }
}

// dW_j = sum of the CTAs' sums: a warp's lanes take 32 columns, the eight
// warps of a CTA every eighth partial, joined in warp order.
__global__ void __launch_bounds__(256) dw_reduce_kernel(const float* partial, int parts, int64_t d, float* dW) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.f;
    if (c < d)
        for (int i = warp; i < parts; i += 8) s += partial[static_cast<int64_t>(i) * d + c];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < d) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += red[i][lane];
        dW[c] = s;
    }
}

bool al16(const void* p, int64_t pitch_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && pitch_bytes % 16 == 0;
}

// Threads and vectors per thread of a row of d elements: 4 vectors per thread
// keep enough loads in flight when many rows run at once; a few rows run
// sooner with one vector per thread.
void row_shape(int64_t rows, int64_t d, int num_sms, int* threads, int* vecs) {
    const int64_t nv = (d + 7) / 8;
    int v = rows > 2 * static_cast<int64_t>(num_sms) ? 4 : 1;
    while (v < 4 && (nv + v - 1) / v > 1024) v *= 2;
    int64_t t = ((nv + v - 1) / v + 31) / 32 * 32;
    *threads = static_cast<int>(t);
    *vecs = v;
}

template <typename T, int V>
cudaError_t fwd_launch(const NormFwd& a, int threads, cudaStream_t stream) {
    const int64_t es = sizeof(T);
    const bool vec = al16(a.X, a.ldx * es) && (!a.R || al16(a.R, a.ldr * es)) && (!a.H || al16(a.H, a.ldh * es));
    const bool qvec = reinterpret_cast<uintptr_t>(a.Q) % 8 == 0 && a.ldq % 8 == 0;
    const bool wvec = reinterpret_cast<uintptr_t>(a.W) % 16 == 0;
    if (a.to_i8)
        norm_fwd_kernel<T, V, true><<<static_cast<unsigned>(a.rows), threads, 0, stream>>>(a, vec, qvec, wvec);
    else
        norm_fwd_kernel<T, V, false><<<static_cast<unsigned>(a.rows), threads, 0, stream>>>(a, vec, qvec, wvec);
    return cudaGetLastError();
}

void bwd_shape(int64_t d, int* threads, int* vecs) {
    const int64_t nv = (d + 7) / 8;
    int v = 1;
    while (v < 4 && (nv + v - 1) / v > 512) v *= 2;
    *threads = static_cast<int>(((nv + v - 1) / v + 31) / 32 * 32);
    *vecs = v;
}

template <typename T, int V>
cudaError_t bwd_launch(const NormBwd& a, int threads, cudaStream_t stream) {
    const int64_t es = sizeof(T);
    const bool vec = al16(a.dY, a.lddy * es) && al16(a.H, a.ldh * es) && (!a.dR || al16(a.dR, a.lddr * es)) &&
                     al16(a.dX, a.lddx * es);
    const bool wvec = reinterpret_cast<uintptr_t>(a.W) % 16 == 0;
    const size_t smem = a.dW ? static_cast<size_t>(a.d) * 4 : 0;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel<T, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   GEMM_NORM_MAX_D * 4);
        if (e != cudaSuccess) return e;
    }
    norm_bwd_kernel<T, V><<<a.grid, threads, smem, stream>>>(a, vec, wvec);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.dW && a.grid > 1) {
        dw_reduce_kernel<<<static_cast<unsigned>((a.d + 31) / 32), 256, 0, stream>>>(a.partial, a.grid, a.d, a.dW);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwd& a, cudaStream_t stream) {
    int t, v;
    row_shape(a.rows, a.d, a.num_sms, &t, &v);
    if (a.x_type == GEMM_DTYPE_BF16)
        return v == 1 ? fwd_launch<__nv_bfloat16, 1>(a, t, stream)
               : v == 2 ? fwd_launch<__nv_bfloat16, 2>(a, t, stream) : fwd_launch<__nv_bfloat16, 4>(a, t, stream);
    return v == 1 ? fwd_launch<float, 1>(a, t, stream)
           : v == 2 ? fwd_launch<float, 2>(a, t, stream) : fwd_launch<float, 4>(a, t, stream);
}

int norm_bwd_grid(int64_t rows, int64_t d, int num_sms) {
    (void)d;
    const int64_t g = 2 * static_cast<int64_t>(num_sms);
    return static_cast<int>(rows < g ? rows : g);
}

cudaError_t launch_norm_bwd(const NormBwd& a, cudaStream_t stream) {
    int t, v;
    bwd_shape(a.d, &t, &v);
    if (a.x_type == GEMM_DTYPE_BF16)
        return v == 1 ? bwd_launch<__nv_bfloat16, 1>(a, t, stream)
               : v == 2 ? bwd_launch<__nv_bfloat16, 2>(a, t, stream) : bwd_launch<__nv_bfloat16, 4>(a, t, stream);
    return v == 1 ? bwd_launch<float, 1>(a, t, stream)
           : v == 2 ? bwd_launch<float, 2>(a, t, stream) : bwd_launch<float, 4>(a, t, stream);
}

}  // namespace gemm
