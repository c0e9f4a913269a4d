// Layer norm with the residual's addition, and its gradient.
//
//   h = x + r,  mean = mean(h),  rstd = 1 / sqrt(mean((h - mean)^2) + eps),  y = (h - mean) * rstd * w + b
//   dx = dr + rstd * (g - mean(g) - xhat * mean(g * xhat)),  g = dy * w, xhat = (h - mean) * rstd
//   dw = sum over rows of dy * xhat,  db = sum over rows of dy
//
// Both are bound by DRAM.  The variance is taken of h - mean, not of h^2: the
// row is in registers, so the second pass costs no memory traffic, and a mean
// far from zero cancels nothing.
#include "f8.cuh"
#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

namespace gemm {

namespace {

// Sum over the CTA; `red` is used by this call alone.
__device__ __forceinline__ float cta_sum(float v, float* red) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum((threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f);
}

// One CTA per row, or (WARP, rows of at most 768 elements) a warp per row and
// kWarpRows rows per CTA.  The row stays in registers: V vectors of eight values
// per thread, vector v of thread t at column 8 * (v * threads + t).  Mean and
// variance are taken of h as it is stored.
constexpr int kWarpRows = 8;
template <typename T, typename TY, int V, bool VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : 1024) layer_norm_fwd_kernel(const LayerNormFwd p, bool wvec, bool bvec) {
    __shared__ float red[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= p.rows) return;   // whole warps, and no barrier of the CTA
    const T* x = static_cast<const T*>(p.X) + row * p.ldx;
    const T* r = p.R ? static_cast<const T*>(p.R) + row * p.ldr : nullptr;
    auto column = [&](int v) { return 8 * (static_cast<int64_t>(v) * nt + t); };
    Vec8<T> h[V];
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = load8<VEC>(x, column(v), p.d);
        if (r) {
            float a[8], b[8];
            h[v].get(a);
            load8<VEC>(r, column(v), p.d).get(b);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] += b[i];
            h[v].set(a);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (p.H) store8<VEC>(static_cast<T*>(p.H) + row * p.ldh, column(v), p.d, h[v]);
        float a[8];
        h[v].get(a);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += a[i];   // (columns past the row are zero)
    }
    const float mean = (WARP ? warp_sum(sum) : cta_sum(sum, red[0])) / static_cast<float>(p.d);
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float a[8];
        h[v].get(a);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = column(v) + i < p.d ? a[i] - mean : 0.f;
            ss += c * c;
        }
    }
    ss = WARP ? warp_sum(ss) : cta_sum(ss, red[1]);
    const float rstd = 1.f / sqrtf(ss / static_cast<float>(p.d) + p.eps);
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float a[8], w[8], b[8];
        h[v].get(a);
        load8_f32(p.W, column(v), p.d, wvec, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = 0.f;
        if (p.bias) load8_f32(p.bias, column(v), p.d, bvec, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = fmaf((a[i] - mean) * rstd, w[i], b[i]);
        Vec8<TY> y;
        y.set(a);
        store8<VEC>(static_cast<TY*>(p.Y) + row * p.ldy, column(v), p.d, y);
    }
}

// dx: one CTA per row, the row in registers.
template <typename T, typename TY, int V, bool VEC>
__global__ void __launch_bounds__(1024) layer_norm_dx_kernel(const LayerNormBwd p, bool wvec) {
    __shared__ float red[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x;
    auto column = [&](int v) { return 8 * (static_cast<int64_t>(v) * blockDim.x + threadIdx.x); };
    const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
    Vec8<TY> dy[V];
    Vec8<T> h[V], dr[V];
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        dy[v] = load8<VEC>(static_cast<const TY*>(p.dY) + row * p.lddy, column(v), p.d);
        h[v] = load8<VEC>(static_cast<const T*>(p.H) + row * p.ldh, column(v), p.d);
        if (p.dR)
            dr[v] = load8<VEC>(static_cast<const T*>(p.dR) + row * p.lddr, column(v), p.d);
        else
            dr[v].zero();
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float w[8], a[8], b[8];
        load8_f32(p.W, column(v), p.d, wvec, w);
        dy[v].get(a);
        h[v].get(b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // (past the row dy and w are zero)
            const float g = a[i] * w[i];
            sum += g;
            dot += column(v) + i < p.d ? g * ((b[i] - mean) * rstd) : 0.f;
        }
    }
    const float inv_d = 1.f / static_cast<float>(p.d);
    const float mg = cta_sum(sum, red[0]) * inv_d, mx = cta_sum(dot, red[1]) * inv_d;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float w[8], a[8], b[8], o[8];
        load8_f32(p.W, column(v), p.d, wvec, w);
        dy[v].get(a);
        h[v].get(b);
        dr[v].get(o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float xhat = (b[i] - mean) * rstd;
            o[i] = fmaf(rstd, fmaf(-xhat, mx, fmaf(a[i], w[i], -mg)), o[i]);
        }
        Vec8<T> out;
        out.set(o);
        store8<VEC>(static_cast<T*>(p.dX) + row * p.lddx, column(v), p.d, out);
    }
}

// dw and db: a thread takes eight columns of a range of rows, `lanes`
// neighbouring threads the columns of a row; a CTA's sums are joined in shared
// memory in a fixed order.
constexpr int kColThreads = 256;
constexpr int kColRows = 4;   // rows in flight per thread
template <typename T, typename TY, bool VEC>
__global__ void __launch_bounds__(kColThreads) layer_norm_dw_kernel(const LayerNormBwd p, int lanes) {
    __shared__ float red[2][kColThreads * 8];
    pdl_launch_dependents();
    pdl_wait();
    const int groups = kColThreads / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * lanes + lane) * 8;
    const int64_t per = (p.rows + p.parts - 1) / p.parts;
    const int64_t lo = per * blockIdx.y, hi = lo + per < p.rows ? lo + per : p.rows;
    float dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.f;
    for (int64_t r0 = lo + group; r0 < hi; r0 += static_cast<int64_t>(kColRows) * groups) {
        Vec8<TY> dy[kColRows];
        Vec8<T> h[kColRows];
        float mean[kColRows], rstd[kColRows];
#pragma unroll
        for (int k = 0; k < kColRows; ++k) {
            const int64_t r = r0 + static_cast<int64_t>(k) * groups;
            dy[k].zero();
            h[k].zero();
            mean[k] = rstd[k] = 0.f;
            if (r < hi && c < p.d) {
                dy[k] = load8<VEC>(static_cast<const TY*>(p.dY) + r * p.lddy, c, p.d);
                h[k] = load8<VEC>(static_cast<const T*>(p.H) + r * p.ldh, c, p.d);
                mean[k] = __ldg(p.mean + r);
                rstd[k] = __ldg(p.rstd + r);
            }
        }
#pragma unroll
        for (int k = 0; k < kColRows; ++k) {
            float a[8], b[8];
            dy[k].get(a);
            h[k].get(b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[i] = fmaf(a[i], (b[i] - mean[k]) * rstd[k], dw[i]);
                db[i] += a[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        red[0][(group * lanes + lane) * 8 + i] = dw[i];
        red[1][(group * lanes + lane) * 8 + i] = db[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * lanes; i += kColThreads) {
        const int which = i / (8 * lanes), j = i % (8 * lanes);
        float* out = which == 0 ? p.dW : p.dbias;
        if (!out) continue;
        float v = red[which][j];
        for (int g = 1; g < groups; ++g) v += red[which][g * lanes * 8 + j];
        const int64_t col = static_cast<int64_t>(blockIdx.x) * lanes * 8 + j;
        if (p.parts > 1) out = p.partial + (static_cast<int64_t>(which) * p.parts + blockIdx.y) * p.d;
        if (col < p.d) out[col] = v;
    }
}

bool al16(const void* p, int64_t pitch_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && pitch_bytes % 16 == 0;
}

// Threads and vectors per thread of a row of d elements; many rows at once
// run best with two vectors per thread, a few rows sooner with one.
void row_shape(int64_t rows, int64_t d, int num_sms, int* threads, int* vecs) {
    const int64_t nv = (d + 7) / 8;
    int v = rows <= 2 * static_cast<int64_t>(num_sms) ? 1 : 2;
    while (v < 4 && (nv + v - 1) / v > 1024) v *= 2;
    *threads = static_cast<int>(((nv + v - 1) / v + 31) / 32 * 32);
    *vecs = v;
}

template <typename T, typename TY, int V, bool VEC, bool WARP>
cudaError_t fwd_launch(const LayerNormFwd& a, int threads, cudaStream_t stream) {
    const bool wvec = reinterpret_cast<uintptr_t>(a.W) % 16 == 0, bvec = reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    const int64_t grid = WARP ? (a.rows + kWarpRows - 1) / kWarpRows : a.rows;
    return launch_chained(layer_norm_fwd_kernel<T, TY, V, VEC, WARP>, dim3(static_cast<unsigned>(grid)), threads, 0, stream, a,
                          wvec, bvec);
}

template <typename T, typename TY, bool VEC>
cudaError_t fwd_aligned(const LayerNormFwd& a, cudaStream_t stream) {
    // a warp per row, once there is a CTA of such for every SM
    if (a.d <= 768 && a.rows >= static_cast<int64_t>(kWarpRows) * a.num_sms) {
        constexpr int kThreads = 32 * kWarpRows;
        return a.d <= 256 ? fwd_launch<T, TY, 1, VEC, true>(a, kThreads, stream)
               : a.d <= 512 ? fwd_launch<T, TY, 2, VEC, true>(a, kThreads, stream)
                            : fwd_launch<T, TY, 3, VEC, true>(a, kThreads, stream);
    }
    int t, v;
    row_shape(a.rows, a.d, a.num_sms, &t, &v);
    return v == 1 ? fwd_launch<T, TY, 1, VEC, false>(a, t, stream)
           : v == 2 ? fwd_launch<T, TY, 2, VEC, false>(a, t, stream) : fwd_launch<T, TY, 4, VEC, false>(a, t, stream);
}

template <typename T, typename TY>
cudaError_t fwd_type(const LayerNormFwd& a, cudaStream_t stream) {
    const int64_t es = sizeof(T);
    const bool vec = al16(a.X, a.ldx * es) && (!a.R || al16(a.R, a.ldr * es)) && (!a.H || al16(a.H, a.ldh * es)) &&
                     al16(a.Y, a.ldy * static_cast<int64_t>(sizeof(TY)));
    return vec ? fwd_aligned<T, TY, true>(a, stream) : fwd_aligned<T, TY, false>(a, stream);
}

template <typename T, typename TY>
bool bwd_vec(const LayerNormBwd& a) {
    const int64_t es = sizeof(T);
    return al16(a.dY, a.lddy * static_cast<int64_t>(sizeof(TY))) && al16(a.H, a.ldh * es) && (!a.dR || al16(a.dR, a.lddr * es)) &&
           al16(a.dX, a.lddx * es);
}

// Lanes of a row in the column sums: whole warps unless the row is shorter.
int col_lanes(int64_t d) {
    int lanes = 32;
    while (lanes > 1 && 4 * lanes >= d) lanes /= 2;
    return lanes;
}

template <typename T, typename TY, bool VEC>
cudaError_t dx_launch(const LayerNormBwd& a, cudaStream_t stream) {
    int t, v;
    row_shape(a.rows, a.d, a.num_sms, &t, &v);
    const bool wvec = reinterpret_cast<uintptr_t>(a.W) % 16 == 0;
    const auto kern = v == 1 ? layer_norm_dx_kernel<T, TY, 1, VEC>
                      : v == 2 ? layer_norm_dx_kernel<T, TY, 2, VEC> : layer_norm_dx_kernel<T, TY, 4, VEC>;
    return launch_chained(kern, dim3(static_cast<unsigned>(a.rows)), t, 0, stream, a, wvec);
}

template <typename T, typename TY>
cudaError_t bwd_type(const LayerNormBwd& a, cudaStream_t stream, int* launches) {
    const bool vec = bwd_vec<T, TY>(a);
    *launches = 0;
    if (a.dW || a.dbias) {   // first: dX may be dR, or dY
        const int lanes = col_lanes(a.d);
        const dim3 grid(static_cast<unsigned>((a.d + 8 * lanes - 1) / (8 * lanes)), static_cast<unsigned>(a.parts));
        cudaError_t e = vec ? launch_chained(layer_norm_dw_kernel<T, TY, true>, grid, kColThreads, 0, stream, a, lanes)
                            : launch_chained(layer_norm_dw_kernel<T, TY, false>, grid, kColThreads, 0, stream, a, lanes);
        if (e != cudaSuccess) return e;
        ++*launches;
        if (a.parts > 1) {
            if (a.dW) {
                e = launch_column_sums(a.partial, a.parts, a.d, a.dW, stream);
                if (e != cudaSuccess) return e;
                ++*launches;
            }
            if (a.dbias) {
                e = launch_column_sums(a.partial + static_cast<int64_t>(a.parts) * a.d, a.parts, a.d, a.dbias, stream);
                if (e != cudaSuccess) return e;
                ++*launches;
            }
        }
    }
    ++*launches;
    return vec ? dx_launch<T, TY, true>(a, stream) : dx_launch<T, TY, false>(a, stream);
}

}  // namespace

cudaError_t launch_layer_norm_fwd(const LayerNormFwd& a, cudaStream_t stream) {
    const bool xb = a.x_type == GEMM_DTYPE_BF16, yb = a.y_type == GEMM_DTYPE_BF16;
    return xb ? (yb ? fwd_type<__nv_bfloat16, __nv_bfloat16>(a, stream) : fwd_type<__nv_bfloat16, float>(a, stream))
              : (yb ? fwd_type<float, __nv_bfloat16>(a, stream) : fwd_type<float, float>(a, stream));
}

int layer_norm_bwd_parts(const LayerNormBwd& a) {
    const int lanes = col_lanes(a.d);
    const int64_t blocks = (a.d + 8 * lanes - 1) / (8 * lanes);
    const int64_t turn = static_cast<int64_t>(kColRows) * (kColThreads / lanes);
    int64_t parts = (8 * static_cast<int64_t>(a.num_sms) + blocks - 1) / blocks;
    const int64_t most = (a.rows + 2 * turn - 1) / (2 * turn);
    if (parts > most) parts = most;
    return static_cast<int>(parts < 1 ? 1 : parts);
}

cudaError_t launch_layer_norm_bwd(const LayerNormBwd& a, cudaStream_t stream, int* launches) {
    const bool xb = a.x_type == GEMM_DTYPE_BF16, yb = a.y_type == GEMM_DTYPE_BF16;
    return xb ? (yb ? bwd_type<__nv_bfloat16, __nv_bfloat16>(a, stream, launches) : bwd_type<__nv_bfloat16, float>(a, stream, launches))
              : (yb ? bwd_type<float, __nv_bfloat16>(a, stream, launches) : bwd_type<float, float>(a, stream, launches));
}

}  // namespace gemm
