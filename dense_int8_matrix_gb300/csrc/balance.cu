// Balance loss of a router with the experts' counts, and its gradient.
//
//   p = softmax(x),  f = counts / sum(counts),  P = mean of p over the rows that take part
//   loss = coef * E * sum(f * P)
//   dx = dr + dloss * coef * E / T * p * (f - sum(f * p))
//
// Bound by DRAM: the logits are read once by each pass.  A warp takes a row at
// a time, its lanes the columns lane + 32 v, so that each lane keeps the sums of
// p over its own columns in registers.  A CTA writes its sums of p and its
// counts; a second kernel adds them in CTA order and forms the loss.
#include "f8.cuh"
#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

namespace gemm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerSum = 32;   // rows added in a row before they join the running sum

// exp(a - largest) of a warp's row in place, and 1 / their sum (0 for a row of
// -infinity alone, whose p are 0); a NaN or +infinity makes the sum NaN.
// Columns past the row hold -infinity.
template <int V>
__device__ __forceinline__ float exponentials(float (&a)[V], float& base, float& sum) {
    float top = a[0];
#pragma unroll
    for (int v = 1; v < V; ++v) top = fmaxf(top, a[v]);
    top = warp_max(top);
    base = top == -__int_as_float(0x7f800000) ? 0.f : top;
    sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        a[v] = expf(a[v] - base);
        sum += a[v];
    }
    sum = warp_sum(sum);
    return sum == 0.f ? 0.f : 1.f / sum;
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) balance_rows_kernel(const Balance p) {
    extern __shared__ int32_t shared[];   // counts[experts + 1] (the last one: used rows), then sums[warps][experts]
    int32_t* hist = shared;
    float* sums = reinterpret_cast<float*>(shared + p.experts + 1);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = p.experts;
    for (int i = threadIdx.x; i <= e; i += kThreads) hist[i] = 0;
    __syncthreads();
    float total[V], part[V];
#pragma unroll
    for (int v = 0; v < V; ++v) total[v] = part[v] = 0.f;
    int pending = 0, mine = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp; row < p.rows; row += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int32_t* index = p.index + row * p.top_k;
        bool taken = false;
        for (int k = lane; k < p.top_k; k += 32) {
            const int32_t i = __ldg(index + k);
            if (i >= 0 && i < e) {
                taken = true;
                atomicAdd(hist + i, 1);
            }
        }
        if (!__any_sync(0xffffffffu, taken)) {   // padding: not read
            if (lane == 0) p.lse[row] = __int_as_float(0x7f800000);
            continue;
        }
        ++mine;
        const T* x = static_cast<const T*>(p.X) + row * p.ldx;
        float a[V], base, sum;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = lane + 32 * v;
            a[v] = c < e ? to_f32(x[c]) : -__int_as_float(0x7f800000);
        }
        const float inv = exponentials<V>(a, base, sum);
        if (lane == 0) p.lse[row] = base + logf(sum);
#pragma unroll
        for (int v = 0; v < V; ++v) part[v] = fmaf(a[v], inv, part[v]);
        if (++pending == kRowsPerSum) {
            pending = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                total[v] += part[v];
                part[v] = 0.f;
            }
        }
    }
    if (lane == 0 && mine) atomicAdd(hist + e, mine);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (lane + 32 * v < e) sums[warp * e + lane + 32 * v] = total[v] + part[v];
    __syncthreads();
    for (int i = threadIdx.x; i <= e; i += kThreads) {
        p.partial_c[static_cast<int64_t>(blockIdx.x) * (e + 1) + i] = hist[i];
        if (i == e) break;
        float s = sums[i];
        for (int w = 1; w < kWarps; ++w) s += sums[w * e + i];
        p.partial_p[static_cast<int64_t>(blockIdx.x) * e + i] = s;
    }
}

// One CTA: a thread per expert adds the CTAs' sums, then counts, offsets and
// the loss.
__global__ void __launch_bounds__(1024) balance_loss_kernel(const Balance p) {
    __shared__ int32_t scan[32];
    __shared__ float red[32];
    pdl_launch_dependents();
    pdl_wait();
    const int e = p.experts, t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = blockDim.x >> 5;
    int32_t count = 0, rows = 0;
    float sum = 0.f;
    if (t < e)
        for (int i = 0; i < p.parts; ++i) {
            count += p.partial_c[static_cast<int64_t>(i) * (e + 1) + t];
            sum += p.partial_p[static_cast<int64_t>(i) * e + t];
        }
    for (int i = lane; i < p.parts; i += 32) rows += p.partial_c[static_cast<int64_t>(i) * (e + 1) + e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, o);
    int32_t before = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t up = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += up;
    }
    if (lane == 31) scan[warp] = before;
    __syncthreads();
    int32_t slots = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before += scan[w];
        slots += scan[w];
    }
    const float prob = rows > 0 ? sum / static_cast<float>(rows) : 0.f;
    const float share = slots > 0 ? static_cast<float>(count) / static_cast<float>(slots) : 0.f;
    float l = warp_sum(t < e ? share * prob : 0.f);
    if (lane == 0) red[warp] = l;
    __syncthreads();
    if (warp == 0) l = warp_sum(lane < warps ? red[lane] : 0.f);
    if (t < e) {
        p.counts[t] = count;
        p.probs[t] = prob;
        if (p.offsets) p.offsets[t + 1] = before;
    }
    if (t == 0) {
        if (p.offsets) p.offsets[0] = 0;
        *p.used = rows;
        *p.loss = p.coef * static_cast<float>(e) * l;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(const BalanceBwd p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = p.experts;
    int32_t slots = 0;
    float f[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int32_t c = lane + 32 * v < e ? __ldg(p.counts + lane + 32 * v) : 0;
        slots += c;
        f[v] = static_cast<float>(c);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) slots += __shfl_xor_sync(0xffffffffu, slots, o);
    const int32_t used = __ldg(p.used);
    const float per_slot = slots > 0 ? 1.f / static_cast<float>(slots) : 0.f;
    const float scale = used > 0 ? __ldg(p.dloss) * p.coef * static_cast<float>(e) / static_cast<float>(used) : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] *= per_slot;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp; row < p.rows; row += static_cast<int64_t>(gridDim.x) * kWarps) {
        const float lse = __ldg(p.lse + row);
        const bool part = !isinf(lse);
        const T* x = static_cast<const T*>(p.X) + row * p.ldx;
        const T* dr = p.dR ? static_cast<const T*>(p.dR) + row * p.lddr : nullptr;
        T* dx = static_cast<T*>(p.dX) + row * p.lddx;
        float a[V], d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = lane + 32 * v;
            a[v] = part && c < e ? to_f32(x[c]) : -__int_as_float(0x7f800000);
            d[v] = dr && c < e ? to_f32(dr[c]) : 0.f;
        }
        // p is formed from the row again: exp(x - lse) would carry lse's rounding
        float base, sum, mix = 0.f;
        const float inv = exponentials<V>(a, base, sum);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            a[v] *= inv;
            if (lane + 32 * v < e) mix = fmaf(a[v], f[v], mix);
        }
        mix = warp_sum(mix);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane + 32 * v < e) from_f32(part ? fmaf(scale * a[v], f[v] - mix, d[v]) : d[v], dx + lane + 32 * v);
    }
}

int columns_per_lane(int experts) {
    int v = 1;
    while (32 * v < experts) v *= 2;
    return v;
}

template <typename T>
cudaError_t rows_launch(const Balance& a, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(a.experts + 1 + kWarps * a.experts) * 4;   // at most 37 KB
    auto go = [&](auto kern) { return launch_chained(kern, dim3(static_cast<unsigned>(a.parts)), kThreads, smem, stream, a); };
    switch (columns_per_lane(a.experts)) {
        case 1: return go(balance_rows_kernel<T, 1>);
        case 2: return go(balance_rows_kernel<T, 2>);
        case 4: return go(balance_rows_kernel<T, 4>);
        case 8: return go(balance_rows_kernel<T, 8>);
        case 16: return go(balance_rows_kernel<T, 16>);
        default: return go(balance_rows_kernel<T, 32>);
    }
}

template <typename T>
cudaError_t bwd_launch(const BalanceBwd& a, cudaStream_t stream) {
    const int64_t blocks = (a.rows + kWarps - 1) / kWarps, most = 8 * static_cast<int64_t>(a.num_sms);
    auto go = [&](auto kern) {
        return launch_chained(kern, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), kThreads, 0, stream, a);
    };
    switch (columns_per_lane(a.experts)) {
        case 1: return go(balance_bwd_kernel<T, 1>);
        case 2: return go(balance_bwd_kernel<T, 2>);
        case 4: return go(balance_bwd_kernel<T, 4>);
        case 8: return go(balance_bwd_kernel<T, 8>);
        case 16: return go(balance_bwd_kernel<T, 16>);
        default: return go(balance_bwd_kernel<T, 32>);
    }
}

}  // namespace

int balance_parts(const Balance& a) {
    const int64_t blocks = (a.rows + kWarps - 1) / kWarps, most = a.num_sms;
    return static_cast<int>(blocks < most ? blocks : most);
}

cudaError_t launch_balance(const Balance& a, cudaStream_t stream, int* launches) {
    *launches = 0;
    cudaError_t e = a.x_type == GEMM_DTYPE_BF16 ? rows_launch<__nv_bfloat16>(a, stream) : rows_launch<float>(a, stream);
    if (e != cudaSuccess) return e;
    ++*launches;
    e = launch_chained(balance_loss_kernel, dim3(1), static_cast<unsigned>((a.experts + 31) / 32 * 32), 0, stream, a);
    if (e == cudaSuccess) ++*launches;
    return e;
}

cudaError_t launch_balance_bwd(const BalanceBwd& a, cudaStream_t stream) {
    return a.x_type == GEMM_DTYPE_BF16 ? bwd_launch<__nv_bfloat16>(a, stream) : bwd_launch<float>(a, stream);
}

}  // namespace gemm
