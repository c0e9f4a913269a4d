// Layer norm with the residual's addition.
//
//   h = x + r,  mean = mean(h),  rstd = 1 / sqrt(mean((h - mean)^2) + eps),  y = (h - mean) * rstd * w + b
//
// Bound by DRAM.  The variance is taken of h - mean, not of h^2: the row is in
// registers, so the second pass costs no memory traffic, and a mean far from
// zero cancels nothing.  That pass also gives the mean's own rounding error
// (settle).  Rows come through a ring of bulk copies where there are
// many and they are longer, or not aligned; short aligned rows take a warp, or part
// of one, each; few rows a CTA each.
#include <algorithm>

#include "internal.h"
#include "layer.h"
#include "row_ring.cuh"

namespace gemm {

namespace {

// Sum over the CTA; `red` is used by this call alone until the CTA's next
// barrier.
__device__ __forceinline__ float cta_sum(float v, float* red) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum((threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f);
}
__device__ __forceinline__ float2 cta_sum(float2 v, float2* red) {
    v = make_float2(warp_sum(v.x), warp_sum(v.y));
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// h = x + r as stored, in place of x; the sum of its eight values.
template <typename T>
__device__ __forceinline__ void add_to(Vec8<T>& x, const Vec8<T>& r) {
    float a[8], b[8];
    x.get(a);
    r.get(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] += b[i];
    x.set(a);
}
template <typename T>
__device__ __forceinline__ float sum8(const Vec8<T>& x) {
    float a[8], s = 0.f;
    x.get(a);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += a[i];
    return s;
}
// Sums of h - mean and of its square over the eight values that lie in the row.
template <typename T>
__device__ __forceinline__ float2 residuals8(const Vec8<T>& x, float mean, int64_t c, int64_t d) {
    float a[8];
    float2 s = make_float2(0.f, 0.f);
    x.get(a);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float e = c + i < d ? a[i] - mean : 0.f;
        s.x += e;
        s.y += e * e;
    }
    return s;
}
// A row's rstd from the sums of e = h - mean and of e^2, and its mean without the
// rounding error of the sum that it came from: that error is the mean of e.
//   mean' = mean + off,  sum (h - mean')^2 = sum e^2 - 2 off sum e + d off^2,
// less d rest^2 for what the rounding of mean' leaves.  In a constant row every e
// is k units in the last place, k <= 22 (as many roundings lead to the mean, each
// of half a unit at most), and k^2 d < 2^24: both sums are exact, mean' is the
// value itself, and y = bias whatever the value, d and the kernel are.  (The
// rounded mean alone: a row of 1000 with d = 776 gave 0.019 W.)
__device__ __forceinline__ void settle(float sum, float squares, float d, float inv_d, float eps, float& mean, float& rstd) {
    const float all = __fmul_rn(sum, inv_d), to = mean + all, off = to - mean, rest = all - off;
    float q = fmaf(off, fmaf(d, off, -2.f * sum), squares);
    q = fmaf(-d * rest, rest, q);
    mean = to;
    rstd = 1.f / sqrtf((q < 0.f ? 0.f : q * inv_d) + eps);   // (NaN stays)
}
template <typename T, typename TY>
__device__ __forceinline__ Vec8<TY> normed(const Vec8<T>& x, float mean, float rstd, const float (&w)[8], const float (&b)[8]) {
    float a[8];
    x.get(a);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = fmaf((a[i] - mean) * rstd, w[i], b[i]);
    Vec8<TY> y;
    y.set(a);
    return y;
}
__device__ __forceinline__ void load_wb(const LayerNormFwd& p, int64_t c, bool wvec, bool bvec, float (&w)[8], float (&b)[8]) {
    load8_f32(p.W, c, p.d, wvec, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 0.f;
    if (p.bias) load8_f32(p.bias, c, p.d, bvec, b);
}

// One CTA per row, or (WARP) a warp per row: V vectors of eight values per
// thread, vector v of thread t at column 8 * (v * threads + t).  Bound by latency
// (1 x 8192 3.4 us); with long rows one CTA's loads wait for its sums: 2048 x
// 16384 bfloat16 77 us, 3.5 TB/s.  A warp per row: 43690 x 768 54 us, 5.0 TB/s
// (fp32 70 us, 6.7 TB/s).
constexpr int kWarpThreads = 256;
template <typename T, typename TY, int V, bool VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpThreads : 1024) layer_norm_fwd_kernel(const LayerNormFwd p, bool wvec, bool bvec) {
    __shared__ float red[32];
    __shared__ float2 red2[32];
    pdl_launch_dependents();
    pdl_wait();
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (kWarpThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= p.rows) return;   // whole warps, and no barrier of the CTA
    auto column = [&](int v) { return 8 * (static_cast<int64_t>(v) * nt + t); };
    Vec8<T> h[V];
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = load8<VEC>(static_cast<const T*>(p.X) + row * p.ldx, column(v), p.d);
        if (p.R) add_to(h[v], load8<VEC>(static_cast<const T*>(p.R) + row * p.ldr, column(v), p.d));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (p.H) store8<VEC>(static_cast<T*>(p.H) + row * p.ldh, column(v), p.d, h[v]);
        sum += sum8(h[v]);   // (columns past the row are zero)
    }
    const float d = static_cast<float>(p.d), inv_d = 1.f / d;
    float mean = __fmul_rn(WARP ? warp_sum(sum) : cta_sum(sum, red), inv_d), rstd;   // (rounded: settle counts on it)
    float2 e = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float2 s = residuals8(h[v], mean, column(v), p.d);
        e.x += s.x;
        e.y += s.y;
    }
    e = WARP ? make_float2(warp_sum(e.x), warp_sum(e.y)) : cta_sum(e, red2);
    settle(e.x, e.y, d, inv_d, p.eps, mean, rstd);
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float w[8], b[8];
        load_wb(p, column(v), wvec, bvec, w, b);
        store8<VEC>(static_cast<TY*>(p.Y) + row * p.ldy, column(v), p.d, normed<T, TY>(h[v], mean, rstd, w, b));
    }
}

// Short aligned rows: L lanes hold a row (eight values each), 32 / L rows per
// warp, w and b in registers, and the next rows on their way while these are
// worked on.  Bound by DRAM: 524288 x 64 and 262144 x 128 bfloat16 47 us, 5.7 TB/s.
template <typename T, typename TY, int L>
__global__ void __launch_bounds__(kWarpThreads) layer_norm_fwd_warp_kernel(const LayerNormFwd p, bool wvec, bool bvec) {
    constexpr int kRows = 32 / L, V = 1;
    constexpr bool VEC = true;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, l = lane % L, group = lane / L;
    auto column = [&](int v) { return 8 * (v * L + l); };
    float w[V][8], b[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) load_wb(p, column(v), wvec, bvec, w[v], b[v]);
    const float d = static_cast<float>(p.d), inv_d = 1.f / d;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kWarpThreads / 32) * kRows;
    int64_t first = (static_cast<int64_t>(blockIdx.x) * (kWarpThreads / 32) + (threadIdx.x >> 5)) * kRows;
    Vec8<T> x[V], r[V];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v].zero();
            r[v].zero();
            if (row < p.rows) {
                x[v] = load8<VEC>(static_cast<const T*>(p.X) + row * p.ldx, column(v), p.d);
                if (p.R) r[v] = load8<VEC>(static_cast<const T*>(p.R) + row * p.ldr, column(v), p.d);
            }
        }
    };
    fetch(first + group);
    for (; first < p.rows; first += step) {   // (the whole warp alike)
        const int64_t row = first + group;
        const bool mine = row < p.rows;
        Vec8<T> h[V];
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = x[v];
            if (p.R) add_to(h[v], r[v]);
            sum += sum8(h[v]);
        }
        fetch(row + step);
        float mean = __fmul_rn(lanes_sum<L>(sum), inv_d), rstd;
        float2 e = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 s = residuals8(h[v], mean, column(v), p.d);
            e.x += s.x;
            e.y += s.y;
        }
        settle(lanes_sum<L>(e.x), lanes_sum<L>(e.y), d, inv_d, p.eps, mean, rstd);
        if (!mine) continue;
        if (l == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (p.H) store8<VEC>(static_cast<T*>(p.H) + row * p.ldh, column(v), p.d, h[v]);
            store8<VEC>(static_cast<TY*>(p.Y) + row * p.ldy, column(v), p.d, normed<T, TY>(h[v], mean, rstd, w[v], b[v]));
        }
    }
}

// What the ring kernels begin with: the team's ring, its first chunks on their
// way.
template <typename T>
__device__ __forceinline__ void start_ring(ChunkRing& ring, const LayerNormFwd& p, const RingShape& shape, const Team& team,
                                           uint32_t ring_at, uint64_t* bars, int64_t first) {
    ring.set(0, p.X, p.ldx, sizeof(T), p.d);
    ring.set(1, p.R, p.ldr, sizeof(T), p.d);
    ring.set(2, nullptr, 0, 0, 0);
    ring.ring = ring_at;
    if (team.thread == 0) {
        for (int s = 0; s < shape.slots; ++s) mbar_init(smem_u32(bars + s), 1);
        fence_barrier_init();
        pdl_wait();
        for (int s = 0; s < shape.slots; ++s) ring.fill(first + s * ring.by, s);
    }
}

// Longer aligned rows, many of them: two rows per team from its ring, V vectors
// of eight values per thread and row.  Bound by DRAM (8192 x 8192 bfloat16 85 us, 6.3
// TB/s; 32768 x 1024 47 us, 5.7), with the issue slots half used (118 us by a CTA
// per row, whose two sums nothing hides).
template <typename T, typename TY, int V>
__global__ void __launch_bounds__(kRingThreads, 1) layer_norm_fwd_ring_kernel(const LayerNormFwd p, const RingShape shape, bool wvec, bool bvec) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 red[kRingThreads / 32];
    __shared__ float4 red4[kRingThreads / 32];
    __shared__ __align__(8) uint64_t bars[kRingThreads / 32][ChunkRing::kSlots];
    __shared__ uint32_t abort_flag;
    const int d = static_cast<int>(p.d), lane = threadIdx.x & 31;
    const Team team(shape.team);
    const int64_t first = blockIdx.x + static_cast<int64_t>(team.id) * gridDim.x;
    ChunkRing ring;
    ring.init(p.rows, kPair, false, shape.slots, static_cast<int64_t>(gridDim.x) * shape.teams, smem_u32(bars[team.id]));
    pdl_launch_dependents();
    if (threadIdx.x == 0) abort_flag = 0u;
    const int64_t room = shape.smem / shape.teams;
    start_ring<T>(ring, p, shape, team, smem_u32(smem) + team.id * static_cast<uint32_t>(room), bars[team.id], first);
    pdl_wait();
    __syncthreads();
    const uint8_t* slots = smem + team.id * room;
    auto column = [&](int v) { return 8 * (v * team.threads + team.thread); };
    Pairs w[V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float f[8], g[8];
        load_wb(p, column(v), wvec, bvec, f, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[v].p[i] = pair_of(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
            b[v].p[i] = pair_of(__float_as_uint(g[2 * i]), __float_as_uint(g[2 * i + 1]));
        }
    }
    // sums of both rows over the team
    auto sums = [&](uint64_t x, uint64_t y) {
        float2 v = make_float2(warp_sum(sum_of(x)), warp_sum(sum_of(y)));
        if (team.warps == 1) {
            __syncwarp();
            return v;
        }
        if (lane == 0) red[threadIdx.x >> 5] = v;
        team.sync();
        v = lane < team.warps ? red[team.id * team.warps + lane] : make_float2(0.f, 0.f);
        return make_float2(warp_sum(v.x), warp_sum(v.y));
    };
    auto sums4 = [&](const uint64_t (&x)[kPair], const uint64_t (&y)[kPair]) {
        auto warps = [](const float4& v) { return make_float4(warp_sum(v.x), warp_sum(v.y), warp_sum(v.z), warp_sum(v.w)); };
        float4 v = warps(make_float4(sum_of(x[0]), sum_of(y[0]), sum_of(x[1]), sum_of(y[1])));
        if (team.warps == 1) return v;
        if (lane == 0) red4[threadIdx.x >> 5] = v;
        team.sync();
        v = lane < team.warps ? red4[team.id * team.warps + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        return warps(v);
    };
    const float inv_d = 1.f / static_cast<float>(d);
    int s = 0;
    uint32_t ph = 0;
    for (int64_t c = first; c < ring.chunks; c += ring.by) {
        // a wait that gives up is recorded; the rows are then wrong
        wait_bounded(ring.full0 + 8u * s, ph, &abort_flag, p.err, kDevErrTimeoutEpilogue);
        const int n = ring.rows_of(c);
        const int64_t row = c * kPair;
        Vec8<T> h[kPair][V];
        uint64_t part[kPair] = {0, 0};
#pragma unroll
        for (int r = 0; r < kPair; ++r) {
            if (r >= n) break;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (column(v) >= d) continue;
                h[r][v].load(reinterpret_cast<const T*>(slots + ring.aligned_row(0, s, r)) + column(v));
                Pairs x = pairs(h[r][v]);
                if (p.R) {
                    Vec8<T> res;
                    res.load(reinterpret_cast<const T*>(slots + ring.aligned_row(1, s, r)) + column(v));
                    const Pairs y = pairs(res);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x.p[i] = add2(x.p[i], y.p[i]);
                    h[r][v] = vec<T>(x);
                    x = pairs(h[r][v]);
                }
                if (p.H) h[r][v].store(static_cast<T*>(p.H) + (row + r) * p.ldh + column(v));
#pragma unroll
                for (int i = 0; i < 4; ++i) part[r] = add2(part[r], x.p[i]);
            }
        }
        const float2 total = sums(part[0], part[1]);
        if (team.thread == 0) ring.fill(c + shape.slots * ring.by, s);   // the whole team has read the slot
        float mean[kPair] = {__fmul_rn(total.x, inv_d), __fmul_rn(total.y, inv_d)}, rstd[kPair];
        uint64_t square[kPair] = {0, 0};
        part[0] = part[1] = 0;
#pragma unroll
        for (int r = 0; r < kPair; ++r) {
            if (r >= n) break;
            const uint64_t minus = both(-mean[r]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (column(v) >= d) continue;
                const Pairs x = pairs(h[r][v]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t e = add2(x.p[i], minus);
                    part[r] = add2(part[r], e);
                    square[r] = fma2(e, e, square[r]);
                }
            }
        }
        const float4 e = sums4(part, square);
        settle(e.x, e.y, static_cast<float>(d), inv_d, p.eps, mean[0], rstd[0]);
        settle(e.z, e.w, static_cast<float>(d), inv_d, p.eps, mean[1], rstd[1]);
#pragma unroll
        for (int r = 0; r < kPair; ++r) {
            if (r >= n) break;
            if (team.thread == 0) {
                if (p.mean) p.mean[row + r] = mean[r];
                if (p.rstd) p.rstd[row + r] = rstd[r];
            }
            const uint64_t minus = both(-mean[r]), scale = both(rstd[r]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (column(v) >= d) continue;
                Pairs x = pairs(h[r][v]);
#pragma unroll
                for (int i = 0; i < 4; ++i) x.p[i] = fma2(mul2(add2(x.p[i], minus), scale), w[v].p[i], b[v].p[i]);
                vec<TY>(x).store(static_cast<TY*>(p.Y) + (row + r) * p.ldy + column(v));
            }
        }
        if (++s == shape.slots) {
            s = 0;
            ph ^= 1u;
        }
    }
}

// Rows that are not aligned (or not of whole vectors): they come through the
// ring as runs of bytes and leave through staging buffers the same way, and in
// between each value is taken by itself, neighbouring lanes neighbouring values,
// J values per thread and row.  Dense short rows: a warp per team, which takes
// several rows at a time.  Bound by the instructions that each value takes and
// the rows' sums: 33520 x 1001 bfloat16 94 us, 2.9 TB/s, 4096 x 8191 90 us (137 by a CTA
// per row), 516222 x 65 204 us, 1.3 TB/s; 20919 x 401 fp32 32 us, 4.2 TB/s.  (Of that the
// mean's correction is 1 to 6 %.)
template <typename T, typename TY, int J>
__global__ void __launch_bounds__(kRingThreads, 1) layer_norm_fwd_odd_kernel(const LayerNormFwd p, const RingShape shape) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int kRows = rows_together(J);
    __shared__ float red[kRingThreads / 32 * kRows], red2[2 * (kRingThreads / 32 * kRows)];
    __shared__ __align__(8) uint64_t bars[kRingThreads / 32][ChunkRing::kSlots];
    __shared__ uint32_t abort_flag;
    const int d = static_cast<int>(p.d), lane = threadIdx.x & 31;
    const bool dense = shape.dense != 0;
    const Team team(shape.team);
    const int64_t begin = blockIdx.x + static_cast<int64_t>(team.id) * gridDim.x;
    ChunkRing ring;
    ring.init(p.rows, shape.per, dense, shape.slots, static_cast<int64_t>(gridDim.x) * shape.teams, smem_u32(bars[team.id]));
    pdl_launch_dependents();
    if (threadIdx.x == 0) abort_flag = 0u;
    const int64_t room = shape.smem / shape.teams;
    uint8_t* slots = smem + team.id * room;
    start_ring<T>(ring, p, shape, team, smem_u32(slots), bars[team.id], begin);
    pdl_wait();
    __syncthreads();
    uint8_t* out = slots + shape.slots * ring.slot_bytes;
    const uint32_t h_run = static_cast<uint32_t>(ChunkRing::run_place(p.d * sizeof(T))), y_run = static_cast<uint32_t>(ChunkRing::run_place(p.d * sizeof(TY)));
    const uint32_t h_place = p.H ? static_cast<uint32_t>(ChunkRing::place(p.d * sizeof(T), shape.per, dense)) : 0u;
    const uint32_t out_bytes = h_place + static_cast<uint32_t>(ChunkRing::place(p.d * sizeof(TY), shape.per, dense));
    const int first = team.thread, stride = team.threads;
    constexpr int P = J / 2;   // pairs of values, at 2 i and 2 i + 1 strides
    auto in = [&](int j) { return first + j * stride < d; };
    uint64_t w[P], b[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        w[i] = pair_at(p.W + first + 2 * i * stride, stride, in(2 * i), in(2 * i + 1));
        b[i] = p.bias ? pair_at(p.bias + first + 2 * i * stride, stride, in(2 * i), in(2 * i + 1)) : 0ull;
    }
    const float inv_d = 1.f / static_cast<float>(d);
    int s = 0, buf = 0;
    uint32_t ph = 0;
    for (int64_t c = begin; c < ring.chunks; c += ring.by, buf ^= 1) {
        // a wait that gives up is recorded; the rows are then wrong
        wait_bounded(ring.full0 + 8u * s, ph, &abort_flag, p.err, kDevErrTimeoutEpilogue);
        if (!ring.whole(c)) load_ends(ring, slots, s, c, team);
        const int n = ring.rows_of(c);
        const int64_t row0 = c * shape.per;
        // where row r goes, and where it is staged
        auto h_to = [&](int r) { return reinterpret_cast<uintptr_t>(p.H) + (row0 + r) * p.ldh * sizeof(T); };
        auto y_to = [&](int r) { return reinterpret_cast<uintptr_t>(p.Y) + (row0 + r) * p.ldy * sizeof(TY); };
        auto h_at = [&](int r) { return out + buf * out_bytes + (dense ? (h_to(0) & 15) + r * d * sizeof(T) : r * h_run + (h_to(r) & 15)); };
        auto y_at = [&](int r) {
            return out + buf * out_bytes + h_place + (dense ? (y_to(0) & 15) + r * d * sizeof(TY) : r * y_run + (y_to(r) & 15));
        };
        for (int r0 = 0; r0 < n; r0 += kRows) {
            uint64_t a[kRows][P];
            float mean[kRows], rstd[kRows], e2[2 * kRows];
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                mean[q] = 0.f;
                if (r0 + q >= n) continue;
                const T* x = reinterpret_cast<const T*>(slots + ring.row(0, s, c, r0 + q)) + first;
                const T* res = reinterpret_cast<const T*>(slots + ring.row(1, s, c, r0 + q)) + first;
                T* h = reinterpret_cast<T*>(h_at(r0 + q)) + first;
                uint64_t sum2 = 0;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int e = 2 * i * stride;
                    a[q][i] = pair_at(x + e, stride, in(2 * i), in(2 * i + 1));
                    if (p.R) a[q][i] = rounded_pair<T>(add2(a[q][i], pair_at(res + e, stride, in(2 * i), in(2 * i + 1))));
                    if (p.H) put_pair(a[q][i], h + e, stride, in(2 * i), in(2 * i + 1));
                    sum2 = add2(sum2, a[q][i]);
                }
                mean[q] = sum_of(sum2);
            }
            team.sum(mean, red);
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                e2[2 * q] = e2[2 * q + 1] = 0.f;
                if (r0 + q >= n) continue;
                mean[q] = __fmul_rn(mean[q], inv_d);
                const uint64_t minus = both(-mean[q]);
                uint64_t sum2 = 0, ss2 = 0;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    // (a value past the row stays zero)
                    a[q][i] = add2(a[q][i], pair_of(in(2 * i) ? static_cast<uint32_t>(minus) : 0u, in(2 * i + 1) ? static_cast<uint32_t>(minus) : 0u));
                    sum2 = add2(sum2, a[q][i]);
                    ss2 = fma2(a[q][i], a[q][i], ss2);
                }
                e2[2 * q] = sum_of(sum2);
                e2[2 * q + 1] = sum_of(ss2);
            }
            team.sum(e2, red2);
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                if (r0 + q >= n) continue;
                const float before = mean[q];
                settle(e2[2 * q], e2[2 * q + 1], static_cast<float>(d), inv_d, p.eps, mean[q], rstd[q]);
                if (first == 0) {
                    if (p.mean) p.mean[row0 + r0 + q] = mean[q];
                    if (p.rstd) p.rstd[row0 + r0 + q] = rstd[q];
                }
                TY* y = reinterpret_cast<TY*>(y_at(r0 + q)) + first;
                const uint64_t scale = both(rstd[q]), minus = both(before - mean[q]);
#pragma unroll
                for (int i = 0; i < P; ++i)
                    put_pair(fma2(mul2(add2(a[q][i], minus), scale), w[i], b[i]), y + 2 * i * stride, stride, in(2 * i), in(2 * i + 1));
            }
        }
        // What was staged leaves; the buffer before it has been read by then.
        fence_proxy_async_smem();
        if (team.thread == 0) bulk_wait_read_all();
        team.sync();
        const int runs = dense ? 1 : n;
        const uint32_t values = static_cast<uint32_t>(dense ? n * d : d);
        if (team.thread == 0) {
            ring.fill(c + shape.slots * ring.by, s);
            for (int r = 0; r < runs; ++r) {
                if (p.H) store_run(h_to(r), smem_u32(h_at(r)), values * sizeof(T));
                store_run(y_to(r), smem_u32(y_at(r)), values * sizeof(TY));
            }
            bulk_commit();
        }
        if (team.warp == team.warps - 1)
            for (int r = 0; r < runs; ++r) {
                if (p.H) store_ends<T>(h_to(r), h_at(r), values * sizeof(T), lane);
                store_ends<TY>(y_to(r), y_at(r), values * sizeof(TY), lane);
            }
        if (++s == shape.slots) {
            s = 0;
            ph ^= 1u;
        }
    }
    if (team.thread == 0) bulk_wait_all();
}

bool al16(const void* p, int64_t pitch_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && pitch_bytes % 16 == 0;
}

// Bytes of a slot and of a team's staging buffers (unaligned rows: two of them).
template <typename T>
int64_t slot_bytes(const LayerNormFwd& a, int per, bool dense) { return (a.R ? 2 : 1) * ChunkRing::place(a.d * sizeof(T), per, dense); }
template <typename T, typename TY>
int64_t out_bytes(const LayerNormFwd& a, int per, bool dense) {
    return 2 * (ChunkRing::place(a.d * sizeof(TY), per, dense) + (a.H ? ChunkRing::place(a.d * sizeof(T), per, dense) : 0));
}

template <typename K, typename... A>
cudaError_t ring_launch(K kern, const LayerNormFwd& a, const RingShape& r, bool holds, cudaStream_t stream, A... more) {
    if (!holds) return cudaErrorInvalidValue;
    const cudaError_t e = kernel_attrs_once(reinterpret_cast<const void*>(kern), static_cast<int>(kRingSmem), true);
    if (e != cudaSuccess) return e;
    return launch_chained(kern, dim3(static_cast<unsigned>(r.grid)), r.team * r.teams, static_cast<size_t>(r.smem), stream, a, r, more...);
}

template <typename T, typename TY, bool VEC>
cudaError_t fwd_aligned(const LayerNormFwd& a, cudaStream_t stream) {
    const bool wvec = reinterpret_cast<uintptr_t>(a.W) % 16 == 0, bvec = reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    const int64_t nv = (a.d + 7) / 8, sms = a.num_sms;
    const int64_t es = sizeof(T), ey = sizeof(TY);
    const bool whole = VEC && a.d % 8 == 0;
    const bool many = a.rows > 4 * sms;
    // Short rows: one warp's in the ring (two at a time) once there are many of
    // bfloat16 (87381 x 384: 51 us, 67 by a warp per row; 2000 x 384 5.4, 5.1); fp32 and
    // up to 768 elements a warp per row (52428 x 640: 64 us, 73 through the ring).
    if (whole && many && a.d <= 8192 && (a.d > 768 || (es == 2 && a.d > 128 && a.d <= 512 && a.rows >= 32 * sms))) {
        RingShape r;
        r.per = kPair;
        r.dense = 0;
        team_of(&r, nv, {2, 1});
        if (fit_ring(&r, a.rows, slot_bytes<T>(a, r.per, false), 0, a.num_sms)) {
            const bool holds = !r.dense && ring_holds(r, kPair, nv, slot_bytes<T>(a, kPair, false), 0, 0);
            return r.each == 2 ? ring_launch(layer_norm_fwd_ring_kernel<T, TY, 2>, a, r, holds, stream, wvec, bvec)
                               : ring_launch(layer_norm_fwd_ring_kernel<T, TY, 1>, a, r, holds, stream, wvec, bvec);
        }
    }
    if (!whole && many && a.d <= 8192 && a.d > 16) {
        RingShape r;
        r.dense = a.ldx == a.d && (!a.R || a.ldr == a.d) && (!a.H || a.ldh == a.d) && a.ldy == a.d;
        if (r.dense && a.d <= 512) {   // a warp's rows
            r.per = rows_of_a_warp(a.d * std::max(es, ey));
            r.team = 32;
            const int j = static_cast<int>((a.d + 31) / 32);
            r.each = j + j % 2;
        } else {
            r.per = 2;
            team_of(&r, a.d, {16, 14, 12, 10, 8});
        }
        auto fits = [&] { return fit_ring(&r, a.rows, slot_bytes<T>(a, r.per, r.dense), out_bytes<T, TY>(a, r.per, r.dense), a.num_sms); };
        bool fit = fits();
        if (!fit && r.per == 2) {   // longer rows one by one
            r.per = 1;
            fit = fits();
        }
        const bool holds = fit && ring_holds(r, r.per, a.d, slot_bytes<T>(a, r.per, r.dense), out_bytes<T, TY>(a, r.per, r.dense), 0);
        if (fit)
            switch (r.each) {
                case 2: return ring_launch(layer_norm_fwd_odd_kernel<T, TY, 2>, a, r, holds, stream);
                case 4: return ring_launch(layer_norm_fwd_odd_kernel<T, TY, 4>, a, r, holds, stream);
                case 6: return ring_launch(layer_norm_fwd_odd_kernel<T, TY, 6>, a, r, holds, stream);
                case 8: return ring_launch(layer_norm_fwd_odd_kernel<T, TY, 8>, a, r, holds, stream);
                case 10: return ring_launch(layer_norm_fwd_odd_kernel<T, TY, 10>, a, r, holds, stream);
                case 14: return ring_launch(layer_norm_fwd_odd_kernel<T, TY, 14>, a, r, holds, stream);
                case 12: return ring_launch(layer_norm_fwd_odd_kernel<T, TY, 12>, a, r, holds, stream);
                default: return ring_launch(layer_norm_fwd_odd_kernel<T, TY, 16>, a, r, holds, stream);
            }
    }
    if (a.d <= 768 && a.rows >= 8 * sms) {   // a warp per row, once there are eight for every SM
        if constexpr (VEC) {
            auto go = [&](auto kern, int lanes) {
                const int64_t rows = kWarpThreads / lanes, blocks = (a.rows + rows - 1) / rows, most = 8 * sms;
                return launch_chained(kern, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), kWarpThreads, 0, stream,
                                      a, wvec, bvec);
            };
            if (a.d <= 64) return go(layer_norm_fwd_warp_kernel<T, TY, 8>, 8);
            if (a.d <= 128) return go(layer_norm_fwd_warp_kernel<T, TY, 16>, 16);
            if (a.d <= 256) return go(layer_norm_fwd_warp_kernel<T, TY, 32>, 32);
        }
        const dim3 grid(static_cast<unsigned>((a.rows + kWarpThreads / 32 - 1) / (kWarpThreads / 32)));
        auto go = [&](auto kern) { return launch_chained(kern, grid, kWarpThreads, 0, stream, a, wvec, bvec); };
        return a.d <= 256 ? go(layer_norm_fwd_kernel<T, TY, 1, VEC, true>)
               : a.d <= 512 ? go(layer_norm_fwd_kernel<T, TY, 2, VEC, true>) : go(layer_norm_fwd_kernel<T, TY, 3, VEC, true>);
    }
    int v = many ? 2 : 1;   // a few rows are done sooner with one
    while (v < 4 && (nv + v - 1) / v > 1024) v *= 2;
    const unsigned threads = static_cast<unsigned>(((nv + v - 1) / v + 31) / 32 * 32);
    const auto kern = v == 1 ? layer_norm_fwd_kernel<T, TY, 1, VEC, false>
                      : v == 2 ? layer_norm_fwd_kernel<T, TY, 2, VEC, false> : layer_norm_fwd_kernel<T, TY, 4, VEC, false>;
    return launch_chained(kern, dim3(static_cast<unsigned>(a.rows)), threads, 0, stream, a, wvec, bvec);
}

template <typename T, typename TY>
cudaError_t fwd_type(const LayerNormFwd& a, cudaStream_t stream) {
    const int64_t es = sizeof(T);
    const bool vec = al16(a.X, a.ldx * es) && (!a.R || al16(a.R, a.ldr * es)) && (!a.H || al16(a.H, a.ldh * es)) &&
                     al16(a.Y, a.ldy * static_cast<int64_t>(sizeof(TY)));
    return vec ? fwd_aligned<T, TY, true>(a, stream) : fwd_aligned<T, TY, false>(a, stream);
}

}  // namespace

cudaError_t launch_layer_norm_fwd(const LayerNormFwd& a, cudaStream_t stream) {
    const bool xb = a.x_type == GEMM_DTYPE_BF16, yb = a.y_type == GEMM_DTYPE_BF16;
    return xb ? (yb ? fwd_type<__nv_bfloat16, __nv_bfloat16>(a, stream) : fwd_type<__nv_bfloat16, float>(a, stream))
              : (yb ? fwd_type<float, __nv_bfloat16>(a, stream) : fwd_type<float, float>(a, stream));
}

}  // namespace gemm
