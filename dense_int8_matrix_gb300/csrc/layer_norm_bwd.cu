// Gradient of the layer norm.
//
//   dx = dr + rstd * (g - mean(g) - xhat * mean(g * xhat)),  g = dy * w, xhat = (h - mean) * rstd
//   dw = sum over rows of dy * xhat,  db = sum over rows of dy
//
// Bound by DRAM.  Where there are many rows of at most 8192 elements, one kernel
// reads everything once: short rows by warps, longer ones by CTAs that take
// them from a ring of bulk copies; each thread has the same columns of every
// row and keeps their dw and db in registers.  The rest (few rows, or long
// ones, whose sums no CTA could hold) takes a pass over the columns for dw and
// db and one over the rows for dx.  All partial sums are joined in a fixed order.
#include <algorithm>

#include "internal.h"
#include "layer.h"
#include "row_ring.cuh"

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
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// What eight columns of a row give to the sums of g and of g * xhat.
template <typename T, typename TY>
__device__ __forceinline__ void row_sums(const Vec8<TY>& dy, const Vec8<T>& h, const float (&w)[8], float mean, float rstd,
                                         int64_t c, int64_t d, float& sum, float& dot) {
    float a[8], b[8];
    dy.get(a);
    h.get(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float g = __fmul_rn(a[i], w[i]);
        sum += g;
        dot += c + i < d ? g * __fmul_rn(b[i] - mean, rstd) : 0.f;   // (past the row dy and w are zero)
    }
}
// dx of them (written out so that it has the same bits whatever else is asked
// for), and their dw and db.
template <typename T, typename TY>
__device__ __forceinline__ Vec8<T> row_dx(const Vec8<TY>& dy, const Vec8<T>& h, const Vec8<T>& dr, const float (&w)[8], float mean,
                                          float rstd, float mg, float mx, float (&dw)[8], float (&db)[8]) {
    float a[8], b[8], o[8];
    dy.get(a);
    h.get(b);
    dr.get(o);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float xhat = __fmul_rn(b[i] - mean, rstd);
        o[i] = __fmaf_rn(rstd, __fmaf_rn(-xhat, mx, __fmaf_rn(a[i], w[i], -mg)), o[i]);
        dw[i] = __fmaf_rn(a[i], xhat, dw[i]);
        db[i] += a[i];
    }
    Vec8<T> out;
    out.set(o);
    return out;
}

// Short aligned rows: L lanes hold a row (V vectors of eight values each), 32 / L
// rows per warp; the next rows are on their way while these are worked on.
// 524288 x 64 and 262144 x 128 bfloat16 58 us, 4.6 TB/s.  (L = 32, V = 2, rows of 257 to
// 512 elements that are too few for the ring: 128 to 532 bytes spill.)
constexpr int kWarpThreads = 256;
template <typename T, typename TY, int L, int V>
__global__ void __launch_bounds__(kWarpThreads, 2) layer_norm_bwd_warp_kernel(const LayerNormBwd p, bool wvec) {
    constexpr int kRows = 32 / L, kWarps = kWarpThreads / 32, kCols = 8 * L * V;
    __shared__ float red[kWarps][kCols];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % L, group = lane / L;
    auto column = [&](int v) { return 8 * (v * L + l); };
    float w[V][8], dw[V][8], db[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        load8_f32(p.W, column(v), p.d, wvec, w[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = db[v][i] = 0.f;
    }
    const float inv_d = 1.f / static_cast<float>(p.d);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kRows;
    int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kRows;
    Vec8<TY> dy[V], next_dy[V];
    Vec8<T> h[V], dr[V], next_h[V], next_dr[V];
    float mean, rstd, next_mean, next_rstd;
    auto fetch = [&](int64_t row) {
        next_mean = next_rstd = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            next_dy[v].zero();
            next_h[v].zero();
            next_dr[v].zero();
            if (row < p.rows) {
                next_dy[v] = load8<true>(static_cast<const TY*>(p.dY) + row * p.lddy, column(v), p.d);
                next_h[v] = load8<true>(static_cast<const T*>(p.H) + row * p.ldh, column(v), p.d);
                if (p.dR) next_dr[v] = load8<true>(static_cast<const T*>(p.dR) + row * p.lddr, column(v), p.d);
            }
        }
        if (row < p.rows) {
            next_mean = __ldg(p.mean + row);
            next_rstd = __ldg(p.rstd + row);
        }
    };
    fetch(first + group);
    for (; first < p.rows; first += step) {   // (the whole warp alike)
        const int64_t row = first + group;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dy[v] = next_dy[v];
            h[v] = next_h[v];
            dr[v] = next_dr[v];
        }
        mean = next_mean;
        rstd = next_rstd;
        fetch(row + step);
        float sum = 0.f, dot = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) row_sums(dy[v], h[v], w[v], mean, rstd, column(v), p.d, sum, dot);
        const float mg = lanes_sum<L>(sum) * inv_d, mx = lanes_sum<L>(dot) * inv_d;
        if (row >= p.rows) continue;
#pragma unroll
        for (int v = 0; v < V; ++v)
            store8<true>(static_cast<T*>(p.dX) + row * p.lddx, column(v), p.d,
                         row_dx(dy[v], h[v], dr[v], w[v], mean, rstd, mg, mx, dw[v], db[v]));
    }
    // the warp's row groups, then the CTA's warps
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float* out = which == 0 ? p.dW : p.dbias;
        if (!out) continue;
        if (p.parts > 1) out = p.partial + (static_cast<int64_t>(which) * p.parts + blockIdx.x) * p.d;
        if (which == 1) __syncthreads();   // the sums before have been read
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float x = which == 0 ? dw[v][i] : db[v][i];
#pragma unroll
                for (int o = L; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (group == 0) red[warp][column(v) + i] = x;
            }
        __syncthreads();
        for (int c = threadIdx.x; c < p.d; c += kWarpThreads) {
            float x = red[0][c];
#pragma unroll
            for (int k = 1; k < kWarps; ++k) x += red[k][c];
            out[c] = x;
        }
    }
}

// The teams' sums of dw or db (one row of d floats each, in shared memory),
// added in their order into the CTA's partial.  The whole CTA.
__device__ __forceinline__ void join_teams(const LayerNormBwd& p, int which, const float* sums, int teams) {
    float* out = which == 0 ? p.dW : p.dbias;
    if (p.parts > 1) out = p.partial + (static_cast<int64_t>(which) * p.parts + blockIdx.x) * p.d;
    const int d = static_cast<int>(p.d);
    for (int e = threadIdx.x; e < d; e += blockDim.x) {
        float x = sums[e];
        for (int k = 1; k < teams; ++k) x += sums[k * d + e];
        out[e] = x;
    }
}

template <typename T, typename TY>
__device__ __forceinline__ void start_ring(ChunkRing& ring, const LayerNormBwd& p, const RingShape& shape, const Team& team,
                                           uint32_t ring_at, uint64_t* bars, int64_t first) {
    ring.set(0, p.dY, p.lddy, sizeof(TY), p.d);
    ring.set(1, p.H, p.ldh, sizeof(T), p.d);
    ring.set(2, p.dR, p.lddr, sizeof(T), p.d);
    ring.ring = ring_at;
    if (team.thread == 0) {
        for (int s = 0; s < shape.slots; ++s) mbar_init(smem_u32(bars + s), 1);
        fence_barrier_init();
        pdl_wait();
        for (int s = 0; s < shape.slots; ++s) ring.fill(first + s * ring.by, s);
    }
}

// Longer aligned rows: two rows per team from its ring, V vectors of eight
// values per thread and row, whose w, dw and db stay in registers.  Bound by a
// row's two sums as much as by DRAM: 4096 x 8192 bfloat16 54 us, 5.0 TB/s (50 without
// dw and db; 91 with one row in a CTA), 16384 x 2048 fp32 78 us, 6.0 TB/s.
template <typename T, typename TY, int V>
__global__ void __launch_bounds__(kRingThreads, 1) layer_norm_bwd_ring_kernel(const LayerNormBwd p, const RingShape shape, bool wvec) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float4 red[kRingThreads / 32];
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
    start_ring<T, TY>(ring, p, shape, team, smem_u32(smem) + team.id * static_cast<uint32_t>(room), bars[team.id], first);
    pdl_wait();
    __syncthreads();
    const uint8_t* slots = smem + team.id * room;
    auto column = [&](int v) { return 8 * (v * team.threads + team.thread); };
    Pairs w[V], dw[V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float f[8];
        load8_f32(p.W, column(v), d, wvec, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[v].p[i] = pair_of(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
            dw[v].p[i] = db[v].p[i] = 0;
        }
    }
    const float inv_d = 1.f / static_cast<float>(d);
    int s = 0;
    uint32_t ph = 0;
    float mean[kPair], rstd[kPair];
    auto statistics = [&](int64_t c) {   // of the next chunk, while this one is worked on
#pragma unroll
        for (int r = 0; r < kPair; ++r) {
            const bool in = c * kPair + r < p.rows;
            mean[r] = in ? __ldg(p.mean + c * kPair + r) : 0.f;
            rstd[r] = in ? __ldg(p.rstd + c * kPair + r) : 0.f;
        }
    };
    statistics(first);
    for (int64_t c = first; c < ring.chunks; c += ring.by) {
        uint64_t minus[kPair], scale[kPair];
#pragma unroll
        for (int r = 0; r < kPair; ++r) {
            minus[r] = both(-mean[r]);
            scale[r] = both(rstd[r]);
        }
        statistics(c + ring.by);
        // a wait that gives up is recorded; the rows are then wrong
        wait_bounded(ring.full0 + 8u * s, ph, &abort_flag, p.err, kDevErrTimeoutEpilogue);
        const int n = ring.rows_of(c);
        const int64_t row = c * kPair;
        uint64_t sum2[kPair] = {0, 0}, dot2[kPair] = {0, 0};
        auto in = [&](int array, int r, int v) { return slots + ring.aligned_row(array, s, r) + column(v) * (array == 0 ? sizeof(TY) : sizeof(T)); };
#pragma unroll
        for (int r = 0; r < kPair; ++r) {
            if (r >= n) break;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (column(v) >= d) continue;
                Vec8<TY> dy;
                Vec8<T> h;
                dy.load(reinterpret_cast<const TY*>(in(0, r, v)));
                h.load(reinterpret_cast<const T*>(in(1, r, v)));
                const Pairs y = pairs(dy), x = pairs(h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t g = mul2(y.p[i], w[v].p[i]);
                    sum2[r] = add2(sum2[r], g);
                    dot2[r] = fma2(g, mul2(add2(x.p[i], minus[r]), scale[r]), dot2[r]);
                }
            }
        }
        float4 all = make_float4(warp_sum(sum_of(sum2[0])), warp_sum(sum_of(dot2[0])), warp_sum(sum_of(sum2[1])), warp_sum(sum_of(dot2[1])));
        if (team.warps > 1) {
            if (lane == 0) red[threadIdx.x >> 5] = all;
            team.sync();
            all = lane < team.warps ? red[team.id * team.warps + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
            all = make_float4(warp_sum(all.x), warp_sum(all.y), warp_sum(all.z), warp_sum(all.w));
        }
        const uint64_t mg[kPair] = {both(-all.x * inv_d), both(-all.z * inv_d)}, mx[kPair] = {both(-all.y * inv_d), both(-all.w * inv_d)};
#pragma unroll
        for (int r = 0; r < kPair; ++r) {
            if (r >= n) break;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (column(v) >= d) continue;
                Vec8<TY> dy;
                Vec8<T> h, dr;
                dy.load(reinterpret_cast<const TY*>(in(0, r, v)));
                h.load(reinterpret_cast<const T*>(in(1, r, v)));
                if (p.dR)
                    dr.load(reinterpret_cast<const T*>(in(2, r, v)));
                else
                    dr.zero();
                const Pairs y = pairs(dy), x = pairs(h), q = pairs(dr);
                Pairs o;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t xhat = mul2(add2(x.p[i], minus[r]), scale[r]);
                    o.p[i] = fma2(scale[r], fma2(xhat, mx[r], fma2(y.p[i], w[v].p[i], mg[r])), q.p[i]);
                    dw[v].p[i] = fma2(y.p[i], xhat, dw[v].p[i]);
                    db[v].p[i] = add2(db[v].p[i], y.p[i]);
                }
                vec<T>(o).store(static_cast<T*>(p.dX) + (row + r) * p.lddx + column(v));
            }
        }
        team.sync();   // the whole team has read the slot, and the sums
        if (team.thread == 0) ring.fill(c + shape.slots * ring.by, s);
        if (++s == shape.slots) {
            s = 0;
            ph ^= 1u;
        }
    }
    float* sums = reinterpret_cast<float*>(smem);   // every chunk has been taken by then
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (!(which == 0 ? p.dW : p.dbias)) continue;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (column(v) < d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint64_t*>(sums + team.id * d + column(v) + 2 * i) = which == 0 ? dw[v].p[i] : db[v].p[i];
        __syncthreads();
        join_teams(p, which, sums, shape.teams);
    }
}

// Rows that are not aligned (or not of whole vectors): they come through the
// ring as runs of bytes and dx leaves through staging buffers the same way; in
// between each value is taken by itself, neighbouring lanes neighbouring values,
// J values per thread and row.  Dense short rows: a warp per team, which takes
// several rows at a time.  Bound by the instructions that each value takes: 33520 x
// 1001 bfloat16 91 us, 2.9 TB/s, 4096 x 8191 91 us, 516222 x 65 143 us, 1.9 TB/s.  (J = 12 and
// 16 spill 12 to 16 bytes.)
template <typename T, typename TY, int J>
__global__ void __launch_bounds__(kRingThreads, 1) layer_norm_bwd_odd_kernel(const LayerNormBwd p, const RingShape shape) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int kRows = rows_together(J);
    __shared__ float red[kRingThreads / 32 * 2 * kRows];
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
    start_ring<T, TY>(ring, p, shape, team, smem_u32(slots), bars[team.id], begin);
    pdl_wait();
    __syncthreads();
    uint8_t* out = slots + shape.slots * ring.slot_bytes;
    const uint32_t run = static_cast<uint32_t>(ChunkRing::run_place(p.d * sizeof(T)));
    const uint32_t out_bytes = static_cast<uint32_t>(ChunkRing::place(p.d * sizeof(T), shape.per, dense));
    const int first = team.thread, stride = team.threads;
    constexpr int P = J / 2;   // pairs of values, at 2 i and 2 i + 1 strides
    auto in = [&](int j) { return first + j * stride < d; };
    uint64_t w[P], dw[P], db[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        w[i] = pair_at(p.W + first + 2 * i * stride, stride, in(2 * i), in(2 * i + 1));
        dw[i] = db[i] = 0;
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
        auto to = [&](int r) { return reinterpret_cast<uintptr_t>(p.dX) + (row0 + r) * p.lddx * sizeof(T); };
        auto at = [&](int r) { return out + buf * out_bytes + (dense ? (to(0) & 15) + r * d * sizeof(T) : r * run + (to(r) & 15)); };
        for (int r0 = 0; r0 < n; r0 += kRows) {
            float sums[2 * kRows];
            uint64_t y[kRows][P], xhat[kRows][P], scale[kRows];
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                sums[2 * q] = sums[2 * q + 1] = 0.f;
                if (r0 + q >= n) continue;
                const uint64_t minus = both(-__ldg(p.mean + row0 + r0 + q));
                scale[q] = both(__ldg(p.rstd + row0 + r0 + q));
                const TY* from = reinterpret_cast<const TY*>(slots + ring.row(0, s, c, r0 + q)) + first;
                const T* h = reinterpret_cast<const T*>(slots + ring.row(1, s, c, r0 + q)) + first;
                uint64_t sum2 = 0, dot2 = 0;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int e = 2 * i * stride;
                    y[q][i] = pair_at(from + e, stride, in(2 * i), in(2 * i + 1));
                    xhat[q][i] = mul2(add2(pair_at(h + e, stride, in(2 * i), in(2 * i + 1)), minus), scale[q]);
                    const uint64_t g = mul2(y[q][i], w[i]);
                    sum2 = add2(sum2, g);
                    dot2 = fma2(g, xhat[q][i], dot2);   // (past the row g is zero)
                }
                sums[2 * q] = sum_of(sum2);
                sums[2 * q + 1] = sum_of(dot2);
            }
            team.sum(sums, red);
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                if (r0 + q >= n) continue;
                const T* dr = reinterpret_cast<const T*>(slots + ring.row(2, s, c, r0 + q)) + first;
                T* dx = reinterpret_cast<T*>(at(r0 + q)) + first;
                const uint64_t mg = both(-sums[2 * q] * inv_d), mx = both(-sums[2 * q + 1] * inv_d);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int e = 2 * i * stride;
                    const uint64_t o = p.dR ? pair_at(dr + e, stride, in(2 * i), in(2 * i + 1)) : 0ull;
                    put_pair(fma2(scale[q], fma2(xhat[q][i], mx, fma2(y[q][i], w[i], mg)), o), dx + e, stride, in(2 * i), in(2 * i + 1));
                    dw[i] = fma2(y[q][i], xhat[q][i], dw[i]);
                    db[i] = add2(db[i], y[q][i]);
                }
            }
            if (team.warps > 1 && r0 + kRows < n) team.sync();   // (the sums have been read)
        }
        // What was staged leaves; the buffer before it has been read by then.
        fence_proxy_async_smem();
        if (team.thread == 0) bulk_wait_read_all();
        team.sync();
        const int runs = dense ? 1 : n;
        const uint32_t bytes = static_cast<uint32_t>((dense ? n * d : d) * sizeof(T));
        if (team.thread == 0) {
            ring.fill(c + shape.slots * ring.by, s);
            for (int r = 0; r < runs; ++r) store_run(to(r), smem_u32(at(r)), bytes);
            bulk_commit();
        }
        if (team.warp == team.warps - 1)
            for (int r = 0; r < runs; ++r) store_ends<T>(to(r), at(r), bytes, lane);
        if (++s == shape.slots) {
            s = 0;
            ph ^= 1u;
        }
    }
    if (team.thread == 0) bulk_wait_all();
    float* sums = reinterpret_cast<float*>(smem);   // every chunk has been taken, and has left, by then
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (!(which == 0 ? p.dW : p.dbias)) continue;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < P; ++i)
            put_pair(which == 0 ? dw[i] : db[i], sums + team.id * d + first + 2 * i * stride, stride, in(2 * i), in(2 * i + 1));
        __syncthreads();
        join_teams(p, which, sums, shape.teams);
    }
}

// dW and dbias from the CTAs' sums, both in one launch: a CTA takes sixteen
// columns; its 16 groups of sixteen lanes take every 16th partial, ten loads at a
// time, and are joined in a fixed order.  Latency: about 4 us of a call (4096 x 8192
// 56.2 us with sixteen columns, 58.7 with eight, 57.2 with 32).
__global__ void __launch_bounds__(256) layer_norm_join_kernel(const LayerNormBwd p, int from) {
    constexpr int kCols = 16, kLoads = 10, kGroups = 256 / kCols;
    __shared__ float red[8][kCols];
    pdl_launch_dependents();
    pdl_wait();
    const int which = from + static_cast<int>(blockIdx.y);
    const float* partial = p.partial + static_cast<int64_t>(which) * p.parts * p.d;
    float* out = which == 0 ? p.dW : p.dbias;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kCols + lane % kCols;
    float s = 0.f;
    if (c < p.d) {
        for (int i = static_cast<int>(threadIdx.x) / kCols; i < p.parts; i += kLoads * kGroups) {
            float v[kLoads];
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                v[j] = i + j * kGroups < p.parts ? partial[static_cast<int64_t>(i + j * kGroups) * p.d + c] : 0.f;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) s += v[j];
        }
    }
#pragma unroll
    for (int o = kCols; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane < kCols) red[warp][lane] = s;
    __syncthreads();
    if (threadIdx.x < kCols && c < p.d) {
        s = red[0][lane];
#pragma unroll
        for (int i = 1; i < 8; ++i) s += red[i][lane];
        out[c] = s;
    }
}

// dx: one CTA per row, the row in registers.  With the pass below: 300 x 4096
// bfloat16 11 us (latency), 2048 x 16384 103 us and 4096 x 8192 fp32 126 us, 2.6 and
// 3.7 TB/s of what one pass would move.  (V = 4, rows beyond 16384 elements: a CTA's 1024
// threads have 64 registers each, and 136 to 544 bytes spill; V = 2 of unaligned
// fp32 rows 12 to 16.)
template <typename T, typename TY, int V, bool VEC>
__global__ void __launch_bounds__(1024, 1) layer_norm_dx_kernel(const LayerNormBwd p, bool wvec) {
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
        float w[8];
        load8_f32(p.W, column(v), p.d, wvec, w);
        row_sums(dy[v], h[v], w, mean, rstd, column(v), p.d, sum, dot);
    }
    const float inv_d = 1.f / static_cast<float>(p.d);
    const float mg = cta_sum(sum, red[0]) * inv_d, mx = cta_sum(dot, red[1]) * inv_d;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float w[8], unused[2][8] = {};
        load8_f32(p.W, column(v), p.d, wvec, w);
        store8<VEC>(static_cast<T*>(p.dX) + row * p.lddx, column(v), p.d,
                    row_dx(dy[v], h[v], dr[v], w, mean, rstd, mg, mx, unused[0], unused[1]));
    }
}

// dw and db: a thread takes eight columns of a range of rows, `lanes`
// neighbouring threads the columns of a row; a CTA's sums are joined in shared
// memory in a fixed order.
constexpr int kColThreads = 256;
constexpr int kColRows = 4;   // rows in flight per thread
template <typename T, typename TY, bool VEC>
__global__ void __launch_bounds__(kColThreads) layer_norm_dw_kernel(const LayerNormBwd p, int lanes, int cluster) {
    __shared__ float red[2][kColThreads * 8];
    pdl_launch_dependents();
    pdl_wait();
    const int groups = kColThreads / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * lanes + lane) * 8;
    const int64_t per = (p.rows + gridDim.y - 1) / gridDim.y;
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
    const int n = 8 * lanes;   // (at most kColThreads)
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float* out = which == 0 ? p.dW : p.dbias;
        if (!out) continue;   // (every CTA alike)
        if (threadIdx.x < n) {
            float v = red[which][threadIdx.x];
            for (int g = 1; g < groups; ++g) v += red[which][g * n + threadIdx.x];
            red[which][threadIdx.x] = v;   // (its only reader)
        }
        if (p.parts > 1) out = p.partial + (static_cast<int64_t>(which) * p.parts + blockIdx.y / cluster) * p.d;
        join_cluster(red[which], n, cluster, [&](int i, float v) {
            const int64_t col = static_cast<int64_t>(blockIdx.x) * n + i;
            if (col < p.d) out[col] = v;
        });
    }
}

bool al16(const void* p, int64_t pitch_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && pitch_bytes % 16 == 0;
}

bool bwd_vec(const LayerNormBwd& a) {
    const int64_t es = a.x_type == GEMM_DTYPE_BF16 ? 2 : 4, ey = a.y_type == GEMM_DTYPE_BF16 ? 2 : 4;
    return al16(a.dY, a.lddy * ey) && al16(a.H, a.ldh * es) && (!a.dR || al16(a.dR, a.lddr * es)) && al16(a.dX, a.lddx * es);
}

// Which kernels take the call.
enum Way { kByWarps, kByRing, kOdd, kTwoPasses };
struct Choice {
    Way way;
    int lanes;        // of a row (kByWarps)
    RingShape ring;   // (kByRing, kOdd)
    int grid;         // CTAs; row ranges (kTwoPasses)
    int parts;        // sums to be joined through scratch
};

// Lanes of a row in the column sums: whole warps unless the row is shorter.
int col_lanes(int64_t d) {
    int lanes = 32;
    while (lanes > 1 && 4 * lanes >= d) lanes /= 2;
    return lanes;
}

// Bytes of a slot and of a team's staging buffers (unaligned rows: two of them).
int64_t slot_bytes(const LayerNormBwd& a, int per, bool dense) {
    const int64_t es = a.x_type == GEMM_DTYPE_BF16 ? 2 : 4, ey = a.y_type == GEMM_DTYPE_BF16 ? 2 : 4;
    return ChunkRing::place(a.d * ey, per, dense) + (a.dR ? 2 : 1) * ChunkRing::place(a.d * es, per, dense);
}
int64_t out_bytes(const LayerNormBwd& a, int per, bool dense) {
    return 2 * ChunkRing::place(a.d * (a.x_type == GEMM_DTYPE_BF16 ? 2 : 4), per, dense);
}

Choice choose(const LayerNormBwd& a) {
    Choice c{};
    const bool vec = bwd_vec(a), whole = vec && a.d % 8 == 0;
    const int64_t es = a.x_type == GEMM_DTYPE_BF16 ? 2 : 4, ey = a.y_type == GEMM_DTYPE_BF16 ? 2 : 4;
    const int64_t sms = a.num_sms;
    RingShape& r = c.ring;
    // (87381 x 384: 96 us by warps, 61 through the ring; 2000 x 384 8.0, 9.8)
    if (whole && (a.d <= 128 || (a.d <= 512 && a.rows < 32 * sms)) && a.rows >= 8 * sms) {
        c.way = kByWarps;
        c.lanes = a.d <= 64 ? 8 : a.d <= 128 ? 16 : 32;
        const int64_t rows = kWarpThreads / c.lanes;
        c.parts = c.grid = static_cast<int>(std::min<int64_t>((a.rows + 2 * rows - 1) / (2 * rows), 2 * sms));
        return c;
    }
    if (a.rows > 2 * sms && a.d <= 8192 && a.d > 16) {
        r.dense = !whole && a.lddy == a.d && a.ldh == a.d && (!a.dR || a.lddr == a.d) && a.lddx == a.d;
        r.per = 1;
        if (whole) {
            r.per = kPair;
            team_of(&r, a.d / 8, {2, 1});
        } else if (r.dense && a.d <= 512) {   // a warp's rows
            r.per = rows_of_a_warp(a.d * std::max(es, ey));
            r.team = 32;
            const int j = static_cast<int>((a.d + 31) / 32);
            r.each = j + j % 2;
        } else {
            r.per = 2;
            team_of(&r, a.d, {16, 14, 12, 10, 8});
        }
        auto fits = [&] { return fit_ring(&r, a.rows, slot_bytes(a, r.per, r.dense), whole ? 0 : out_bytes(a, r.per, r.dense), a.num_sms); };
        bool fit = fits();
        if (!fit && !whole && r.per == 2) {   // longer unaligned rows one by one (the aligned kernel takes kPair)
            r.per = 1;
            fit = fits();
        }
        if (fit) {
            c.way = whole ? kByRing : kOdd;
            c.parts = c.grid = r.grid;
            return c;
        }
    }
    c.way = kTwoPasses;
    const int lanes = col_lanes(a.d);
    const int64_t blocks = (a.d + 8 * lanes - 1) / (8 * lanes), turn = static_cast<int64_t>(kColRows) * (kColThreads / lanes);
    // Up to eight ranges are one cluster and joined in it; of more, the sums go
    // through scratch.
    c.grid = static_cast<int>(std::max<int64_t>(1, std::min((8 * sms + blocks - 1) / blocks, (a.rows + 2 * turn - 1) / (2 * turn))));
    c.parts = c.grid <= kMostClusterCtas ? 1 : c.grid;
    return c;
}

template <typename T, typename TY>
cudaError_t by_warps(const LayerNormBwd& a, const Choice& c, cudaStream_t stream) {
    auto go = [&](auto kern) {
        return launch_chained(kern, dim3(static_cast<unsigned>(c.grid)), kWarpThreads, 0, stream, a,
                              reinterpret_cast<uintptr_t>(a.W) % 16 == 0);
    };
    return c.lanes == 8 ? go(layer_norm_bwd_warp_kernel<T, TY, 8, 1>)
           : c.lanes == 16 ? go(layer_norm_bwd_warp_kernel<T, TY, 16, 1>)
           : a.d <= 256 ? go(layer_norm_bwd_warp_kernel<T, TY, 32, 1>) : go(layer_norm_bwd_warp_kernel<T, TY, 32, 2>);
}

// (the teams' sums, d floats each, take the slots' place)
template <typename K, typename... A>
cudaError_t ring_launch(K kern, const LayerNormBwd& a, const RingShape& r, bool holds, cudaStream_t stream, A... more) {
    if (!holds) return cudaErrorInvalidValue;
    const cudaError_t e = kernel_attrs_once(reinterpret_cast<const void*>(kern), static_cast<int>(kRingSmem), true);
    if (e != cudaSuccess) return e;
    return launch_chained(kern, dim3(static_cast<unsigned>(r.grid)), r.team * r.teams, static_cast<size_t>(r.smem), stream, a, r, more...);
}
template <typename T, typename TY>
cudaError_t by_ring(const LayerNormBwd& a, const RingShape& r, cudaStream_t stream) {
    const bool wvec = reinterpret_cast<uintptr_t>(a.W) % 16 == 0;
    const bool holds = !r.dense && ring_holds(r, kPair, a.d / 8, slot_bytes(a, kPair, false), 0, 4 * a.d);
    return r.each == 1 ? ring_launch(layer_norm_bwd_ring_kernel<T, TY, 1>, a, r, holds, stream, wvec)
                       : ring_launch(layer_norm_bwd_ring_kernel<T, TY, 2>, a, r, holds, stream, wvec);
}
template <typename T, typename TY>
cudaError_t by_odd(const LayerNormBwd& a, const RingShape& r, cudaStream_t stream) {
    const bool holds = ring_holds(r, r.per, a.d, slot_bytes(a, r.per, r.dense), out_bytes(a, r.per, r.dense), 4 * a.d);
    switch (r.each) {
        case 2: return ring_launch(layer_norm_bwd_odd_kernel<T, TY, 2>, a, r, holds, stream);
        case 4: return ring_launch(layer_norm_bwd_odd_kernel<T, TY, 4>, a, r, holds, stream);
        case 6: return ring_launch(layer_norm_bwd_odd_kernel<T, TY, 6>, a, r, holds, stream);
        case 8: return ring_launch(layer_norm_bwd_odd_kernel<T, TY, 8>, a, r, holds, stream);
        case 10: return ring_launch(layer_norm_bwd_odd_kernel<T, TY, 10>, a, r, holds, stream);
        case 14: return ring_launch(layer_norm_bwd_odd_kernel<T, TY, 14>, a, r, holds, stream);
        case 12: return ring_launch(layer_norm_bwd_odd_kernel<T, TY, 12>, a, r, holds, stream);
        default: return ring_launch(layer_norm_bwd_odd_kernel<T, TY, 16>, a, r, holds, stream);
    }
}

template <typename T, typename TY, bool VEC>
cudaError_t two_passes(const LayerNormBwd& a, const Choice& c, cudaStream_t stream, int* launches) {
    if (a.dW || a.dbias) {   // first: dX may be dR, or dY
        const int lanes = col_lanes(a.d);
        const dim3 grid(static_cast<unsigned>((a.d + 8 * lanes - 1) / (8 * lanes)), static_cast<unsigned>(c.grid));
        const int cluster = c.parts == 1 ? c.grid : 1;
        const cudaError_t e = launch_clusters(layer_norm_dw_kernel<T, TY, VEC>, grid, dim3(1, static_cast<unsigned>(cluster), 1),
                                              kColThreads, 0, stream, a, lanes, cluster);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    const int64_t nv = (a.d + 7) / 8;
    int v = a.rows <= 2 * static_cast<int64_t>(a.num_sms) ? 1 : 2;
    while (v < 4 && (nv + v - 1) / v > 1024) v *= 2;
    const unsigned threads = static_cast<unsigned>(((nv + v - 1) / v + 31) / 32 * 32);
    const auto kern = v == 1 ? layer_norm_dx_kernel<T, TY, 1, VEC>
                      : v == 2 ? layer_norm_dx_kernel<T, TY, 2, VEC> : layer_norm_dx_kernel<T, TY, 4, VEC>;
    return launch_chained(kern, dim3(static_cast<unsigned>(a.rows)), threads, 0, stream, a,
                          reinterpret_cast<uintptr_t>(a.W) % 16 == 0);
}

template <typename T, typename TY>
cudaError_t bwd_type(const LayerNormBwd& a, cudaStream_t stream, int* launches) {
    const Choice c = choose(a);
    const bool vec = bwd_vec(a);
    *launches = 0;
    cudaError_t e;
    if (c.way == kByWarps)
        e = by_warps<T, TY>(a, c, stream);
    else if (c.way == kByRing)
        e = by_ring<T, TY>(a, c.ring, stream);
    else if (c.way == kOdd)
        e = by_odd<T, TY>(a, c.ring, stream);
    else
        e = vec ? two_passes<T, TY, true>(a, c, stream, launches) : two_passes<T, TY, false>(a, c, stream, launches);
    if (e != cudaSuccess) return e;
    ++*launches;
    if (a.parts == 1 || !(a.dW || a.dbias)) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>((a.d + 15) / 16), a.dW && a.dbias ? 2 : 1);
    e = launch_chained(layer_norm_join_kernel, grid, 256, 0, stream, a, a.dW ? 0 : 1);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace

int layer_norm_bwd_parts(const LayerNormBwd& a) { return choose(a).parts; }

cudaError_t launch_layer_norm_bwd(const LayerNormBwd& a, cudaStream_t stream, int* launches) {
    const bool xb = a.x_type == GEMM_DTYPE_BF16, yb = a.y_type == GEMM_DTYPE_BF16;
    return xb ? (yb ? bwd_type<__nv_bfloat16, __nv_bfloat16>(a, stream, launches) : bwd_type<__nv_bfloat16, float>(a, stream, launches))
              : (yb ? bwd_type<float, __nv_bfloat16>(a, stream, launches) : bwd_type<float, float>(a, stream, launches));
}

}  // namespace gemm
