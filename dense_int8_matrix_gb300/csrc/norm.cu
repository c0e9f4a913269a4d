// RMS norm with the residual's addition and an 8-bit output, and its
// gradient.
//
//   h = x + r,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * w
//   dx = dr + rstd * (g - xhat * mean(g * xhat)),  g = dy * w, xhat = h * rstd
//   dw = sum over rows of dy * xhat
//
// Both are bound by DRAM: every element is read and written once.  GB300,
// 8192 x 8192: bfloat16 forward with residual 81 us (86 % of the measured copy
// rate; int8 95 us), backward with dw 83 us (97 %); fp32 139 and 223 us (93 and
// 72 %).  Rows that are not whole 16-byte words: forward 39 to 48 % (8192 x 8191
// 145 us, 16385 x 1001 37), backward 33 to 58 % (138 and 54 us).
#include "f8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gemm {

namespace {

// Sum (or largest, NaN if any value is) over the CTA; `red` is used by this
// call alone.
template <bool MAX>
__device__ __forceinline__ float cta_reduce(float v, float* red) {
    v = MAX ? warp_max_or_nan(v) : warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
    return MAX ? warp_max_or_nan(v) : warp_sum(v);
}

// One CTA per row, or (WARP, rows of at most 768 elements) a warp per row and
// kWarpRows rows per CTA, which spares the CTA's barriers and most of its
// launches (bfloat16 on GB300: 46323 x 622 95 -> 76 us, 19018 x 384 22 -> 15; at
// 1024 elements a CTA per row is faster, 23 against 25).  The row stays in
// registers (V vectors of eight values per thread, vector v of thread t at
// column 8 * (v * threads + t), so sixteen neighbouring lanes hold one block of
// 128 columns).  The mean square is taken of h as it is stored.
constexpr int kWarpRows = 8;
template <typename T, int V, bool I8, bool VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : 1024) norm_fwd_kernel(const NormFwd p, bool qvec, bool wvec) {
    __shared__ float red[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= p.rows) return;   // whole warps, and no barrier of the CTA
    const T* x = static_cast<const T*>(p.X) + row * p.ldx;
    const T* r = p.R ? static_cast<const T*>(p.R) + row * p.ldr : nullptr;
    Vec8<T> h[V];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = 8 * (static_cast<int64_t>(v) * nt + t);
        h[v] = load8<VEC>(x, c, p.d);
        if (r) {
            float a[8], b[8];
            h[v].get(a);
            load8<VEC>(r, c, p.d).get(b);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] += b[i];
            h[v].set(a);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = 8 * (static_cast<int64_t>(v) * nt + t);
        if (p.H) store8<VEC>(static_cast<T*>(p.H) + row * p.ldh, c, p.d, h[v]);
        float a[8];
        h[v].get(a);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += a[i] * a[i];
    }
    ss = WARP ? warp_sum(ss) : cta_reduce<false>(ss, red[0]);
    const float mean = ss / static_cast<float>(p.d) + p.eps;
    const float rstd = 1.f / sqrtf(mean);
    if (t == 0 && p.rstd) p.rstd[row] = rstd;
    float y[V][8];
    float amax = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = 8 * (static_cast<int64_t>(v) * nt + t);
        float w[8];
        load8_f32(p.W, c, p.d, wvec, w);
        h[v].get(y[v]);
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[v][i] = y[v][i] * rstd * w[i];
            a = I8 ? max_or_nan(a, fabsf(y[v][i])) : fmaxf(a, fabsf(y[v][i]));
        }
        if constexpr (I8) {
            amax = max_or_nan(amax, a);
        } else {
            const float s = block_scale(half_warp_max(a), kE4M3Step);
            const float inv = __frcp_rn(s);
            if (c < p.d) {
                store8_bytes(static_cast<uint8_t*>(p.Q) + row * p.ldq, c, p.d, qvec,
                             f8x4<GEMM_F8_E4M3>(y[v][0] * inv, y[v][1] * inv, y[v][2] * inv, y[v][3] * inv),
                             f8x4<GEMM_F8_E4M3>(y[v][4] * inv, y[v][5] * inv, y[v][6] * inv, y[v][7] * inv));
                if ((t & 15) == 0) p.scale[(c / kF8Block) * p.rows + row] = s;
            }
        }
    }
    if constexpr (I8) {
        amax = WARP ? warp_max_or_nan(amax) : cta_reduce<true>(amax, red[1]);
        // int8 holds no NaN: the row's scale carries it, be it of h (mean) or of
        // y alone (a NaN in w, 0 * inf), and the row's values are then zeros
        const float s = isfinite(mean) && !isnan(amax) ? block_scale(amax, kI8Step) : __int_as_float(0x7fc00000);
        const float inv = __frcp_rn(s);
        if (t == 0) p.scale[row] = s;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = 8 * (static_cast<int64_t>(v) * nt + t);
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

// Persistent CTAs over the rows.  A thread owns the same columns of every row
// (eight per vector), and dw's running sums of the CTA's rows stay in shared
// memory, one word per thread and column so that no two lanes share a bank.
// They go to `partial`, which dw_reduce_kernel adds up in CTA order.  It takes
// what the ring kernel below does not: fp32, rows beyond 8192 elements, few
// rows.  The whole row is held in registers, which 1024 threads do not have for
// wide rows: bfloat16 with four vectors per thread and fp32 with two spill 160 to
// 256 bytes, fp32 with four (32 registers) about 2 KB.  GB300, bfloat16 2048 x
// 16384 79 us (51 % of the measured copy rate), 2048 x 32768 185 (43 %); fp32
// 8192 x 8192 223 (72 %), 2048 x 16384 140 (57 %), 2048 x 32768 559 (29 %).
template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const NormBwd p, bool wvec) {
    extern __shared__ float dw[];   // [V * 8][threads]
    __shared__ float red[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int threads = blockDim.x, t = threadIdx.x;
    if (p.dW)
#pragma unroll
        for (int i = 0; i < 8 * V; ++i) dw[i * threads + t] = 0.f;
    auto column = [&](int v) { return 8 * (static_cast<int64_t>(v) * threads + t); };
    struct Row {
        Vec8<T> dy[V], h[V], dr[V];
        float rstd;
    };
    auto fetch = [&](int64_t row, Row& x) {
        x.rstd = __ldg(p.rstd + row);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x.dy[v] = load8<VEC>(static_cast<const T*>(p.dY) + row * p.lddy, column(v), p.d);
            x.h[v] = load8<VEC>(static_cast<const T*>(p.H) + row * p.ldh, column(v), p.d);
            if (p.dR)
                x.dr[v] = load8<VEC>(static_cast<const T*>(p.dR) + row * p.lddr, column(v), p.d);
            else
                x.dr[v].zero();
        }
    };
    Row x;
    if (blockIdx.x < p.rows) fetch(blockIdx.x, x);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float w[8], a[8], b[8];
            load8_f32(p.W, column(v), p.d, wvec, w);
            x.dy[v].get(a);
            x.h[v].get(b);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot += a[i] * w[i] * (b[i] * x.rstd);
        }
        const float mean = cta_reduce<false>(dot, red[turn]) / static_cast<float>(p.d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float w[8], a[8], b[8], o[8];
            load8_f32(p.W, column(v), p.d, wvec, w);
            x.dy[v].get(a);
            x.h[v].get(b);
            x.dr[v].get(o);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // written out so that dX has the same bits with and without dW
                const float xhat = __fmul_rn(b[i], x.rstd);
                o[i] = __fmaf_rn(x.rstd, __fmaf_rn(a[i], w[i], -__fmul_rn(xhat, mean)), o[i]);
                float* s = dw + (v * 8 + i) * threads + t;
                if (p.dW) *s = __fmaf_rn(a[i], xhat, *s);
            }
            Vec8<T> out;
            out.set(o);
            store8<VEC>(static_cast<T*>(p.dX) + row * p.lddx, column(v), p.d, out);
        }
        if (row + gridDim.x < p.rows) fetch(row + gridDim.x, x);
    }
    if (p.dW) {
        float* out = gridDim.x > 1 ? p.partial + static_cast<int64_t>(blockIdx.x) * p.d : p.dW;
#pragma unroll
        for (int i = 0; i < 8 * V; ++i) {
            const int64_t c = column(i / 8) + i % 8;
            if (c < p.d) out[c] = dw[i * threads + t];
        }
    }
}

// The same for bfloat16 rows of at most 1024 vectors, as training has them: w
// and dw's running sums stay in registers (512 threads at most, V vectors
// each), and the rows come through a ring in shared memory, copied several
// rows ahead by one thread (bulk copies, up to 200 KB per SM on their way).
// VEC: rows are 16-byte aligned and of whole vectors.  Otherwise a row is
// copied with the 16-byte words that it shares with its neighbours and shifted
// on the way to the registers; a row whose words would reach past the matrix
// (the first or the last) is loaded without the ring.
constexpr int kBwdThreads = 512;
constexpr int kBwdRingBytes = 200 * 1024;
constexpr int kBwdSlots = 8;
constexpr int kRowsPerCta = 6;

// Bytes of one array's row in a slot, and of a slot.
__host__ __device__ inline uint32_t ring_row_bytes(int64_t d, bool vec) {
    return static_cast<uint32_t>(vec ? d * 2 : (d * 2 + 15) / 16 * 16 + 32);   // + the shared words, + what the last shift reads
}

template <int V, bool VEC>
__global__ void __launch_bounds__(kBwdThreads, 1) norm_bwd_ring_kernel(const NormBwd p, bool wvec, int slots, int* err) {
    using T = __nv_bfloat16;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][32];
    __shared__ __align__(8) uint64_t bars[kBwdSlots];
    __shared__ uint32_t abort_flag;
    const int threads = blockDim.x, t = threadIdx.x;
    const uint32_t row_bytes = ring_row_bytes(p.d, VEC);
    const uint32_t slot_bytes = row_bytes * (p.dR ? 3 : 2);
    const uint32_t ring0 = smem_u32(ring), bar0 = smem_u32(bars);
    if (t == 0) {
        for (int s = 0; s < slots; ++s) mbar_init(bar0 + 8u * s, 1);
        abort_flag = 0u;
        fence_barrier_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();
    auto column = [&](int v) { return 8 * (v * threads + t); };
    const int d = static_cast<int>(p.d);
    const uintptr_t len = static_cast<uintptr_t>(d) * 2;
    auto row_at = [&](const void* base, int64_t ld, int64_t row) { return reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + row * ld); };
    // the 16-byte words of a row lie inside the matrix if 15 bytes before and
    // behind it do: all rows but the first and the last few
    int64_t least = p.lddy < p.ldh ? p.lddy : p.ldh;
    if (p.dR && p.lddr < least) least = p.lddr;
    const int64_t margin = (15 + 2 * least - 1) / (2 * least);
    auto ringed = [&](int64_t row) { return VEC || (row >= margin && row < p.rows - margin); };
    // copies row `row` into slot s (one thread)
    auto copy_row = [&](int64_t row, int s) {
        const uint32_t bar = bar0 + 8u * s, dst = ring0 + s * slot_bytes;
        if (!ringed(row)) {
            mbar_arrive(bar);
            return;
        }
        const uintptr_t a[3] = {row_at(p.dY, p.lddy, row), row_at(p.H, p.ldh, row), p.dR ? row_at(p.dR, p.lddr, row) : 0};
        uint32_t n[3], all = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            n[i] = i < 2 || p.dR ? static_cast<uint32_t>(((a[i] + len + 15) & ~static_cast<uintptr_t>(15)) - (a[i] & ~static_cast<uintptr_t>(15))) : 0;
            all += n[i];
        }
        mbar_arrive_expect_tx(bar, all);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (n[i]) bulk_load(dst + i * row_bytes, reinterpret_cast<const void*>(a[i] & ~static_cast<uintptr_t>(15)), n[i], bar);
    };
    const int64_t step = gridDim.x;
    if (t == 0)
        for (int s = 0; s < slots && blockIdx.x + s * step < p.rows; ++s) copy_row(blockIdx.x + s * step, s);
    float w[V][8], dw[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        load8_f32(p.W, column(v), p.d, wvec, w[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.f;
    }
    const float inv_d = 1.f / static_cast<float>(p.d);
    int s = 0, turn = 0;
    uint32_t ph = 0;
    float rs = blockIdx.x < p.rows ? __ldg(p.rstd + blockIdx.x) : 0.f;
    for (int64_t row = blockIdx.x; row < p.rows; row += step, turn ^= 1) {
        const float rstd = rs;
        if (row + step < p.rows) rs = __ldg(p.rstd + row + step);
        // a wait that gives up is recorded; the rows are then wrong, and every
        // copy still lands in the ring before the CTA ends (see below)
        wait_bounded(bar0 + 8u * s, ph, &abort_flag, err, kDevErrTimeoutProducer);
        Vec8<T> dy[V], h[V], dr[V];
        const bool in_ring = ringed(row);
        auto take = [&](int array, const void* base, int64_t ld, int v, Vec8<T>& x) {
            const uint8_t* src = ring + s * slot_bytes + array * row_bytes + column(v) * 2;
            if (column(v) >= d) {
                x.zero();
            } else if (VEC) {
                x.u = *reinterpret_cast<const uint4*>(src);
            } else if (in_ring) {
                const uint4 a = reinterpret_cast<const uint4*>(src)[0], b = reinterpret_cast<const uint4*>(src)[1];
                const uint32_t in[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                uint32_t out[4];
                shift_words<4>(in, static_cast<int>(row_at(base, ld, row) & 15), out);
                if (column(v) + 8 > d) {   // what lies behind the row's end is not its own
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (column(v) + 2 * i >= d) out[i] = 0u;
                        else if (column(v) + 2 * i + 1 >= d) out[i] &= 0xffffu;
                    }
                }
                x.words(out);
            } else {
                x = load8<false>(reinterpret_cast<const T*>(row_at(base, ld, row)), column(v), d);
            }
        };
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            take(0, p.dY, p.lddy, v, dy[v]);
            take(1, p.H, p.ldh, v, h[v]);
            if (p.dR)
                take(2, p.dR, p.lddr, v, dr[v]);
            else
                dr[v].zero();
            float a[8], x[8];
            dy[v].get(a);
            h[v].get(x);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot += a[i] * w[v][i] * (x[i] * rstd);
        }
        // every thread has read the slot once it is past this reduction
        dot = warp_sum(dot);
        if ((t & 31) == 0) red[turn][t >> 5] = dot;
        __syncthreads();
        if (t == 0 && row + slots * step < p.rows) copy_row(row + slots * step, s);
        dot = (t & 31) < (threads >> 5) ? red[turn][t & 31] : 0.f;
        const float mean = warp_sum(dot) * inv_d;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a[8], x[8], o[8];
            dy[v].get(a);
            h[v].get(x);
            dr[v].get(o);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // written out so that dX has the same bits with and without dW
                const float xhat = __fmul_rn(x[i], rstd);
                o[i] = __fmaf_rn(rstd, __fmaf_rn(a[i], w[v][i], -__fmul_rn(xhat, mean)), o[i]);
                dw[v][i] = __fmaf_rn(a[i], xhat, dw[v][i]);
            }
            Vec8<T> out;
            out.set(o);
            store8<VEC>(static_cast<T*>(p.dX) + row * p.lddx, column(v), p.d, out);
        }
        if (++s == slots) {
            s = 0;
            ph ^= 1u;
        }
    }
    // Every copy has been waited for above, unless a wait gave up: then the
    // last phase of each slot once more, so that nothing lands after the end.
    if (abort_flag && t == 0) {
        const int64_t mine = blockIdx.x < p.rows ? (p.rows - blockIdx.x + step - 1) / step : 0;
        for (int64_t j = mine > slots ? mine - slots : 0; j < mine; ++j)
            wait_bounded(bar0 + 8u * static_cast<uint32_t>(j % slots), static_cast<uint32_t>(j / slots) & 1u, nullptr, err,
                         kDevErrTimeoutTeardown);
    }
    if (p.dW) {
        float* out = gridDim.x > 1 ? p.partial + static_cast<int64_t>(blockIdx.x) * p.d : p.dW;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float4* o = reinterpret_cast<float4*>(out + column(v));
            if (column(v) + 8 <= d && reinterpret_cast<uintptr_t>(o) % 16 == 0) {
                o[0] = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
                o[1] = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (column(v) + i < d) out[column(v) + i] = dw[v][i];
            }
        }
    }
}

// dW_j = sum of the CTAs' sums.  A CTA takes eight columns (a sector of 32
// bytes of each partial), so that short rows, which leave many partials and few
// columns, still use many SMs; its 32 groups of eight lanes take every 32nd
// partial, four loads at a time, and are joined in a fixed order.
__global__ void __launch_bounds__(256) dw_reduce_kernel(const float* partial, int parts, int64_t d, float* dW) {
    constexpr int kLoads = 4, kGroups = 32;
    __shared__ float red[8][8];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 8 + (lane & 7);
    float s = 0.f;
    if (c < d) {
        for (int i = warp * 4 + (lane >> 3); i < parts; i += kLoads * kGroups) {
            float v[kLoads];
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                v[j] = i + j * kGroups < parts ? partial[static_cast<int64_t>(i + j * kGroups) * d + c] : 0.f;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) s += v[j];
        }
    }
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if (lane < 8) red[warp][lane] = s;
    __syncthreads();
    if (threadIdx.x < 8 && c < d) {
        s = red[0][lane];
#pragma unroll
        for (int i = 1; i < 8; ++i) s += red[i][lane];
        dW[c] = s;
    }
}

bool al16(const void* p, int64_t pitch_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && pitch_bytes % 16 == 0;
}

// Threads and vectors per thread of a row of d elements.  Many rows at once
// run best with two vectors per thread (8192 x 8192 bfloat16 on GB300: 1, 2 and
// 4 vectors 92, 79 and 88 us), int8 ones of more than 6144 elements, which wait
// at a second barrier, with four (97, 106 and 93; 2048 x 12288 two 56, four 47);
// a few rows run sooner with one.
void row_shape(int64_t rows, int64_t d, bool to_i8, int num_sms, int* threads, int* vecs) {
    const int64_t nv = (d + 7) / 8;
    int v = rows <= 2 * static_cast<int64_t>(num_sms) ? 1 : to_i8 && d > 6144 ? 4 : 2;
    while (v < 4 && (nv + v - 1) / v > 1024) v *= 2;
    *threads = static_cast<int>(((nv + v - 1) / v + 31) / 32 * 32);
    *vecs = v;
}

template <typename T>
bool fwd_vec(const NormFwd& a) {
    const int64_t es = sizeof(T);
    return al16(a.X, a.ldx * es) && (!a.R || al16(a.R, a.ldr * es)) && (!a.H || al16(a.H, a.ldh * es));
}

template <typename T, int V, bool VEC, bool WARP>
cudaError_t fwd_launch(const NormFwd& a, int threads, cudaStream_t stream) {
    const bool qvec = reinterpret_cast<uintptr_t>(a.Q) % 8 == 0 && a.ldq % 8 == 0;
    const bool wvec = reinterpret_cast<uintptr_t>(a.W) % 16 == 0;
    const int64_t grid = WARP ? (a.rows + kWarpRows - 1) / kWarpRows : a.rows;
    return launch_chained(a.to_i8 ? norm_fwd_kernel<T, V, true, VEC, WARP> : norm_fwd_kernel<T, V, false, VEC, WARP>,
                          dim3(static_cast<unsigned>(grid)), threads, 0, stream, a, qvec, wvec);
}

template <typename T, bool VEC>
cudaError_t fwd_aligned(const NormFwd& a, cudaStream_t stream) {
    // a warp per row, once there is a CTA of such for every SM
    if (a.d <= 768 && a.rows >= static_cast<int64_t>(kWarpRows) * a.num_sms) {
        constexpr int kThreads = 32 * kWarpRows;
        return a.d <= 256 ? fwd_launch<T, 1, VEC, true>(a, kThreads, stream)
               : a.d <= 512 ? fwd_launch<T, 2, VEC, true>(a, kThreads, stream) : fwd_launch<T, 3, VEC, true>(a, kThreads, stream);
    }
    int t, v;
    row_shape(a.rows, a.d, a.to_i8, a.num_sms, &t, &v);
    return v == 1 ? fwd_launch<T, 1, VEC, false>(a, t, stream) : v == 2 ? fwd_launch<T, 2, VEC, false>(a, t, stream)
                                                                        : fwd_launch<T, 4, VEC, false>(a, t, stream);
}

template <typename T>
cudaError_t fwd_type(const NormFwd& a, cudaStream_t stream) {
    return fwd_vec<T>(a) ? fwd_aligned<T, true>(a, stream) : fwd_aligned<T, false>(a, stream);
}

// One vector per thread up to 8192 columns.
void bwd_shape(int64_t d, int* threads, int* vecs) {
    const int64_t nv = (d + 7) / 8;
    int v = 1;
    while ((nv + v - 1) / v > 1024) v *= 2;
    *threads = static_cast<int>(((nv + v - 1) / v + 31) / 32 * 32);
    *vecs = v;
}

// Whether the ring kernel takes the call: bfloat16 rows that fit its registers
// and enough of them to fill its rings.
bool bwd_ring(const NormBwd& a) { return a.x_type == GEMM_DTYPE_BF16 && a.d <= 16 * kBwdThreads && a.rows > a.num_sms; }

template <typename T>
bool bwd_vec(const NormBwd& a) {
    const int64_t es = sizeof(T);
    return al16(a.dY, a.lddy * es) && al16(a.H, a.ldh * es) && (!a.dR || al16(a.dR, a.lddr * es)) && al16(a.dX, a.lddx * es);
}
bool ring_vec(const NormBwd& a) { return a.d % 8 == 0 && bwd_vec<__nv_bfloat16>(a); }

// Threads of a ring CTA, CTAs per SM (two vectors per thread take 128
// registers) and rows in its ring.  At least six rows per CTA where two CTAs
// per SM leave that many: each CTA adds d sums to what dw_reduce_kernel reads
// (8192 x 512 on GB300: 17.7 us with all 16 CTAs per SM, 13.2 with eight).  The
// count takes 1024 threads per SM, which the form for aligned rows has registers
// for (63 a thread).  That for unaligned ones (95) has them for 640, so of eight
// CTAs of 128 threads five run at once and the others start as these end; and of
// 32 CTAs of one warp with full rings about 30 fit in shared memory, of which
// each holds 1 KiB besides.
void ring_shape(const NormBwd& a, int* threads, int* per_sm, int* slots) {
    const int64_t nv = (a.d + 7) / 8;
    const int v = nv <= kBwdThreads ? 1 : 2;
    *threads = static_cast<int>(((nv + v - 1) / v + 31) / 32 * 32);
    const int64_t enough = a.rows / (kRowsPerCta * static_cast<int64_t>(a.num_sms));
    const int most = v == 1 ? 1024 / *threads : 1;
    *per_sm = enough < 2 ? (most < 2 ? most : 2) : enough < most ? static_cast<int>(enough) : most;
    const int64_t fit = kBwdRingBytes / *per_sm / (static_cast<int64_t>(ring_row_bytes(a.d, ring_vec(a))) * (a.dR ? 3 : 2));
    *slots = static_cast<int>(fit < kBwdSlots ? fit : kBwdSlots);
}

template <int V, bool VEC>
cudaError_t ring_launch(const NormBwd& a, cudaStream_t stream) {
    int threads, per_sm, slots;
    ring_shape(a, &threads, &per_sm, &slots);
    const auto kern = norm_bwd_ring_kernel<V, VEC>;
    const cudaError_t e = kernel_attrs_once(reinterpret_cast<const void*>(kern), kBwdRingBytes, true);
    if (e != cudaSuccess) return e;
    return launch_chained(kern, dim3(static_cast<unsigned>(a.grid)), threads,
                          static_cast<size_t>(slots) * ring_row_bytes(a.d, VEC) * (a.dR ? 3 : 2), stream, a,
                          reinterpret_cast<uintptr_t>(a.W) % 16 == 0, slots, a.err);
}

template <typename T, int V, bool VEC>
cudaError_t rows_launch(const NormBwd& a, int threads, cudaStream_t stream) {
    const size_t smem = a.dW ? static_cast<size_t>(8 * V) * threads * 4 : 0;
    const auto kern = norm_bwd_kernel<T, V, VEC>;
    if (smem > 47 * 1024) {   // 48 KiB hold the static arrays too
        const cudaError_t e = kernel_attrs_once(reinterpret_cast<const void*>(kern), GEMM_NORM_MAX_D * 4, false);
        if (e != cudaSuccess) return e;
    }
    return launch_chained(kern, dim3(static_cast<unsigned>(a.grid)), threads, smem, stream, a,
                          reinterpret_cast<uintptr_t>(a.W) % 16 == 0);
}

template <typename T, bool VEC>
cudaError_t rows_aligned(const NormBwd& a, cudaStream_t stream) {
    int t, v;
    bwd_shape(a.d, &t, &v);
    return v == 1 ? rows_launch<T, 1, VEC>(a, t, stream) : v == 2 ? rows_launch<T, 2, VEC>(a, t, stream)
                                                                  : rows_launch<T, 4, VEC>(a, t, stream);
}

template <typename T>
cudaError_t rows_type(const NormBwd& a, cudaStream_t stream) {
    return bwd_vec<T>(a) ? rows_aligned<T, true>(a, stream) : rows_aligned<T, false>(a, stream);
}

cudaError_t ring_type(const NormBwd& a, cudaStream_t stream) {
    if (ring_vec(a)) return a.d <= 8 * kBwdThreads ? ring_launch<1, true>(a, stream) : ring_launch<2, true>(a, stream);
    return a.d <= 8 * kBwdThreads ? ring_launch<1, false>(a, stream) : ring_launch<2, false>(a, stream);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwd& a, cudaStream_t stream) {
    return a.x_type == GEMM_DTYPE_BF16 ? fwd_type<__nv_bfloat16>(a, stream) : fwd_type<float>(a, stream);
}

// Persistent CTAs, each with its own dw: as many as run at once (more of some
// unaligned and short rows, see ring_shape).
int norm_bwd_grid(const NormBwd& a) {
    if (bwd_ring(a)) {
        int threads, per_sm, slots;
        ring_shape(a, &threads, &per_sm, &slots);
        const int64_t g = static_cast<int64_t>(a.num_sms) * per_sm;
        return static_cast<int>(a.rows < g ? a.rows : g);
    }
    int t, v;
    bwd_shape(a.d, &t, &v);
    const int64_t g = static_cast<int64_t>(a.num_sms) * (1024 / t);
    return static_cast<int>(a.rows < g ? a.rows : g);
}

cudaError_t launch_norm_bwd(const NormBwd& a, cudaStream_t stream) {
    cudaError_t e = bwd_ring(a) ? ring_type(a, stream)
                    : a.x_type == GEMM_DTYPE_BF16 ? rows_type<__nv_bfloat16>(a, stream) : rows_type<float>(a, stream);
    if (e == cudaSuccess && a.dW && a.grid > 1)
        e = launch_chained(dw_reduce_kernel, dim3(static_cast<unsigned>((a.d + 7) / 8)), 256, 0, stream, a.partial, a.grid,
                           a.d, a.dW);
    return e;
}

}  // namespace gemm
