// Balance loss of a router with the experts' counts, and its gradient.
//
//   p = softmax(x),  f = counts / sum(counts),  P = mean of p over the rows that take part
//   loss = coef * E * sum(f * P)
//   dx = dr + dloss * coef * E / T * p * (f - sum(f * p))
//
// The logits are read once by each pass.  65536 x 256 fp32: forward 25 us (20 of them
// the rows, bound by instructions and the latency of a row's sums: 20
// instructions per logit, as long from the L2 as from DRAM), gradient 32 us, 6.3
// TB/s, bound by DRAM.  L lanes (as many as
// have sixteen columns each, 32 at most) hold a row, so that a warp takes 32 / L
// rows at once, whatever the number of experts, and a lane has the same columns
// of every row: its sums of p stay with it.  (Four columns per lane leave the
// same work per row to be done for fewer rows at once.)  The next row is on its
// way while one is worked on (with nine to sixteen experts, a row to a lane, 216 to 316
// bytes of its registers spill; otherwise eight at most).  Sums are joined in a fixed order: rows of a lane, row
// groups of a warp, warps of a CTA, the eight CTAs of a cluster (through
// distributed shared memory), and clusters by a second kernel.  Batches that
// one cluster (or one CTA) takes in a few turns need no second kernel.
#include <algorithm>
#include <type_traits>

#include "activation.cuh"
#include "f8_tc.cuh"
#include "internal.h"
#include "layer.h"

namespace gemm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kLossThreads = 1024;
constexpr int kRowsPerSum = 32;   // rows added in a row before they join the running sum
constexpr int kFewTurns = 4;      // of rows, up to which one cluster takes a whole batch
constexpr float kInf = __builtin_huge_valf();
constexpr int kExpertsPerThread = GEMM_BALANCE_MAX_EXPERTS / kThreads;
constexpr int kMaxParts = 256;
static_assert(kLossThreads >= GEMM_BALANCE_MAX_EXPERTS && kMaxParts <= kLossThreads && kLossThreads == 1024, "a thread per expert and per part");

__device__ __forceinline__ int32_t ld_cluster_i32(uint32_t addr) {
    int32_t v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// A lane's columns of a row: four at 4 * (l + L * u) for each u < U; -infinity
// past the row.  VEC: rows take vectors of four.
template <int L, int U>
__device__ __forceinline__ int column(int l, int i) { return 4 * (l + L * (i >> 2)) + (i & 3); }
template <typename T, int L, int U, bool VEC>
__device__ __forceinline__ void load_row(const T* x, int l, int e, float fill, float (&a)[4 * U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = 4 * (l + L * u);
        if constexpr (VEC) {
            if (c < e) {
                if constexpr (sizeof(T) == 4) {
                    const float4 v = *reinterpret_cast<const float4*>(x + c);
                    a[4 * u] = v.x; a[4 * u + 1] = v.y; a[4 * u + 2] = v.z; a[4 * u + 3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(x + c);
                    a[4 * u] = __uint_as_float(v.x << 16); a[4 * u + 1] = __uint_as_float(v.x & 0xffff0000u);
                    a[4 * u + 2] = __uint_as_float(v.y << 16); a[4 * u + 3] = __uint_as_float(v.y & 0xffff0000u);
                }
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t) a[4 * u + t] = fill;
            }
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) a[4 * u + t] = c + t < e ? to_f32(x[c + t]) : fill;
        }
    }
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int L, typename V>
__device__ __forceinline__ V group_sum(V v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// exp(a - largest) of a row in place, and 1 / their sum (0 for a row of
// -infinity alone, whose p are 0); a NaN or +infinity makes the sum NaN.
template <int L, int N>
__device__ __forceinline__ float exponentials(float (&a)[N], float& base, float& sum) {
    float top = a[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, a[i]);
    top = group_max<L>(top);
    base = top == -kInf ? 0.f : top;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        a[i] = exp_approx(a[i] - base);
        sum += a[i];
    }
    sum = group_sum<L>(sum);
    return sum == 0.f ? 0.f : rcp_approx(sum);
}

// Counts, offsets, means and the loss from the counts and sums of p of experts
// N t .. N t + N - 1 in thread t, and the used rows.  One CTA of WARPS warps.
template <int N, int WARPS>
__device__ __forceinline__ void write_loss(const Balance& p, const int32_t (&count)[N], const float (&sum)[N], int32_t rows) {
    __shared__ int32_t scan[WARPS];
    __shared__ float red[WARPS];
    const int e = p.experts, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int32_t mine = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) mine += count[i];
    int32_t before = mine;   // of the warp's threads up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t up = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += up;
    }
    if (lane == 31) scan[warp] = before;
    before -= mine;
    __syncthreads();
    int32_t slots = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += scan[w];
        slots += scan[w];
    }
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = N * t + i;
        before += count[i];
        if (c >= e) continue;
        const float prob = rows > 0 ? sum[i] / static_cast<float>(rows) : 0.f;
        const float share = slots > 0 ? static_cast<float>(count[i]) / static_cast<float>(slots) : 0.f;
        l += share * prob;
        p.counts[c] = count[i];
        p.probs[c] = prob;
        if (p.offsets) p.offsets[c + 1] = before;
    }
    l = warp_sum(l);
    if (lane == 0) red[warp] = l;
    __syncthreads();
    if (warp == 0) {
        l = warp_sum(lane < WARPS ? red[lane] : 0.f);
        if (lane == 0) {
            if (p.offsets) p.offsets[0] = 0;
            *p.used = rows;
            *p.loss = p.coef * static_cast<float>(e) * l;
        }
    }
}

template <typename T, int L, int U, bool VEC>
__global__ void __launch_bounds__(kThreads, U == 8 ? 2 : 3) balance_rows_kernel(const Balance p, int cluster) {
    constexpr int N = 4 * U, kGroups = 32 / L;
    constexpr bool kCountInRegisters = L == 1;   // (at most 16 experts: shared counters would be fought over)
    // counts[experts + 1] (the last one: used rows), sums[warps][experts], running sums[N][threads]
    extern __shared__ int32_t shared[];
    int32_t* hist = shared;
    float* sums = reinterpret_cast<float*>(shared + p.experts + 1);
    float* total = sums + kWarps * p.experts + threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = p.experts;
    const int l = lane % L, group = lane / L;
    for (int i = threadIdx.x; i <= e; i += kThreads) hist[i] = 0;
    __syncthreads();
    float part[N], x[2][N];
    int32_t slot[2], counted[kCountInRegisters ? N : 1], used_rows = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) total[i * kThreads] = part[i] = 0.f;
#pragma unroll
    for (int32_t& c : counted) c = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kGroups;
    int64_t row = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kGroups + group;
    const T* at = static_cast<const T*>(p.X) + row * p.ldx;
    const int32_t* index = p.index + row * p.top_k + l;
    const int64_t at_step = step * p.ldx, index_step = step * p.top_k;
    int64_t ahead = row;   // the row that `at` and `index` point to
    auto fetch = [&](float (&a)[N], int32_t& s) {
        s = -1;
        if (ahead < p.rows) {
            load_row<T, L, U, VEC>(at, l, e, -kInf, a);
            if (l < p.top_k) s = __ldg(index);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] = -kInf;
        }
        at += at_step;
        index += index_step;
        ahead += step;
    };
    auto work = [&](float (&a)[N], int32_t s) {
        const bool mine = row < p.rows;
        bool taken = false;
        for (int k = 0;;) {
            const bool in = static_cast<uint32_t>(s) < static_cast<uint32_t>(e);
            taken = taken || in;
            if constexpr (kCountInRegisters) {
#pragma unroll
                for (int i = 0; i < N; ++i) counted[i] += s == column<L, U>(l, i) ? 1 : 0;
            } else if (in) {
                atomicAdd(hist + s, 1);
            }
            k += L;
            if (k >= p.top_k) break;
            s = mine && k + l < p.top_k ? __ldg(p.index + row * p.top_k + k + l) : -1;
        }
        const uint32_t votes = __ballot_sync(0xffffffffu, taken);
        const bool used = ((votes >> (lane & ~(L - 1))) & (L == 32 ? 0xffffffffu : (1u << (L % 32)) - 1u)) != 0;
        float base, sum;
        const float inv = exponentials<L, N>(a, base, sum);
        if (l == 0 && mine) p.lse[row] = used ? base + log_approx(sum) : kInf;   // (sum is 1 to 1024, or 0, or NaN)
        if (used) {   // (padding takes no part, whatever it holds)
            if (l == 0) ++used_rows;
#pragma unroll
            for (int i = 0; i < N; ++i) part[i] = fmaf(a[i], inv, part[i]);
        }
        row += step;
    };
    // a warp's rows: while any of its groups has one, and the second of each
    // two may be past the end
    int64_t first = row - group;
    fetch(x[0], slot[0]);
    for (int pending = 0; first < p.rows; first += 2 * step) {
        fetch(x[1], slot[1]);
        work(x[0], slot[0]);
        fetch(x[0], slot[0]);
        work(x[1], slot[1]);
        if ((pending += 2) == kRowsPerSum) {
            pending = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                total[i * kThreads] += part[i];
                part[i] = 0.f;
            }
        }
    }
    // the warp's row groups, then the CTA's warps
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float v = total[i * kThreads] + part[i];
#pragma unroll
        for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int c = column<L, U>(l, i);
        if (group == 0 && c < e) sums[warp * e + c] = v;
        if constexpr (kCountInRegisters) {
#pragma unroll
            for (int o = L; o < 32; o <<= 1) counted[i] += __shfl_xor_sync(0xffffffffu, counted[i], o);
            if (group == 0 && c < e && counted[i]) atomicAdd(hist + c, counted[i]);
        }
    }
    used_rows = group_sum<32>(used_rows);
    if (lane == 0 && used_rows) atomicAdd(hist + e, used_rows);
    __syncthreads();
    for (int c = threadIdx.x; c < e; c += kThreads) {
        float s = sums[c];
        for (int w = 1; w < kWarps; ++w) s += sums[w * e + c];
        sums[c] = s;   // (its only reader)
    }
    // the cluster's CTAs
    const uint32_t hist0 = smem_u32(hist), sums0 = smem_u32(sums);
    auto joined_count = [&](int c) {
        if (cluster == 1) return hist[c];
        int32_t v[kCluster], all = 0;   // (asked for together: a remote read takes its time)
#pragma unroll
        for (int r = 0; r < kCluster; ++r) v[r] = ld_cluster_i32(peer_address(hist0 + 4 * c, r));
#pragma unroll
        for (int r = 0; r < kCluster; ++r) all += v[r];
        return all;
    };
    auto joined_sum = [&](int c) {
        if (cluster == 1) return sums[c];
        float v[kCluster], all = 0.f;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) v[r] = load_in_cluster(peer_address(sums0 + 4 * c, r));
#pragma unroll
        for (int r = 0; r < kCluster; ++r) all += v[r];
        return all;
    };
    if (cluster > 1)
        cluster_barrier();
    else
        __syncthreads();
    const int rank = static_cast<int>(blockIdx.x) % cluster, id = static_cast<int>(blockIdx.x) / cluster;
    if (p.parts == 1) {
        if (rank == 0) {
            auto join = [&](auto n) {   // experts per thread
                constexpr int kPer = decltype(n)::value;
                int32_t count[kPer];
                float sum[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int c = kPer * static_cast<int>(threadIdx.x) + i;
                    count[i] = c < e ? joined_count(c) : 0;
                    sum[i] = c < e ? joined_sum(c) : 0.f;
                }
                write_loss<kPer, kWarps>(p, count, sum, joined_count(e));
            };
            if (e <= kThreads)
                join(std::integral_constant<int, 1>{});
            else
                join(std::integral_constant<int, kExpertsPerThread>{});
        }
    } else {
        for (int c = rank + cluster * static_cast<int>(threadIdx.x); c <= e; c += cluster * kThreads) {
            p.partial_c[static_cast<int64_t>(id) * (e + 1) + c] = joined_count(c);
            if (c < e) p.partial_p[static_cast<int64_t>(id) * e + c] = joined_sum(c);
        }
    }
    if (cluster > 1) cluster_barrier();   // the others' shared memory has been read
}

// The clusters' sums: as many threads per expert as there are, each with every
// groups-th cluster, joined in order.
__global__ void __launch_bounds__(kLossThreads) balance_loss_kernel(const Balance p) {
    __shared__ int32_t counts[kLossThreads], used[kLossThreads / 32];
    __shared__ float sums[kLossThreads];
    pdl_launch_dependents();
    pdl_wait();
    const int e = p.experts, t = threadIdx.x;
    const int per = (e + 31) / 32 * 32, groups = kLossThreads / per;   // (whole warps read neighbouring experts)
    const int c = t % per, g = t / per;
    int32_t count[1] = {0}, rows = 0;
    float sum[1] = {0.f};
    if (t < p.parts) rows = p.partial_c[static_cast<int64_t>(t) * (e + 1) + e];   // (parts are at most kMaxParts)
    if (c < e && g < groups) {
        constexpr int kLoads = 12;   // at a time: the latency of the L2 is what this kernel takes
        for (int j = g; j < p.parts; j += kLoads * groups) {
            int32_t n[kLoads];
            float f[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int64_t part = j + i * groups;
                n[i] = part < p.parts ? p.partial_c[part * (e + 1) + c] : 0;
                f[i] = part < p.parts ? p.partial_p[part * e + c] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                count[0] += n[i];
                sum[0] += f[i];
            }
        }
    }
    counts[t] = count[0];
    sums[t] = sum[0];
    rows = group_sum<32>(rows);
    if ((t & 31) == 0) used[t >> 5] = rows;
    __syncthreads();
    rows = group_sum<32>(used[t & 31]);
    count[0] = 0;
    sum[0] = 0.f;
    if (t < e)
        for (int i = 0; i < groups; ++i) {
            count[0] += counts[i * per + t];
            sum[0] += sums[i * per + t];
        }
    write_loss<1, kLossThreads / 32>(p, count, sum, rows);
}

template <typename T, int L, int U, bool VEC>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(const BalanceBwd p) {
    constexpr int N = 4 * U, kGroups = 32 / L;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = p.experts;
    const int l = lane % L, group = lane / L;
    int32_t slots = 0;
    float f[N], a[N], d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = column<L, U>(l, i);
        const int32_t n = c < e ? __ldg(p.counts + c) : 0;
        slots += n;
        f[i] = static_cast<float>(n);
    }
    slots = group_sum<L>(slots);
    const int32_t used = __ldg(p.used);
    const float per_slot = slots > 0 ? 1.f / static_cast<float>(slots) : 0.f;
    const float scale = used > 0 ? __ldg(p.dloss) * p.coef * static_cast<float>(e) / static_cast<float>(used) : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] *= per_slot;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kGroups;
    for (int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kGroups; first < p.rows; first += step) {
        const int64_t row = first + group;
        const bool mine = row < p.rows;
        const float lse = mine ? __ldg(p.lse + row) : kInf;
        const bool part = !isinf(lse);   // not padding, nor a row without any p
        if (mine) {
            load_row<T, L, U, VEC>(static_cast<const T*>(p.X) + row * p.ldx, l, e, -kInf, a);
            if (p.dR) load_row<T, L, U, VEC>(static_cast<const T*>(p.dR) + row * p.lddr, l, e, 0.f, d);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!mine) a[i] = -kInf;
            if (!mine || !p.dR) d[i] = 0.f;
        }
        // p is formed from the row again: exp(x - lse) would carry lse's rounding
        float base, sum, mix = 0.f;
        const float inv = exponentials<L, N>(a, base, sum);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            a[i] *= inv;
            mix = fmaf(a[i], f[i], mix);   // (past the row both are zero)
        }
        mix = group_sum<L>(mix);
        if (!mine) continue;
        if (part)
#pragma unroll
            for (int i = 0; i < N; ++i) d[i] = fmaf(scale * a[i], f[i] - mix, d[i]);
        T* dx = static_cast<T*>(p.dX) + row * p.lddx;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = 4 * (l + L * u);
            if constexpr (VEC) {
                if (c < e) {
                    if constexpr (sizeof(T) == 4)
                        *reinterpret_cast<float4*>(dx + c) = make_float4(d[4 * u], d[4 * u + 1], d[4 * u + 2], d[4 * u + 3]);
                    else
                        *reinterpret_cast<uint2*>(dx + c) = make_uint2(bf16x2(d[4 * u], d[4 * u + 1]), bf16x2(d[4 * u + 2], d[4 * u + 3]));
                }
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (c + t < e) from_f32(d[4 * u + t], dx + c + t);
            }
        }
    }
}

// Lanes of a row: sixteen columns each, or, for a batch of few rows, four (64
// rows of 32 experts: 4.0 us with sixteen, 2.8 with four).
int lanes_of(int experts, bool few) {
    int l = 1;
    while (l < 32 && (few ? 4 : 16) * l < experts) l *= 2;
    return l;
}
int rows_per_turn(int experts, bool few) { return kWarps * 32 / lanes_of(experts, few); }   // of a CTA
bool few_rows(int64_t rows, int experts) { return rows <= static_cast<int64_t>(kFewTurns) * kCluster * rows_per_turn(experts, true); }

bool takes_fours(const void* p, int64_t ld, int es, int experts) {
    return !p || (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(4 * es) == 0 && ld % 4 == 0 && experts % 4 == 0);
}

// f(L, U as integral constants)
template <typename F>
cudaError_t by_experts(int experts, bool few, F f) {
#define GEMM_LANES(L, U) return f(std::integral_constant<int, L>{}, std::integral_constant<int, U>{});
    if (experts <= 4) GEMM_LANES(1, 1)
    if (few && experts <= 256) switch (lanes_of(experts, true)) {
        case 2: GEMM_LANES(2, 1)
        case 4: GEMM_LANES(4, 1)
        case 8: GEMM_LANES(8, 1)
        case 16: GEMM_LANES(16, 1)
        default: break;
    }
    if (few && experts <= 128) GEMM_LANES(32, 1)
    if (few && experts <= 256) GEMM_LANES(32, 2)
    if (experts <= 8) GEMM_LANES(1, 2)
    switch (lanes_of(experts, false)) {
        case 1: GEMM_LANES(1, 4)
        case 2: GEMM_LANES(2, 4)
        case 4: GEMM_LANES(4, 4)
        case 8: GEMM_LANES(8, 4)
        case 16: GEMM_LANES(16, 4)
        default: break;
    }
    if (experts <= 512) GEMM_LANES(32, 4)
    GEMM_LANES(32, 8)
#undef GEMM_LANES
}

int cluster_of(const Balance& a) {
    return a.rows <= 2 * static_cast<int64_t>(rows_per_turn(a.experts, few_rows(a.rows, a.experts))) ? 1 : kCluster;
}

template <typename T, bool VEC>
cudaError_t rows_launch(const Balance& a, cudaStream_t stream) {
    return by_experts(a.experts, few_rows(a.rows, a.experts), [&](auto L, auto U) -> cudaError_t {
        const auto kern = balance_rows_kernel<T, decltype(L)::value, decltype(U)::value, VEC>;
        constexpr int kRunning = 4 * decltype(U)::value * kThreads * 4;
        const size_t smem = static_cast<size_t>(a.experts + 1 + kWarps * a.experts) * 4 + kRunning;   // at most 69 KB
        const cudaError_t e = kernel_attrs_once(reinterpret_cast<const void*>(kern),
                                                (GEMM_BALANCE_MAX_EXPERTS * (kWarps + 1) + 1) * 4 + kRunning, false);
        if (e != cudaSuccess) return e;
        int cluster = cluster_of(a);
        cudaLaunchConfig_t cfg;
        std::memset(&cfg, 0, sizeof(cfg));
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(a.parts * cluster), 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        const cudaError_t r = cudaLaunchKernelEx(&cfg, kern, a, cluster);
        return r != cudaSuccess ? r : cudaGetLastError();
    });
}

template <typename T, bool VEC>
cudaError_t bwd_launch(const BalanceBwd& a, cudaStream_t stream) {
    const bool few = few_rows(a.rows, a.experts);
    const int64_t turn = rows_per_turn(a.experts, few);
    const int64_t blocks = (a.rows + turn - 1) / turn, most = 8 * static_cast<int64_t>(a.num_sms);
    return by_experts(a.experts, few, [&](auto L, auto U) {
        return launch_chained(balance_bwd_kernel<T, decltype(L)::value, decltype(U)::value, VEC>,
                              dim3(static_cast<unsigned>(blocks < most ? blocks : most)), kThreads, 0, stream, a);
    });
}

}  // namespace

// Clusters of the first kernel: one for batches of a few turns, else as many
// as run at once.  A cluster's CTAs lie in one GPC, so that not every SM is
// full: at three CTAs per SM (two beyond 512 experts) 48 (32) run at once, and
// further ones would start only as those end (65536 x 256: 25.5 us with 48, 37 with
// 54; 16384 x 1024 30.6 with 32, 41.5 with 40).
int balance_parts(const Balance& a) {
    const bool few = few_rows(a.rows, a.experts);
    const int64_t turn = static_cast<int64_t>(kCluster) * rows_per_turn(a.experts, few);
    if (a.rows <= kFewTurns * turn) return 1;
    const int64_t most = static_cast<int64_t>(a.experts <= 512 ? 48 : 32) * a.num_sms / 152, parts = (a.rows + turn - 1) / turn;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(parts, most), kMaxParts)));
}

cudaError_t launch_balance(const Balance& a, cudaStream_t stream, int* launches) {
    *launches = 0;
    const bool bf = a.x_type == GEMM_DTYPE_BF16, vec = takes_fours(a.X, a.ldx, bf ? 2 : 4, a.experts);
    cudaError_t e = bf ? (vec ? rows_launch<__nv_bfloat16, true>(a, stream) : rows_launch<__nv_bfloat16, false>(a, stream))
                       : (vec ? rows_launch<float, true>(a, stream) : rows_launch<float, false>(a, stream));
    if (e != cudaSuccess) return e;
    ++*launches;
    if (a.parts == 1) return cudaSuccess;
    e = launch_chained(balance_loss_kernel, dim3(1), kLossThreads, 0, stream, a);
    if (e == cudaSuccess) ++*launches;
    return e;
}

cudaError_t launch_balance_bwd(const BalanceBwd& a, cudaStream_t stream) {
    const bool bf = a.x_type == GEMM_DTYPE_BF16;
    const int es = bf ? 2 : 4;
    const bool vec = takes_fours(a.X, a.ldx, es, a.experts) && takes_fours(a.dR, a.lddr, es, a.experts) &&
                     takes_fours(a.dX, a.lddx, es, a.experts);
    return bf ? (vec ? bwd_launch<__nv_bfloat16, true>(a, stream) : bwd_launch<__nv_bfloat16, false>(a, stream))
              : (vec ? bwd_launch<float, true>(a, stream) : bwd_launch<float, false>(a, stream));
}

}  // namespace gemm
