// The gradient of an activation and of the bias before it, and the copy of
// unaligned operands to aligned rows.
//
//   dz = dy * act'(z),  dbias[j] = sum_i dy[i][j] * act'(z[i][j])
//
// Bound by DRAM: every element is read and written once (4096 x 16384, GELU_TANH:
// 81 us, 4.9 TB/s; RELU 73 us, 5.5 TB/s; more rows in flight per thread spill or
// cost CTAs).  A thread takes eight columns of a range of rows and keeps their
// sums; the sums of a CTA are joined in shared memory, those of the row ranges
// of a cluster through distributed shared memory, and those of clusters by
// launch_column_sums, all in a fixed order.  Small problems are one cluster
// deep: one launch and no scratch (2050 x 777, the sums alone: 7.3 us, 12.4
// through scratch).
#include <algorithm>
#include <type_traits>

#include "activation.cuh"
#include "f8_tc.cuh"
#include "internal.h"
#include "layer.h"

namespace gemm {

namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kPerSm = 4;        // CTAs (of 64 registers per thread)

// How a row is read.  kVectors: eight columns per thread, sixteen-byte aligned.
// kShifted: the matrices are not aligned so, but lie alike (equal address and
// pitch modulo sixteen bytes): the rows of a thread are a multiple of eight
// apart and all start equally far past a boundary, so that the thread takes the
// eight elements from a boundary to the next, and the ends of a row are what
// the first and last lane hold of it.  kSingles: one column per thread
// (measured, 55369 x 453, GELU_TANH: 45 us shifted, 128 as singles).
enum { kVectors, kShifted, kSingles };

// Rows in flight per thread: about as many as the registers of kPerSm CTAs hold
// (four rows of RELU spill 32 to 100 bytes; the others do not).
template <int ACT, int MODE>
constexpr int kRows = MODE == kSingles ? 8 : ACT <= GEMM_ACT_RELU ? 4 : 2;

// W elements of row r from column c (that may start before the row or end
// behind it).  What is before the matrix's first element or behind its last is
// not read; other elements outside [first, last) are read and not used.
template <int MODE, int W>
__device__ __forceinline__ void load_piece(uint32_t (&w)[(W + 1) / 2], const void* m, int64_t ld, int64_t r, int64_t c, int first,
                                           int last, const ActBwd& p) {
    const int64_t off = r * ld + c;
    const bf16* at = static_cast<const bf16*>(m) + off;
    if (MODE == kSingles) {
        w[0] = *reinterpret_cast<const uint16_t*>(at);
    } else if (MODE == kVectors ? last == W : off >= 0 && off + W <= (p.rows - 1) * ld + p.cols) {
        const uint4 u = *reinterpret_cast<const uint4*>(at);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (i >= first && i < last) w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(at)[i]) << 16 * (i & 1);
    }
}

// `lanes` neighbouring threads (a power of two) hold p's `span` columns of a row.
template <int ACT, int MODE>
__global__ void __launch_bounds__(kThreads, kPerSm) act_bwd_kernel(const ActBwd p, int lanes, int span, int cluster) {
    constexpr int R = kRows<ACT, MODE>, W = MODE == kSingles ? 1 : 8;
    __shared__ float red[kThreads * W];
    pdl_launch_dependents();
    pdl_wait();
    const int groups = kThreads / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int64_t per = (p.rows + p.parts - 1) / p.parts;
    const int64_t lo = per * blockIdx.y, hi = lo + per < p.rows ? lo + per : p.rows;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * span;
    const int limit = p.cols - c0 < span ? static_cast<int>(p.cols - c0) : span;
    // This thread's elements: [first, last) of the W from column c0 + rel.
    const int before = MODE == kShifted
        ? static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const bf16*>(p.dY) + (lo + group) * p.lddy + c0) / 2 % 8) : 0;
    const int rel = lane * W - before, first = rel < 0 ? -rel : 0, last = limit - rel < W ? limit - rel : W;
    float sum[W];
#pragma unroll
    for (int i = 0; i < W; ++i) sum[i] = 0.f;
    for (int64_t r0 = lo + group; r0 < hi && first < last; r0 += static_cast<int64_t>(R) * groups) {
        uint32_t dy[R][(W + 1) / 2], z[R][(W + 1) / 2];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t r = r0 + static_cast<int64_t>(k) * groups;
#pragma unroll
            for (int i = 0; i < (W + 1) / 2; ++i) dy[k][i] = z[k][i] = 0u;
            if (r < hi) {
                load_piece<MODE, W>(dy[k], p.dY, p.lddy, r, c0 + rel, first, last, p);
                if (ACT != GEMM_ACT_NONE) load_piece<MODE, W>(z[k], p.Z, p.ldz, r, c0 + rel, first, last, p);
            }
        }
        auto value = [](const uint32_t(&w)[(W + 1) / 2], int i) { return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16); };
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t r = r0 + static_cast<int64_t>(k) * groups;
            float g[W];
#pragma unroll
            for (int i = 0; i < W; ++i) g[i] = value(dy[k], i);
            activate_each<ACT | GEMM_ACT_GRADIENT, W>(g, [&](int i) { return value(z[k], i); });
#pragma unroll
            for (int i = 0; i < W; ++i) sum[i] += g[i];   // (outside [first, last) another row's, and unused)
            if (!p.dZ || r >= hi) continue;
            bf16* out = static_cast<bf16*>(p.dZ) + r * p.lddz + c0 + rel;
            if (W == 1) {
                out[0] = __float2bfloat16_rn(g[0]);
            } else if (last - first == W) {
                uint4 u;
                u.x = bf16x2(g[0], g[1 % W]); u.y = bf16x2(g[2 % W], g[3 % W]);
                u.z = bf16x2(g[4 % W], g[5 % W]); u.w = bf16x2(g[6 % W], g[7 % W]);
                *reinterpret_cast<uint4*>(out) = u;
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (i >= first && i < last) out[i] = __float2bfloat16_rn(g[i]);
            }
        }
    }
    if (!p.dbias) return;   // (every CTA alike)
#pragma unroll
    for (int i = 0; i < W; ++i)
        if (i >= first && i < last) red[group * span + rel + i] = sum[i];
    __syncthreads();
    if (threadIdx.x < limit) {   // (limit <= span <= kThreads)
        float v = red[threadIdx.x];
        for (int g = 1; g < groups; ++g) v += red[g * span + threadIdx.x];
        red[threadIdx.x] = v;   // (its only reader)
    }
    float* out = p.parts > cluster ? p.partial + static_cast<int64_t>(blockIdx.y / cluster) * p.cols : p.dbias;
    join_cluster(red, limit, cluster, [&](int i, float v) { out[c0 + i] = v; });
}

// Rows of any alignment copied to aligned ones, of one matrix or two.  Eight
// elements of a thread are cut out of the two aligned vectors that they lie
// in (the second is the next lane's first, and mostly in the L1); at the ends
// of the matrix and of a row they are read one by one.  What lies between the
// columns and the pitch is not used.  A warp takes kCopies * 32 vectors of a
// row, or of neighbouring ones where rows are short.  Measured, 224 x 6401 and
// 1692 x 6401 (26 us): the product takes 8 us longer than on aligned rows (14 with
// elements read one by one).
constexpr int kCopies = 2;
// Eight elements from `past` (0 .. 7) on of two aligned vectors.
__device__ __forceinline__ uint4 cut(const uint4& x, const uint4& y, int past) {
    uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = past & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = past & 2 ? w[i + 1] : w[i];
    const uint32_t bits = 16 * (past & 1);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
}
// Lanes of a row: a power of two.
__host__ __device__ inline int repitch_lanes(const Repitch& m) {
    int lanes = 32;
    while (lanes > 1 && lanes * 4 >= m.pitch) lanes /= 2;
    return lanes;
}
// Pieces of kCopies * lanes vectors of a row.
__host__ __device__ inline int64_t repitch_pieces(const Repitch& m) {
    const int64_t span = static_cast<int64_t>(kCopies) * 8 * repitch_lanes(m);
    return (m.pitch + span - 1) / span;
}
__global__ void __launch_bounds__(256) repitch_kernel(const Repitch a, const Repitch b, int blocks_a) {
    pdl_launch_dependents();
    pdl_wait();
    const bool first = static_cast<int>(blockIdx.x) < blocks_a;
    const Repitch& m = first ? a : b;
    const int block = first ? blockIdx.x : blockIdx.x - blocks_a, blocks = first ? blocks_a : gridDim.x - blocks_a;
    const int lanes = repitch_lanes(m), groups = 256 / lanes, lane = threadIdx.x % lanes;
    const int64_t pieces = repitch_pieces(m), all = m.rows * pieces, step = static_cast<int64_t>(blocks) * groups;
    for (int64_t u = static_cast<int64_t>(block) * groups + threadIdx.x / lanes; u < all; u += step) {
        const int64_t r = all <= INT32_MAX ? static_cast<uint32_t>(u) / static_cast<uint32_t>(pieces) : u / pieces;
        const int64_t c0 = (u - r * pieces) * kCopies * 8 * lanes + 8 * lane;
        const bf16* row = static_cast<const bf16*>(m.src) + r * m.ld;
        const int past = static_cast<int>(reinterpret_cast<uintptr_t>(row) / 2 % 8);   // elements past a boundary
        const int64_t end = m.cols + (m.rows - 1 - r) * m.ld;   // the matrix's, from the row's first column
        uint4 x[kCopies], y[kCopies];
        bool whole[kCopies];
#pragma unroll
        for (int k = 0; k < kCopies; ++k) {
            const int64_t c = c0 + 8 * k * lanes;
            whole[k] = c + 8 <= m.cols && r * m.ld + c >= past && c + 16 <= end;
            x[k] = y[k] = make_uint4(0u, 0u, 0u, 0u);
            if (whole[k]) {
                const uint4* at = reinterpret_cast<const uint4*>(row + c - past);
                x[k] = at[0];
                y[k] = at[1];
            }
        }
#pragma unroll
        for (int k = 0; k < kCopies; ++k) {
            const int64_t c = c0 + 8 * k * lanes;
            if (c >= m.pitch) break;
            const uint4 v = whole[k] ? cut(x[k], y[k], past) : load8<false>(row, c, m.cols).u;
            *reinterpret_cast<uint4*>(static_cast<bf16*>(m.dst) + r * m.pitch + c) = v;
        }
    }
}

// How rows are read, and the threads and columns of a row in a CTA.
struct Shape {
    int mode, lanes, span;
};
Shape act_shape(const ActBwd& a) {
    const uintptr_t y = reinterpret_cast<uintptr_t>(a.dY);
    auto like = [&](const void* p, int64_t ld) {   // dY's rows, modulo sixteen bytes
        return !p || ((reinterpret_cast<uintptr_t>(p) - y) % 16 == 0 && (ld - a.lddy) % 8 == 0);
    };
    Shape s;
    s.mode = !like(a.Z, a.ldz) || !like(a.dZ, a.lddz) ? kSingles : y % 16 || a.lddy % 8 ? kShifted : kVectors;
    const int width = s.mode == kSingles ? 1 : 8;
    auto span = [&](int lanes) { return s.mode == kShifted ? (lanes - 1) * width : lanes * width; };
    s.lanes = 32;
    while (s.lanes > 2 && span(s.lanes / 2) >= a.cols) s.lanes /= 2;
    s.span = span(s.lanes);
    return s;
}

}  // namespace

// Row ranges: the CTAs of all column blocks run at once (clusters leave some
// room), each thread has at least two turns of four rows, and more than one
// cluster's are whole clusters.
int act_bwd_parts(const ActBwd& a) {
    const Shape s = act_shape(a);
    const int64_t blocks = (a.cols + s.span - 1) / s.span, turn = 4 * (kThreads / s.lanes);
    const int64_t at_once = std::max<int64_t>(1, static_cast<int64_t>(a.num_sms) * kPerSm * 7 / 8 / blocks);
    int64_t parts = std::min(at_once, (a.rows + 2 * turn - 1) / (2 * turn));
    if (parts > kMostClusterCtas) parts = parts / kMostClusterCtas * kMostClusterCtas;
    return static_cast<int>(parts);
}
int act_bwd_clusters(const ActBwd& a) { return a.parts <= kMostClusterCtas ? 1 : a.parts / kMostClusterCtas; }

cudaError_t launch_act_bwd(const ActBwd& a, cudaStream_t stream) {
    const Shape s = act_shape(a);
    const int cluster = std::min(a.parts, kMostClusterCtas);
    const dim3 grid(static_cast<unsigned>((a.cols + s.span - 1) / s.span), static_cast<unsigned>(a.parts));
    auto launch = [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        const auto kern = s.mode == kVectors ? act_bwd_kernel<ACT, kVectors>
                          : s.mode == kShifted ? act_bwd_kernel<ACT, kShifted> : act_bwd_kernel<ACT, kSingles>;
        return launch_clusters(kern, grid, dim3(1, static_cast<unsigned>(cluster), 1), kThreads, 0, stream, a, s.lanes, s.span, cluster);
    };
    cudaError_t e;
    switch (a.act) {
        case GEMM_ACT_RELU: e = launch(std::integral_constant<int, GEMM_ACT_RELU>{}); break;
        case GEMM_ACT_GELU: e = launch(std::integral_constant<int, GEMM_ACT_GELU>{}); break;
        case GEMM_ACT_GELU_TANH: e = launch(std::integral_constant<int, GEMM_ACT_GELU_TANH>{}); break;
        case GEMM_ACT_SILU: e = launch(std::integral_constant<int, GEMM_ACT_SILU>{}); break;
        default: e = launch(std::integral_constant<int, GEMM_ACT_NONE>{}); break;
    }
    const int clusters = act_bwd_clusters(a);
    if (e == cudaSuccess && a.dbias && clusters > 1) e = launch_column_sums(a.partial, clusters, a.cols, a.dbias, stream);
    return e;
}

cudaError_t launch_repitch(const Repitch& a, const Repitch& b, int num_sms, cudaStream_t stream) {
    const int64_t most = 8 * static_cast<int64_t>(num_sms);
    auto blocks = [&](const Repitch& m) {
        const int64_t groups = 256 / repitch_lanes(m);
        return static_cast<int>(std::min((m.rows * repitch_pieces(m) + groups - 1) / groups, most));
    };
    const int blocks_a = blocks(a);
    return launch_chained(repitch_kernel, dim3(static_cast<unsigned>(blocks_a + blocks(b))), 256, 0, stream, a, b, blocks_a);
}

}  // namespace gemm
