// The gradient of an activation and of the bias before it, and the copy of
// unaligned operands to aligned rows.
//
//   dz = dy * act'(z),  dbias[j] = sum_i dy[i][j] * act'(z[i][j])
//
// Bound by DRAM: every element is read and written once.  A thread takes eight
// columns of a range of rows and keeps their sums; the sums of a CTA are joined
// in shared memory and those of the row ranges by launch_column_sums, both in a
// fixed order.
#include "activation.cuh"
#include "f8.cuh"
#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

namespace gemm {

namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kRowsAtOnce = 4;   // rows in flight per thread

// `lanes` neighbouring threads (a power of two, 32 for unaligned rows, whose
// stores go by whole warps) hold 8 * lanes columns of a row.
template <int ACT, bool VEC>
__global__ void __launch_bounds__(kThreads) act_bwd_kernel(const ActBwd p, int lanes) {
    __shared__ float red[kThreads * 8];
    pdl_launch_dependents();
    pdl_wait();
    const int groups = kThreads / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * lanes + lane) * 8;
    const int64_t per = (p.rows + p.parts - 1) / p.parts;
    const int64_t lo = per * blockIdx.y, hi = lo + per < p.rows ? lo + per : p.rows;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t r0 = lo + group; r0 < hi; r0 += static_cast<int64_t>(kRowsAtOnce) * groups) {
        Vec8<bf16> dy[kRowsAtOnce], z[kRowsAtOnce];
#pragma unroll
        for (int k = 0; k < kRowsAtOnce; ++k) {
            const int64_t r = r0 + static_cast<int64_t>(k) * groups;
            dy[k].zero();
            z[k].zero();
            if (r < hi && c < p.cols) {
                dy[k] = load8<VEC>(static_cast<const bf16*>(p.dY) + r * p.lddy, c, p.cols);
                if (p.Z) z[k] = load8<VEC>(static_cast<const bf16*>(p.Z) + r * p.ldz, c, p.cols);
            }
        }
#pragma unroll
        for (int k = 0; k < kRowsAtOnce; ++k) {
            const int64_t r = r0 + static_cast<int64_t>(k) * groups;
            float g[8], s[8];
            dy[k].get(g);
            z[k].get(s);
            activate_each<ACT | GEMM_ACT_GRADIENT, 8>(g, [&](int i) { return s[i]; });
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += g[i];
            if (p.dZ && r < hi) {   // (lanes == 32 without VEC: the whole warp)
                Vec8<bf16> o;
                o.set(g);
                store8<VEC>(static_cast<bf16*>(p.dZ) + r * p.lddz, c, p.cols, o);
            }
        }
    }
    if (!p.dbias) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) red[group * lanes * 8 + lane * 8 + i] = sum[i];
    __syncthreads();
    float* out = p.parts > 1 ? p.partial + static_cast<int64_t>(blockIdx.y) * p.cols : p.dbias;
    for (int i = threadIdx.x; i < 8 * lanes; i += kThreads) {
        float v = red[i];
        for (int g = 1; g < groups; ++g) v += red[g * lanes * 8 + i];
        const int64_t col = static_cast<int64_t>(blockIdx.x) * lanes * 8 + i;
        if (col < p.cols) out[col] = v;
    }
}

// Eight elements per thread; the destination's rows are aligned, its pitch a
// multiple of eight, so that every store is a whole vector (what lies between
// the columns and the pitch is not used).
__global__ void __launch_bounds__(256) repitch_kernel(const bf16* src, int64_t ld, bf16* dst, int64_t pitch, int64_t rows,
                                                      int64_t cols) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t vecs = pitch / 8, all = rows * vecs, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all; i += step) {
        const int64_t r = i / vecs, c = (i - r * vecs) * 8;
        load8<false>(src + r * ld, c, cols).store(dst + r * pitch + c);
    }
}

bool vec_ok(const void* p, int64_t ld) { return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0); }
bool act_vec(const ActBwd& a) { return vec_ok(a.dY, a.lddy) && vec_ok(a.Z, a.ldz) && vec_ok(a.dZ, a.lddz); }

int act_lanes(const ActBwd& a) {
    int lanes = 32;
    if (act_vec(a))
        while (lanes > 1 && 4 * lanes >= a.cols) lanes /= 2;
    return lanes;
}

}  // namespace

// Row ranges: about eight CTAs per SM over all column blocks, each thread with
// at least two turns of rows.
int act_bwd_parts(const ActBwd& a) {
    const int lanes = act_lanes(a);
    const int64_t blocks = (a.cols + 8 * lanes - 1) / (8 * lanes);
    const int64_t turn = static_cast<int64_t>(kRowsAtOnce) * (kThreads / lanes);
    int64_t parts = (8 * static_cast<int64_t>(a.num_sms) + blocks - 1) / blocks;
    const int64_t most = (a.rows + 2 * turn - 1) / (2 * turn);
    if (parts > most) parts = most;
    return static_cast<int>(parts < 1 ? 1 : parts);
}

cudaError_t launch_act_bwd(const ActBwd& a, cudaStream_t stream) {
    const int lanes = act_lanes(a);
    const dim3 grid(static_cast<unsigned>((a.cols + 8 * lanes - 1) / (8 * lanes)), static_cast<unsigned>(a.parts));
    auto go = [&](auto kern) { return launch_chained(kern, grid, kThreads, 0, stream, a, lanes); };
    const bool vec = act_vec(a);
    cudaError_t e;
    switch (a.act) {
        case GEMM_ACT_RELU: e = go(vec ? act_bwd_kernel<GEMM_ACT_RELU, true> : act_bwd_kernel<GEMM_ACT_RELU, false>); break;
        case GEMM_ACT_GELU: e = go(vec ? act_bwd_kernel<GEMM_ACT_GELU, true> : act_bwd_kernel<GEMM_ACT_GELU, false>); break;
        case GEMM_ACT_GELU_TANH:
            e = go(vec ? act_bwd_kernel<GEMM_ACT_GELU_TANH, true> : act_bwd_kernel<GEMM_ACT_GELU_TANH, false>);
            break;
        case GEMM_ACT_SILU: e = go(vec ? act_bwd_kernel<GEMM_ACT_SILU, true> : act_bwd_kernel<GEMM_ACT_SILU, false>); break;
        default: e = go(vec ? act_bwd_kernel<GEMM_ACT_NONE, true> : act_bwd_kernel<GEMM_ACT_NONE, false>); break;
    }
    if (e == cudaSuccess && a.dbias && a.parts > 1) e = launch_column_sums(a.partial, a.parts, a.cols, a.dbias, stream);
    return e;
}

cudaError_t launch_repitch(const void* src, int64_t ld, void* dst, int64_t pitch, int64_t rows, int64_t cols, int num_sms,
                           cudaStream_t stream) {
    const int64_t blocks = (rows * (pitch / 8) + 255) / 256, most = 16 * static_cast<int64_t>(num_sms);
    return launch_chained(repitch_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, 0, stream,
                          static_cast<const bf16*>(src), ld, static_cast<bf16*>(dst), pitch, rows, cols);
}

}  // namespace gemm
