// What the kernels of the bfloat16 products share: the operands' layouts in
// shared memory, the MMA, and the epilogue.
#pragma once

#include "activation.cuh"
#include "f8_tc.cuh"
#include "layer.h"

namespace gemm {

constexpr int kLinBK = 64;             // K elements per step: 128 bytes of a row
constexpr int kLinMmaK = 16;           // K of one MMA

struct LinearParams {
    const float* bias;
    const void* R;
    __nv_bfloat16* Z;
    void* D;
    int* err;
    int64_t ldd, ldr, ldz;
    int m, n;
    int num_kb;                // K steps
    int tiles_m, tiles_n;
    int act;
    bool grad, out_f32;
    bool mn_a, mn_b;           // A, B stored with their rows (columns of D) contiguous instead of K
    bool vec;                  // D, R, Z and bias take vectors of four elements
    bool halves;               // two-SM kernel: every tile in halves of 128 columns
};

// Shared-memory descriptor of an operand tile written by TMA with the 128-byte
// swizzle, 1024-byte aligned.  K-major: 128-byte rows of 64 K elements, groups
// of eight rows 1024 bytes apart.  MN-major: boxes of 64 rows of the operand
// (contiguous, 128 bytes) by 64 K elements; the stride byte offset is that of
// eight K elements (1024 bytes), the leading byte offset that of the next 64 rows
// (a box of 8 KiB).  Fields as in smem_desc_sw128_kmajor.
constexpr int kLinBoxBytes = 64 * 128;
__device__ __forceinline__ uint64_t smem_desc_linear(uint32_t saddr, bool mn) {
    return smem_desc_sw128_kmajor(saddr) + (mn ? static_cast<uint64_t>((kLinBoxBytes >> 4) - 1) << 16 : 0ull);
}
// What one MMA's 16 K elements add to the descriptor: 32 bytes of a row, or
// sixteen rows of 128 bytes.
__device__ __forceinline__ uint32_t desc_step(bool mn) { return mn ? 128u : 2u; }

// Instruction descriptor: bfloat16 operands (idesc_f16), bits 15 and 16 set
// for MN-major A and B.
__host__ __device__ constexpr uint32_t idesc_linear(bool mn_a, bool mn_b, uint32_t M, uint32_t N) {
    return idesc_f16(1u, M, N) | (mn_a ? 1u << 15 : 0u) | (mn_b ? 1u << 16 : 0u);
}

template <int CTAS>
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
    if constexpr (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        mma_f16_ss(d_tmem, a_desc, b_desc, idesc, accumulate);
}

// Elements of D's type as fp32, and back.
template <bool F32>
__device__ __forceinline__ float load_out(const void* p, int64_t i) {
    if constexpr (F32)
        return static_cast<const float*>(p)[i];
    else
        return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <bool F32>
__device__ __forceinline__ void store_out(void* p, int64_t i, float v) {
    if constexpr (F32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Four values of a row as loaded (bfloat16: two words, fp32: four).
template <bool F32>
struct Four {
    uint32_t w[F32 ? 4 : 2];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        if constexpr (F32) {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
            w[0] = u.x; w[1] = u.y;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (uint32_t& x : w) x = 0u;
    }
    __device__ __forceinline__ float at(int t) const {
        if constexpr (F32) return __uint_as_float(w[t]);
        return __uint_as_float(t & 1 ? w[t >> 1] & 0xffff0000u : w[t >> 1] << 16);
    }
};
template <bool F32>
__device__ __forceinline__ void store_four(void* p, int64_t i, float a, float b, float c, float d) {
    if constexpr (F32)
        *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(a, b, c, d);
    else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) = make_uint2(bf16x2(a, b), bf16x2(c, d));
}

// The epilogue of a warp's 32 x 32 block of sums in its staging buffer
// (stage_rows32): rows row0.., columns col0...  Whole aligned blocks: a lane
// takes four columns of every fourth row, so that eight lanes move one row's
// piece.  What is read (residual, Z) is asked for before the sums are used.
template <bool F32>
__device__ __forceinline__ void finish_block(const LinearParams& p, uint32_t stg, int lane, int row0, int col0) {
    const int col = col0 + (lane & 7) * 4, r0 = lane >> 3;
    auto at = [&](int j, int64_t ld) { return static_cast<int64_t>(row0 + r0 + 4 * j) * ld + col; };
    auto in = [&](int j) { return row0 + r0 + 4 * j < p.m; };
    float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.bias) bias = __ldg(reinterpret_cast<const float4*>(p.bias + col));
    Four<false> z[8];
    Four<F32> r[8];
    const bool read_z = p.grad && p.Z;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        z[j].zero();
        if (read_z && in(j)) z[j].load(p.Z, at(j, p.ldz));
    }
    if (p.R)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (in(j)) r[j].load(p.R, at(j, p.ldr)); else r[j].zero();
    float v[32];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int row = r0 + 4 * j;
        const uint4 u = ld_shared_v4(stg + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
        v[4 * j] = __uint_as_float(u.x) + bias.x;
        v[4 * j + 1] = __uint_as_float(u.y) + bias.y;
        v[4 * j + 2] = __uint_as_float(u.z) + bias.z;
        v[4 * j + 3] = __uint_as_float(u.w) + bias.w;
    }
    if (p.Z && !p.grad)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (in(j)) store_four<false>(p.Z, at(j, p.ldz), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    activate_all<32>(p.act, p.grad, v, [&](int i) { return z[i >> 2].at(i & 3); });
    if (p.R)
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += r[i >> 2].at(i & 3);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (in(j)) store_four<F32>(p.D, at(j, p.ldd), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}

// N rows of one column (row0.. by steps of one; `rows` of them exist), for
// blocks at a ragged edge and unaligned rows: the lanes of a warp hold
// neighbouring columns, so that every access is contiguous along a row
// whatever its alignment.  v: the sums.
template <bool F32, int N>
__device__ __forceinline__ void finish_column(const LinearParams& p, int row0, int rows, int col, float (&v)[N]) {
    if (col >= p.n) rows = 0;
    const float bias = p.bias && rows > 0 ? __ldg(p.bias + col) : 0.f;
    auto at = [&](int i, int64_t ld) { return static_cast<int64_t>(row0 + i) * ld + col; };
    float z[N], r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = p.grad && p.Z && i < rows ? __bfloat162float(p.Z[at(i, p.ldz)]) : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = p.R && i < rows ? load_out<F32>(p.R, at(i, p.ldr)) : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += bias;
    if (p.Z && !p.grad)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < rows) p.Z[at(i, p.ldz)] = __float2bfloat16_rn(v[i]);
    activate_all<N>(p.act, p.grad, v, [&](int i) { return z[i]; });
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < rows) store_out<F32>(p.D, at(i, p.ldd), p.R ? v[i] + r[i] : v[i]);
}
template <bool F32>
__device__ __forceinline__ void finish_ragged(const LinearParams& p, uint32_t stg, int lane, int row0, int col0) {
    constexpr int N = 8;   // rows in flight
#pragma unroll 1
    for (int j = 0; j < 32 && row0 + j < p.m; j += N) {
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __uint_as_float(staged_at(stg, j + i, lane));
        finish_column<F32, N>(p, row0 + j, min(N, p.m - row0 - j), col0 + lane, v);
    }
}

// Host: the kernels' parameters for tiles of bm x bn of D.
LinearParams linear_params(const LinearLaunch& a, int bm, int bn);
// Host: tensor map of a bfloat16 matrix (rows x cols, row pitch ld), boxes of
// 64 columns x box_rows, 128-byte swizzle; what lies outside reads as zero.
bool encode_bf16(CUtensorMap* map, const void* ptr, int64_t cols, int64_t rows, int64_t ld, int box_rows);
// The same for operand A or B of a product, as its form stores it: boxes of
// box_rows of its rows (columns of D for B) x 64 K elements, or, MN-major, of 64
// rows x 64 K elements.
bool encode_operand(CUtensorMap* map, const LinearLaunch& a, bool is_b, int box_rows);

}  // namespace gemm
