// What the kernels of the bfloat16 products share: the operands' layouts in
// shared memory, the MMA, and the epilogue.
#pragma once

#include <type_traits>

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
    int chunk;                 // K steps added up in TMEM, before they join sums in registers
    int first;                 // the same of a two-SM tile's first chunk
    int tiles_m, tiles_n;
    bool out_f32;
    bool mn_a, mn_b;           // A, B stored with their rows (columns of D) contiguous instead of K
    bool vec;                  // rows of D, R, Z and bias take vectors of eight elements
    bool pairs;                // rows of bfloat16 D, R and Z start at even elements
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

// Eight values of a row as loaded (bfloat16: four words, fp32: eight).
template <bool F32>
struct Eight {
    uint4 u[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    // Zeros unless `in`; volatile, as load_if.
    __device__ __forceinline__ void load_if(const uint8_t* p, bool in) {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i)
            asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
                         "mov.b32 %3, 0;\n\t@q ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
                         : "=&r"(u[i].x), "=&r"(u[i].y), "=&r"(u[i].z), "=&r"(u[i].w) : "l"(p + 16 * i), "r"(static_cast<int>(in)));
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (uint4& x : u) x = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ float at(int t) const {
        const uint4& x = u[F32 ? t >> 2 : 0];
        const int w = F32 ? t & 3 : t >> 1;
        const uint32_t y = w == 0 ? x.x : w == 1 ? x.y : w == 2 ? x.z : x.w;
        if constexpr (F32) return __uint_as_float(y);
        return __uint_as_float(t & 1 ? y & 0xffff0000u : y << 16);
    }
};
template <bool F32>
__device__ __forceinline__ void store_eight(uint8_t* p, const float* v) {
    if constexpr (F32) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    }
}

// The epilogue of a warp's 32 x 32 block of sums in its staging buffer
// (stage_rows32): rows row0.., columns col0...  Aligned rows: a lane takes eight
// columns of every eighth row, two rows at a time, so that four lanes move one
// row's piece (both ways through shared memory without bank conflicts).  What
// is read is asked for before the sums are used: all of Z (3373 x 142 x 3024
// with GELU's gradient: 30.0 us, 31.1 half by half), the residual half by half
// (21.4 us, 22.8 by load_if).  ACT: GEMM_ACT_*, with GEMM_ACT_GRADIENT or
// without.
template <bool F32, int ACT>
__device__ __forceinline__ void finish_block(const LinearParams& p, uint32_t stg, int lane, int row0, int row_end, int col0) {
    constexpr bool kReadZ = (ACT & GEMM_ACT_GRADIENT) != 0;
    constexpr int ES = F32 ? 4 : 2;
    const int part = lane & 3, r0 = lane >> 2;
    const int col = col0 + part * 8;
    if (col >= p.n) return;   // (n is a multiple of eight, or the block is whole)
    const int rows = row_end - row0 - r0;   // of the lane's rows r0 + 8 j, those with 8 j < rows exist
    float bias[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) bias[t] = 0.f;
    if (p.bias) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p.bias + col)), b = __ldg(reinterpret_cast<const float4*>(p.bias + col) + 1);
        bias[0] = a.x; bias[1] = a.y; bias[2] = a.z; bias[3] = a.w;
        bias[4] = b.x; bias[5] = b.y; bias[6] = b.z; bias[7] = b.w;
    }
    const int64_t row = row0 + r0;
    uint8_t* d = static_cast<uint8_t*>(p.D) + (row * p.ldd + col) * ES;
    uint8_t* zp = reinterpret_cast<uint8_t*>(p.Z) + (row * p.ldz + col) * 2;
    const uint8_t* rp = static_cast<const uint8_t*>(p.R) + (row * p.ldr + col) * ES;
    const int64_t sd = 8 * ES * p.ldd, sz = 16 * p.ldz, sr = 8 * ES * p.ldr;
    Eight<false> z[kReadZ ? 4 : 1];
    if constexpr (kReadZ)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j].load_if(zp + j * sz, 8 * j < rows);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        Eight<F32> r[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            r[i].zero();
            if (p.R && 8 * (2 * half + i) < rows) r[i].load(rp + (2 * half + i) * sr);
        }
        float v[16];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int rr = r0 + 8 * (2 * half + i);
                const uint4 u = ld_shared_v4(stg + rr * 128 + (((2 * part + k) ^ (rr & 7)) << 4));
                float* x = v + 8 * i + 4 * k;
                x[0] = __uint_as_float(u.x) + bias[4 * k];
                x[1] = __uint_as_float(u.y) + bias[4 * k + 1];
                x[2] = __uint_as_float(u.z) + bias[4 * k + 2];
                x[3] = __uint_as_float(u.w) + bias[4 * k + 3];
            }
        if constexpr (!kReadZ)
            if (p.Z)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (8 * (2 * half + i) < rows) store_eight<false>(zp + (2 * half + i) * sz, v + 8 * i);
        activate_each<ACT, 16>(v, [&](int i) { return kReadZ ? z[kReadZ ? 2 * half + (i >> 3) : 0].at(i & 7) : 0.f; });
        if (p.R)
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += r[i >> 3].at(i & 7);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (8 * (2 * half + i) < rows) store_eight<F32>(d + (2 * half + i) * sd, v + 8 * i);
    }
}

__device__ __forceinline__ void ld_shared_pair(uint32_t at, float& a, float& b) {
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(a), "=f"(b) : "r"(at) : "memory");
}
// Two or four bytes, 0 unless `in`.  (volatile: the loads of a batch are asked
// for together.  The compiler, short of registers, otherwise moves each to its
// use, and every one takes the latency of the L2: the ragged gradient of 3373 x
// 142 x 3021 76 us instead of 38.)
template <int BYTES>
__device__ __forceinline__ uint32_t load_if(const uint8_t* p, bool in) {
    uint32_t v;
    if constexpr (BYTES == 4)
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.b32 %0, [%1];\n\t}"
                     : "=&r"(v) : "l"(p), "r"(static_cast<int>(in)));
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.u16 %0, [%1];\n\t}"
                     : "=&r"(v) : "l"(p), "r"(static_cast<int>(in)));
    return v;
}
// One bfloat16 value, or two at an even element.
template <int W>
__device__ __forceinline__ void store_some(uint8_t* p, const float* v) {
    if constexpr (W == 2)
        *reinterpret_cast<uint32_t*>(p) = bf16x2(v[0], v[W - 1]);
    else
        *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(v[0]);
}

// Asks the L2 for the rows that the epilogue of rows row0 .. row0 + 31 and
// `cols` columns from col0 will read, a row per lane, while the products run.
template <bool READ_Z>
__device__ __forceinline__ void prefetch_rows(const LinearParams& p, int lane, int row0, int col0, int cols) {
    const int64_t row = row0 + lane;
    const int64_t n = min(cols, p.n - col0);
    if (row >= p.m || n <= 0) return;
    auto ask = [](const uint8_t* at, int64_t bytes) {
        for (int64_t i = 0; i < bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at + bytes - 1));
    };
    if constexpr (READ_Z) ask(reinterpret_cast<const uint8_t*>(p.Z + row * p.ldz + col0), 2 * n);
    const int64_t es = p.out_f32 ? 4 : 2;
    if (p.R) ask(static_cast<const uint8_t*>(p.R) + (row * p.ldr + col0) * es, es * n);
}

// N rows of one column (row0.. by steps of one; `rows` of them exist), for
// tiles of few rows, whose sums need no staging: the lanes of a warp hold neighbouring
// columns, so that every access is contiguous along a row whatever its
// alignment.  v: the sums.
template <bool F32, int ACT, int N>
__device__ __forceinline__ void finish_column(const LinearParams& p, int row0, int rows, int col, float (&v)[N]) {
    constexpr bool kReadZ = (ACT & GEMM_ACT_GRADIENT) != 0;
    if (col >= p.n) return;
    const float bias = p.bias ? __ldg(p.bias + col) : 0.f;
    auto at = [&](int i, int64_t ld) { return static_cast<int64_t>(row0 + i) * ld + col; };
    float z[N], r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        z[i] = kReadZ && i < rows ? __bfloat162float(p.Z[at(i, p.ldz)]) : 0.f;
        r[i] = p.R && i < rows ? load_out<F32>(p.R, at(i, p.ldr)) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += bias;
    if (!kReadZ && p.Z)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < rows) p.Z[at(i, p.ldz)] = __float2bfloat16_rn(v[i]);
    activate_each<ACT, N>(v, [&](int i) { return z[i]; });
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < rows) store_out<F32>(p.D, at(i, p.ldd), p.R ? v[i] + r[i] : v[i]);
}
// The same 32 x 32 block of a ragged edge, or of rows that are not aligned
// for vectors: a lane takes one column of every row, or (PAIRS, rows at even
// elements, all columns there) two columns of every other row, so that every
// access is contiguous along a row.  What is read is asked for eight rows
// ahead.
template <bool F32, int ACT, bool PAIRS>
__device__ __forceinline__ void finish_ragged(const LinearParams& p, uint32_t stg, int lane, int row0, int row_end, int col0) {
    constexpr bool kReadZ = (ACT & GEMM_ACT_GRADIENT) != 0;
    constexpr int W = PAIRS ? 2 : 1;          // columns of a lane, and rows of an access
    constexpr int N = 8 / W;                  // accesses in flight; twice as many: 5 to 10 % slower, by the size of the code
    static_assert(!(F32 && PAIRS), "fp32 columns are single");
    const int c = PAIRS ? (lane & 15) * 2 : lane, r0 = PAIRS ? lane >> 4 : 0;
    const int col = col0 + c;
    if (!PAIRS && col >= p.n) return;
    float bias[W];
#pragma unroll
    for (int t = 0; t < W; ++t) bias[t] = p.bias ? __ldg(p.bias + col + t) : 0.f;
    constexpr int ES = F32 ? 4 : 2;
    const int64_t row = row0 + r0;
    uint8_t* z_at = reinterpret_cast<uint8_t*>(p.Z) + (row * p.ldz + col) * 2;
    const uint8_t* r_at = static_cast<const uint8_t*>(p.R) + (row * p.ldr + col) * ES;
    uint8_t* d_at = static_cast<uint8_t*>(p.D) + (row * p.ldd + col) * ES;
    const int64_t z_step = 2 * W * p.ldz, r_step = ES * W * p.ldr, d_step = ES * W * p.ldd;
    const int rows = row_end - row0 - r0;
    // (row r0 + W i of the staging buffer: its 16-byte pieces are XORed with the row modulo 8, of which r0 is the
    // lowest bit or nothing)
    static_assert(W * N == 8, "j + i is i modulo 8 / W");
    uint32_t s_at = stg + r0 * 128;
    const uint32_t piece = (((c >> 2) ^ r0) << 4) + (c & 3) * 4;
#pragma unroll 1
    for (int j = 0; j < 32; j += 8, s_at += 8 * 128) {
        if (j >= rows) break;
        uint32_t z[N], r[N];
        if constexpr (kReadZ)
#pragma unroll
            for (int i = 0; i < N; ++i, z_at += z_step) z[i] = load_if<2 * W>(z_at, j + W * i < rows);
        if (p.R)
#pragma unroll
            for (int i = 0; i < N; ++i, r_at += r_step) r[i] = load_if<F32 ? 4 : 2 * W>(r_at, j + W * i < rows);
        float v[N * W];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t at = s_at + W * i * 128 + (piece ^ (W * i << 4));
            if constexpr (W == 2) {
                ld_shared_pair(at, v[2 * i], v[W * i + W - 1]);
            } else {
                v[i] = __uint_as_float(ld_shared_u32(at));
            }
#pragma unroll
            for (int t = 0; t < W; ++t) v[i * W + t] += bias[t];
        }
        if constexpr (!kReadZ)
            if (p.Z)
#pragma unroll
                for (int i = 0; i < N; ++i, z_at += z_step)
                    if (j + W * i < rows) store_some<W>(z_at, v + i * W);
        activate_each<ACT, N * W>(v, [&](int i) {
            return kReadZ ? __uint_as_float(i % W ? z[i / W] & 0xffff0000u : z[i / W] << 16) : 0.f;
        });
        if (p.R)
#pragma unroll
            for (int i = 0; i < N * W; ++i)
                v[i] += F32 ? __uint_as_float(r[i / W]) : __uint_as_float(i % W ? r[i / W] & 0xffff0000u : r[i / W] << 16);
#pragma unroll
        for (int i = 0; i < N; ++i, d_at += d_step)
            if (j + W * i < rows) {
                if constexpr (F32)
                    *reinterpret_cast<float*>(d_at) = v[i];
                else
                    store_some<W>(d_at, v + i * W);
            }
    }
}
// Either of them for the block at (row0, col0); rows at or past row_end are
// not its own.
template <int ACT>
__device__ __forceinline__ void finish(const LinearParams& p, uint32_t stg, int lane, int row0, int row_end, int col0) {
    const bool vec = p.vec && (p.n % 8 == 0 || col0 + 32 <= p.n);
    if (p.out_f32) {
        if (vec) finish_block<true, ACT>(p, stg, lane, row0, row_end, col0);
        else finish_ragged<true, ACT, false>(p, stg, lane, row0, row_end, col0);
    } else {
        if (vec) finish_block<false, ACT>(p, stg, lane, row0, row_end, col0);
        else if (p.pairs && col0 + 32 <= p.n) finish_ragged<false, ACT, true>(p, stg, lane, row0, row_end, col0);
        else finish_ragged<false, ACT, false>(p, stg, lane, row0, row_end, col0);
    }
}

// Host: calls f(integral constant of the launch's ACT).
template <typename F>
cudaError_t by_activation(const LinearLaunch& a, F f) {
#define GEMM_ACT_CASE(ACT) case ACT: return f(std::integral_constant<int, ACT>{});
    switch (a.act | (a.grad ? GEMM_ACT_GRADIENT : 0)) {
        GEMM_ACT_CASE(GEMM_ACT_RELU)
        GEMM_ACT_CASE(GEMM_ACT_GELU)
        GEMM_ACT_CASE(GEMM_ACT_GELU_TANH)
        GEMM_ACT_CASE(GEMM_ACT_SILU)
        GEMM_ACT_CASE(GEMM_ACT_RELU | GEMM_ACT_GRADIENT)
        GEMM_ACT_CASE(GEMM_ACT_GELU | GEMM_ACT_GRADIENT)
        GEMM_ACT_CASE(GEMM_ACT_GELU_TANH | GEMM_ACT_GRADIENT)
        GEMM_ACT_CASE(GEMM_ACT_SILU | GEMM_ACT_GRADIENT)
        default: return f(std::integral_constant<int, GEMM_ACT_NONE>{});   // (the gradient of none is none: Z is not given)
    }
#undef GEMM_ACT_CASE
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
