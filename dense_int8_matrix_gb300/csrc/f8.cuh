// Device helpers of the 8-bit operators: vectors of eight input values,
// rounding to e4m3 / e5m2, group lookup, warp and CTA reductions.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <cstring>

#include "f8.h"

namespace gemm {

// Reciprocals of the 8-bit types' largest values, rounded to fp32.
constexpr float kE4M3Step = 1.f / 448.f;
constexpr float kE5M2Step = 1.f / 57344.f;
constexpr float kI8Step = 1.f / 127.f;
constexpr float kScaleMin = 1.17549435e-38f;   // 2^-126: scale of a block of zeros; its reciprocal is finite

// The scale of a block of largest magnitude amax, step the reciprocal of the
// type's largest value.
__device__ __forceinline__ float block_scale(float amax, float step) { return fmaxf(__fmul_rn(amax, step), kScaleMin); }

// Two fp32 values to two FP8 values (a in the low byte), round to nearest
// even, clamped to the largest finite value, NaN stays NaN.
template <int F8>
__device__ __forceinline__ uint32_t f8x2(float a, float b) {
    uint16_t r;
    if constexpr (F8 == GEMM_F8_E4M3)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
template <int F8>
__device__ __forceinline__ uint32_t f8x4(float a, float b, float c, float d) {
    return f8x2<F8>(a, b) | (f8x2<F8>(c, d) << 16);
}

// Eight consecutive elements of a row, as stored (16 or 32 bytes).
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {   // rounds to nearest even
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void words(const uint32_t (&w)[4]) { u = make_uint4(w[0], w[1], w[2], w[3]); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ void words(const uint32_t (&w)[8]) {
        a = make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
        b = make_float4(__uint_as_float(w[4]), __uint_as_float(w[5]), __uint_as_float(w[6]), __uint_as_float(w[7]));
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float* p) { *p = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* p) { *p = __float2bfloat16_rn(x); }

// N words from byte `sh` (a multiple of 2 below 16) of the N + 4 words `in`.
template <int N>
__device__ __forceinline__ void shift_words(const uint32_t (&in)[N + 4], int sh, uint32_t (&out)[N]) {
    uint32_t t[N + 4];
#pragma unroll
    for (int i = 0; i < N + 4; ++i) t[i] = in[i];
#pragma unroll
    for (int i = 0; i + 1 < N + 4; ++i) t[i] = sh & 4 ? t[i + 1] : t[i];
#pragma unroll
    for (int i = 0; i + 2 < N + 4; ++i) t[i] = sh & 8 ? t[i + 2] : t[i];
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = __byte_perm(t[i], t[i + 1], sh & 2 ? 0x5432u : 0x3210u);
}

// Elements [c, c + 8) of a row of d; those at or past d are zero.  VEC: the
// row is aligned for whole-vector access (a template parameter, as the code
// for unaligned rows costs aligned ones registers: 8192 x 8192 forward norm 79
// us alone, 117 us with both in one kernel).  Otherwise the aligned 16-byte words
// around the elements are read and shifted together, where all of them lie
// inside the row; its ends are read element by element.
template <bool VEC, typename T>
__device__ __forceinline__ Vec8<T> load8(const T* row, int64_t c, int64_t d) {
    Vec8<T> v;
    if (VEC && c + 8 <= d) {
        v.load(row + c);
    } else if (!VEC && c >= 8 && c + 16 <= d) {
        constexpr int N = sizeof(Vec8<T>) / 4;
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
        const uint4* p = reinterpret_cast<const uint4*>(at & ~static_cast<uintptr_t>(15));
        uint32_t in[N + 4], out[N];
#pragma unroll
        for (int i = 0; i < N / 4 + 1; ++i) {
            const uint4 x = p[i];
            in[4 * i] = x.x; in[4 * i + 1] = x.y; in[4 * i + 2] = x.z; in[4 * i + 3] = x.w;
        }
        shift_words<N>(in, static_cast<int>(at & 15), out);
        v.words(out);
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < d ? to_f32(row[c + i]) : 0.f;
        v.set(f);
    }
    return v;
}

// The same, stored.  Called by whole warps whose lanes hold neighbouring
// vectors.  An unaligned bfloat16 row is written in aligned 16-byte words, each
// made of the end of the lane's left neighbour and the start of its own
// vector; the pieces that have no such word (at the warp's and the row's ends)
// go element by element.
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* row, int64_t c, int64_t d, const Vec8<T>& v) {
    if constexpr (VEC) {
        if (c + 8 <= d) {
            v.store(row + c);
            return;
        }
    } else if constexpr (sizeof(T) == 2) {
        const int lane = threadIdx.x & 31;
        const uintptr_t at = reinterpret_cast<uintptr_t>(row) + c * 2;
        const int sh = static_cast<int>(at & 15);   // the same in every lane
        uint32_t in[8], out[4];
        in[4] = v.u.x; in[5] = v.u.y; in[6] = v.u.z; in[7] = v.u.w;
#pragma unroll
        for (int i = 0; i < 4; ++i) in[i] = __shfl_up_sync(0xffffffffu, in[4 + i], 1);
        const bool whole = c + 8 <= d;
        if (sh == 0) {
            if (whole) {
                v.store(row + c);
                return;
            }
        } else if (whole) {
            const bool word = lane > 0;   // its left neighbour holds the columns before c
            if (word) {
                shift_words<4>(in, 16 - sh, out);
                *reinterpret_cast<uint4*>(at - sh) = make_uint4(out[0], out[1], out[2], out[3]);
            }
            const int first = word ? 8 - sh / 2 : 0;                         // elements not in that word ...
            const int last = lane == 31 || c + 16 > d ? 8 : 8 - sh / 2;      // ... nor in the right neighbour's
            float f[8];
            v.get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= first && i < last) from_f32(f[i], row + c + i);
            return;
        }
    }
    float f[8];
    v.get(f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < d) from_f32(f[i], row + c + i);
}
// Eight bytes (two words) to elements [c, c + 8) of a byte row of d.
__device__ __forceinline__ void store8_bytes(uint8_t* row, int64_t c, int64_t d, bool vec, uint32_t lo, uint32_t hi) {
    if (vec && c + 8 <= d) {
        *reinterpret_cast<uint2*>(row + c) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < d) row[c + i] = static_cast<uint8_t>((i < 4 ? lo >> (8 * i) : hi >> (8 * i - 32)) & 0xffu);
    }
}
__device__ __forceinline__ void load8_f32(const float* w, int64_t c, int64_t d, bool vec, float (&f)[8]) {
    if (vec && c + 8 <= d) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(w + c));
        const float4 b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < d ? __ldg(w + c + i) : 0.f;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// The larger of two values, NaN if either is (fmaxf drops a NaN).
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float warp_max_or_nan(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_or_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// Largest of the 16 lanes of this half warp (one block of 128 columns).
__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Bulk copy of `bytes` (a multiple of 16; both addresses 16-byte aligned) from
// global to shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// Launch with programmatic stream serialization: the kernel may start while
// the one before it ends, and calls pdl_wait() before it touches memory.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Row range of group g, clamped to [0, rows].
__device__ __forceinline__ void group_rows(const int32_t* offsets, int g, int rows, int& lo, int& hi) {
    lo = min(max(__ldg(offsets + g), 0), rows);
    hi = min(max(__ldg(offsets + g + 1), lo), rows);
}

}  // namespace gemm
