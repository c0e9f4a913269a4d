// FP8 product with block scales on the CUDA cores: one thread per element of
// D, straight from the formula.
#include <cuda_fp8.h>

#include "f8.cuh"
#include "ptx.cuh"

namespace gemm {

namespace {

__device__ __forceinline__ float f8_value(uint8_t v, int type) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(v, type == GEMM_F8_E4M3 ? __NV_E4M3 : __NV_E5M2);
    return __half2float(__half(h));
}

__global__ void __launch_bounds__(256) f8_simple_kernel(const F8Launch p) {
    const int64_t j = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x & 15);
    if (j >= p.n) return;
    const int64_t rows = p.group_mode == GEMM_GROUP_K ? p.m * p.groups : p.m;
    const int64_t kb = (p.k + kF8Block - 1) / kF8Block, nb = (p.n + kF8Block - 1) / kF8Block;
    for (int64_t i = static_cast<int64_t>(blockIdx.y) * 16 + (threadIdx.x >> 4); i < rows;
         i += static_cast<int64_t>(gridDim.y) * 16) {
        int64_t ia = i, jb = j, b0 = 0, b1 = kb, bs = j / kF8Block * kb;
        if (p.group_mode == GEMM_GROUP_ROWS) {
            int g = 0, lo = 0, hi = 0;
            for (; g < p.groups; ++g) {
                group_rows(p.offsets, g, static_cast<int>(p.m), lo, hi);
                if (i >= lo && i < hi) break;
            }
            if (g == p.groups) continue;
            jb += g * p.n;
            bs += g * nb * kb;
        } else if (p.group_mode == GEMM_GROUP_K) {
            const int g = static_cast<int>(i / p.m);
            ia = i - g * p.m;
            b1 = 0;
            for (int q = 0; q <= g; ++q) {
                int lo, hi;
                group_rows(p.offsets, q, INT32_MAX, lo, hi);
                b0 = b1;
                b1 += (hi - lo + kF8Block - 1) / kF8Block;
            }
            b0 = min(b0, kb);
            b1 = min(b1, kb);
        }
        float acc = 0.f;
        for (int64_t b = b0; b < b1; ++b) {
            float t = 0.f;
            for (int64_t x = b * kF8Block; x < min((b + 1) * kF8Block, p.k); ++x)
                t += f8_value(p.A[ia * p.lda + x], p.a_type) * f8_value(p.Bt[jb * p.ldb + x], p.b_type);
            const float sb = p.b_scale_mode == GEMM_SCALE_BLOCKS ? p.b_scale[bs + b] : p.b_scale[b * p.rows_b + jb];
            acc += p.a_scale[b * p.rows_a + ia] * sb * t;
        }
        if (p.out_f32)
            static_cast<float*>(p.D)[i * p.ldd + j] = acc;
        else
            static_cast<__nv_bfloat16*>(p.D)[i * p.ldd + j] = __float2bfloat16_rn(acc);
    }
}

}  // namespace

cudaError_t launch_f8_simple(const F8Launch& a, cudaStream_t stream) {
    const int64_t rows = a.group_mode == GEMM_GROUP_K ? a.m * a.groups : a.m;
    const int64_t gy = (rows + 15) / 16;
    f8_simple_kernel<<<dim3(static_cast<unsigned>((a.n + 15) / 16), static_cast<unsigned>(gy < 65535 ? gy : 65535)), 256, 0,
                       stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gemm
