// Skinny int8 GEMM on CUDA cores (m <= 128, in launches of at most 64 rows;
// used when the tensor-core skinny kernel does not apply): C = A x B where B (stored K-major as Bt,
// n x k) is far larger than A, so the kernel's job is to stream Bt from HBM
// once.  The patent CN114238853A (claim 4 S3) notes that such shapes are too
// small to fill the chip with output tiles; here they get their own kernel.
//
// Mapping: a CTA owns 32 output columns j (one per lane) and all m rows of
// C.  Its 8 warps split K into interleaved 16-byte vectors, so the 8 warps of
// a CTA read consecutive 16-byte pieces of the same 128-byte lines of Bt.
// Each lane keeps m int32 partial sums (one per row of A), formed with dp4a
// on its own Bt row and the A vector that all lanes of the warp share (one
// broadcast load).  The warps' partial sums are added in shared memory
// (int32, exact) and written to C with coalesced stores.  This is the
// warp-level partial-sum scheme of "CUDA编程实践" §2 (reduce), with the
// final cross-warp sum in shared memory instead of shuffles.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace gemm {

namespace {

constexpr int kSkWarps = 8;
constexpr int kSkCols = 32;
constexpr int kSkUnroll = 8;

__device__ __forceinline__ uint4 ld_stream16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <int MT>
__global__ void __launch_bounds__(kSkWarps * 32) skinny_dp4a_kernel(const int8_t* __restrict__ A,
                                                                    const int8_t* __restrict__ Bt,
                                                                    int32_t* __restrict__ C, int m, int64_t n,
                                                                    int64_t k) {
    __shared__ int32_t red[MT][kSkCols];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int t = threadIdx.x; t < MT * kSkCols; t += blockDim.x) (&red[0][0])[t] = 0;
    __syncthreads();

    const int64_t j = static_cast<int64_t>(blockIdx.x) * kSkCols + lane;
    const bool col_ok = j < n;
    const int8_t* brow = Bt + (col_ok ? j : 0) * k;
    const int64_t nvec = k / 16;

    int32_t acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = 0;

    for (int64_t v0 = warp; v0 < nvec; v0 += kSkWarps * kSkUnroll) {
        uint4 b[kSkUnroll];
#pragma unroll
        for (int u = 0; u < kSkUnroll; ++u) {
            const int64_t v = v0 + static_cast<int64_t>(u) * kSkWarps;
            b[u] = (v < nvec && col_ok) ? ld_stream16(brow + v * 16) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kSkUnroll; ++u) {
            const int64_t v = v0 + static_cast<int64_t>(u) * kSkWarps;
            if (v < nvec) {
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if (i < m) {
                        const uint4 a = __ldg(reinterpret_cast<const uint4*>(A + static_cast<int64_t>(i) * k + v * 16));
                        int s = acc[i];
                        s = __dp4a(static_cast<int>(a.x), static_cast<int>(b[u].x), s);
                        s = __dp4a(static_cast<int>(a.y), static_cast<int>(b[u].y), s);
                        s = __dp4a(static_cast<int>(a.z), static_cast<int>(b[u].z), s);
                        s = __dp4a(static_cast<int>(a.w), static_cast<int>(b[u].w), s);
                        acc[i] = s;
                    }
                }
            }
        }
    }

#pragma unroll
    for (int i = 0; i < MT; ++i)
        if (i < m) atomicAdd(&red[i][lane], acc[i]);
    __syncthreads();
    for (int i = warp; i < m; i += kSkWarps)
        if (col_ok) C[static_cast<int64_t>(i) * n + j] = red[i][lane];
}

// Any k or alignment, where a row starts at any byte: per step of kRowsK
// elements the CTA copies its columns' rows of Bt and the rows of A into shared
// memory, from the aligned 16-byte words around each piece, shifted to the
// row's own start (zeros behind its end); then its warps take the step's
// 16-byte vectors in turn, with one dp4a per row of A, column and four
// elements, and add their partial sums up as above.  Each byte is loaded once
// per CTA: 55 x 1940 x 620 takes 50 us on GB300 and 64 x 4095 x 256 101, where a
// byte of A and one of Bt loaded per multiply-add took 1121 and 2969.  A step
// takes 1.8 us with one row, the latency of its loads, and 6.3 with 64, where
// the multiply-adds are the larger part.
constexpr int kRowsK = 256;               // elements of K per step
constexpr int kRowsPitch = kRowsK + 16;   // odd in 16-byte units: 32 lanes read 32 rows without bank conflicts
constexpr int kRowsBatch = 3;             // pieces whose loads a thread has on their way at once

// Bytes [at, at + 16) of a matrix [begin, end) in two steps: the words that
// hold them, if all of those lie inside and all 16 bytes are the row's, ...
__device__ __forceinline__ bool words_inside(uintptr_t at, int64_t left, uintptr_t begin, uintptr_t end) {
    const uintptr_t w = at & ~static_cast<uintptr_t>(15);
    return left >= 16 && w >= begin && w + 32 <= end;
}
// ... and the bytes themselves, shifted out of the words, or loaded one by one:
// `left` of them are the row's, the others zero.
__device__ __forceinline__ uint4 shifted_bytes(const uint4& lo, const uint4& hi, int sh) {
    uint32_t t[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i + 1 < 8; ++i) t[i] = sh & 4 ? t[i + 1] : t[i];
#pragma unroll
    for (int i = 0; i + 2 < 8; ++i) t[i] = sh & 8 ? t[i + 2] : t[i];
    const uint32_t bits = 8u * (sh & 3);
    return make_uint4(__funnelshift_r(t[0], t[1], bits), __funnelshift_r(t[1], t[2], bits),
                      __funnelshift_r(t[2], t[3], bits), __funnelshift_r(t[3], t[4], bits));
}
__device__ __forceinline__ uint4 single_bytes(uintptr_t at, int64_t left) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(at);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (e < left) w[e >> 2] |= static_cast<uint32_t>(__ldg(p + e)) << (8 * (e & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int MT>
__global__ void __launch_bounds__(kSkWarps * 32) skinny_rows_kernel(const int8_t* __restrict__ A,
                                                                    const int8_t* __restrict__ Bt,
                                                                    int32_t* __restrict__ C, int m, int64_t n,
                                                                    int64_t k) {
    __shared__ __align__(16) uint8_t rows[(MT + kSkCols) * kRowsPitch];   // of A, then of Bt
    constexpr int kPieces = kRowsK / 16;   // of a row and step
    static_assert(MT * kRowsPitch >= MT * kSkCols * 4, "the sums fit over the rows");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kSkCols, j = j0 + lane;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(A), a1 = a0 + static_cast<uintptr_t>(m * k);
    const uintptr_t b0 = reinterpret_cast<uintptr_t>(Bt), b1 = b0 + static_cast<uintptr_t>(n * k);
    const int cols = static_cast<int>(n - j0 < kSkCols ? n - j0 : kSkCols);
    const int items = (m + cols) * kPieces;

    int32_t acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = 0;

    for (int64_t k0 = 0; k0 < k; k0 += kRowsK) {
        for (int i0 = threadIdx.x; i0 < items; i0 += kRowsBatch * kSkWarps * 32) {
            uint4 lo[kRowsBatch], hi[kRowsBatch];
            uintptr_t at[kRowsBatch];
            int64_t left[kRowsBatch];
            bool inside[kRowsBatch];
#pragma unroll
            for (int u = 0; u < kRowsBatch; ++u) {
                const int i = i0 + u * kSkWarps * 32, r = i / kPieces;
                const bool of_a = r < m;
                const int64_t c = k0 + (i % kPieces) * 16;
                left[u] = i < items ? k - c : 0;
                at[u] = (of_a ? a0 + static_cast<uintptr_t>(r * k) : b0 + static_cast<uintptr_t>((j0 + (r - m)) * k)) +
                        static_cast<uintptr_t>(c);
                inside[u] = words_inside(at[u], left[u], of_a ? a0 : b0, of_a ? a1 : b1);
                const uint4* w = reinterpret_cast<const uint4*>(at[u] & ~static_cast<uintptr_t>(15));
                lo[u] = hi[u] = make_uint4(0u, 0u, 0u, 0u);
                if (inside[u]) {
                    lo[u] = __ldg(w);
                    hi[u] = __ldg(w + 1);
                }
            }
#pragma unroll
            for (int u = 0; u < kRowsBatch; ++u) {
                const int i = i0 + u * kSkWarps * 32, r = i / kPieces;
                if (i >= items) break;
                // rows of Bt lie behind MT rows of A, whatever m
                uint4* to = reinterpret_cast<uint4*>(rows + (r < m ? r : MT + r - m) * kRowsPitch + (i % kPieces) * 16);
                *to = inside[u] ? shifted_bytes(lo[u], hi[u], static_cast<int>(at[u] & 15)) : single_bytes(at[u], left[u]);
            }
        }
        __syncthreads();
        const int vecs = static_cast<int>(k - k0 < kRowsK ? (k - k0 + 15) / 16 : kPieces);
        if (lane < cols)
            for (int v = warp; v < vecs; v += kSkWarps) {
                const uint4 b = *reinterpret_cast<const uint4*>(rows + (MT + lane) * kRowsPitch + v * 16);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if (i < m) {
                        const uint4 a = *reinterpret_cast<const uint4*>(rows + i * kRowsPitch + v * 16);
                        int s = acc[i];
                        s = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), s);
                        s = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), s);
                        s = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), s);
                        s = __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), s);
                        acc[i] = s;
                    }
                }
            }
        __syncthreads();   // the rows are overwritten by the next step, or by the sums
    }

    int32_t* red = reinterpret_cast<int32_t*>(rows);   // [MT][kSkCols]
    for (int t = threadIdx.x; t < MT * kSkCols; t += blockDim.x) red[t] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i)
        if (i < m) atomicAdd(&red[i * kSkCols + lane], acc[i]);
    __syncthreads();
    for (int i = warp; i < m; i += kSkWarps)
        if (lane < cols) C[static_cast<int64_t>(i) * n + j] = red[i * kSkCols + lane];
}

template <int MT>
void launch_rows(unsigned grid, cudaStream_t stream, bool vec, const int8_t* A, const int8_t* Bt, int32_t* C, int m,
                 int64_t n, int64_t k) {
    if (vec)
        skinny_dp4a_kernel<MT><<<grid, kSkWarps * 32, 0, stream>>>(A, Bt, C, m, n, k);
    else
        skinny_rows_kernel<MT><<<grid, kSkWarps * 32, 0, stream>>>(A, Bt, C, m, n, k);
}

}  // namespace

cudaError_t launch_skinny_i8(const int8_t* A, const int8_t* Bt, int32_t* C, int64_t m, int64_t n, int64_t k,
                             int num_sms, cudaStream_t stream) {
    (void)num_sms;
    if (m < 1 || m > 128) return cudaErrorInvalidValue;
    if (m > 64) {
        // rows 0..63, then the rest
        const cudaError_t e = launch_skinny_i8(A, Bt, C, 64, n, k, num_sms, stream);
        if (e != cudaSuccess) return e;
        return launch_skinny_i8(A + 64 * k, Bt, C + 64 * n, m - 64, n, k, num_sms, stream);
    }
    const unsigned grid = static_cast<unsigned>((n + kSkCols - 1) / kSkCols);
    const bool vec = (k % 16) == 0 &&
                     ((reinterpret_cast<uintptr_t>(A) | reinterpret_cast<uintptr_t>(Bt)) & 15u) == 0;
    const int mi = static_cast<int>(m);
    if (m <= 8)
        launch_rows<8>(grid, stream, vec, A, Bt, C, mi, n, k);
    else if (m <= 16)
        launch_rows<16>(grid, stream, vec, A, Bt, C, mi, n, k);
    else if (m <= 32)
        launch_rows<32>(grid, stream, vec, A, Bt, C, mi, n, k);
    else
        launch_rows<64>(grid, stream, vec, A, Bt, C, mi, n, k);
    return cudaGetLastError();
}

}  // namespace gemm
