// Argument checks and the traced launch that the entry points share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <initializer_list>

#include "context.h"

namespace gemm {

constexpr int64_t kMaxDim = int64_t(1) << 30;   // coordinates of tiles past the edge stay in 32 bits

inline bool al(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool dim_ok(int64_t v) { return v >= 1 && v <= kMaxDim; }
// Pitches stay far below where rows * pitch * 4 bytes would pass 63 bits.
inline bool pitch_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= (int64_t(1) << 31); }
inline int elem_bytes(int type) { return type == GEMM_DTYPE_BF16 ? 2 : 4; }
inline bool real_type(int type) { return type == GEMM_DTYPE_BF16 || type == GEMM_DTYPE_F32; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// No output (nullptr: none) is one of the operands, or another output.
inline bool apart(std::initializer_list<const void*> outputs, std::initializer_list<const void*> operands) {
    for (const void* const* o = outputs.begin(); o != outputs.end(); ++o) {
        if (!*o) continue;
        for (const void* p : operands)
            if (*o == p) return false;
        for (const void* const* other = outputs.begin(); other != o; ++other)
            if (*o == *other) return false;
    }
    return true;
}

// One timed unit of kind GEMM_KERNEL_STAGE.
template <typename Launch>
gemm_status staged(Launch launch, cudaStream_t stream) {
    const bool sampled = trace_begin_call();
    void* unit = trace_unit_begin(GEMM_KERNEL_STAGE, stream, sampled);
    const cudaError_t e = launch();
    trace_unit_end(unit, stream);
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    trace_launch(GEMM_KERNEL_STAGE);
    return GEMM_OK;
}

}  // namespace gemm
