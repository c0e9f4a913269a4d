// Per-device state and tracing of api.cpp, for the entry points in other
// translation units.
#pragma once

#include <cuda_runtime.h>

#include "../../include/dense_int8_matrix.h"

namespace gemm {

struct DeviceContext {
    int num_sms = 0;
    int* err_word = nullptr;        // device error word
    cudaMemPool_t pool = nullptr;   // the library's stream-ordered scratch
    int pairs = 0;                  // co-resident CTA pairs of a one-CTA-per-SM kernel (0: unknown)
};

// The current device's state; GEMM_ERR_UNSUPPORTED_DEVICE unless it is sm_103.
gemm_status device_context(DeviceContext* out);
// Its SM count, whatever the device.
gemm_status device_sms(int* num_sms);

// Tracing of a run call: whether the call is sampled (once per call), a
// launch made, and the events around a timed unit (nullptr: not recorded).
bool trace_begin_call();
void trace_launch(int kind);
void* trace_unit_begin(int kind, cudaStream_t stream, bool sampled);
void trace_unit_end(void* unit, cudaStream_t stream);

}  // namespace gemm
