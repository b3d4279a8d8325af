// Host-side set-up shared by the library's entry points (defined in fa2_api.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

namespace fa2 {

// Checks the current device, binds its context to the calling thread, and
// gives its multiprocessor count and the device address of its status word.
int host_device_setup(int* num_sms, int** status);

// Records a CUDA error for fa2_last_cuda_error and returns FA2_ERR_CUDA.
int host_cuda_fail(cudaError_t e);

// Tensor map over [BH][N][d] 16-bit rows: boxes of 128 rows x 64 columns,
// 128-byte swizzled, zero fill past row N.
int host_map_16bit(CUtensorMap* m, const void* ptr, int BH, int N, int d, int dtype);

// 1 if the fault of this kind is armed, which disarms it and sets the wait
// bound that came with it; else 0.
int host_take_fault(int kind, unsigned long long* timeout_ns);

}  // namespace fa2
