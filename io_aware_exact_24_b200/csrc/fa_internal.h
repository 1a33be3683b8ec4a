// fa_internal.h -- host helpers of fa_api.cu that the library's other sources share.
#pragma once

#include <cuda_runtime.h>

namespace fa {
namespace kv4 {
struct RowsParams;
}
}  // namespace fa

namespace fa_internal {

// Launches the 4-bit cache attention for many rows (fa_kv4_rows.cuh): q and o are bf16
// [B, H_kv, rows, d].  A p.wait_limit of 0 is the default.
int launch_kv4_rows(const void* q, void* o, int B, int d, fa::kv4::RowsParams p, cudaStream_t stream);

// Records a failed CUDA call for fa_last_error on this thread; returns FA_ERR_CUDA.
int cuda_fail(const char* what, cudaError_t e);

// The current device, checked (and its kernels' attributes set) once: FA_OK with its
// number and SM count, or FA_ERR_NO_DEVICE / FA_ERR_UNSUPPORTED / FA_ERR_CUDA.
int ready_device(int* dev, int* num_sms);

// SM count of the current device; 148 (a B200) where none is visible.
int current_num_sms();

// Launches a kernel that may be set up while the one before it on the stream still runs
// (programmatic dependent launch): it calls fa::kv4::after_previous() before it touches memory.
template <typename... P, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) cudaGetLastError();   // reported here, not by a later call
    return e;
}

}  // namespace fa_internal
