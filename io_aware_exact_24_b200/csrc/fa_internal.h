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
// [B, H_kv, rows, d].  p.wait_limit is set here.
int launch_kv4_rows(const void* q, void* o, int B, int d, fa::kv4::RowsParams p, cudaStream_t stream);

// Records a failed CUDA call for fa_last_error on this thread; returns FA_ERR_CUDA.
int cuda_fail(const char* what, cudaError_t e);

// The current device, checked (and its kernels' attributes set) once: FA_OK with its
// number and SM count, or FA_ERR_NO_DEVICE / FA_ERR_UNSUPPORTED / FA_ERR_CUDA.
int ready_device(int* dev, int* num_sms);

// SM count of the current device; 148 (a B200) where none is visible.
int current_num_sms();

}  // namespace fa_internal
