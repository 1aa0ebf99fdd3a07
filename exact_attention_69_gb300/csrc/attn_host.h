// attn_host.h -- what the translation units of the C ABI share: the calling
// thread's error message and stream, the driver's tensor-map encoder and the
// device check. Defined in attn_host.cu.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace attn {
namespace host {

constexpr uint64_t kTimeoutNs = 2000000000ull;  // bound on device-side waits when the caller gives none

// Set the thread's message; returns the code.
int fail_with(int code, const char* fmt, ...);
int cuda_error(cudaError_t e, const char* what);
void clear_error();
cudaStream_t stream_of(void* given);  // the given stream or the thread's
int tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn);
// The current device, checked to be an sm_103 GPU, and its SM count. Allocates nothing.
int this_device(int* dev, int* sms);
void paged_used(int dev);  // from now on attn_get_device_status reads the paged kernels' word there
void long_used(int dev);   // the same for the long-cache kernels

}  // namespace host
}  // namespace attn
