// host_state.h - the host-side state of gsr_api.cu (devices, per-stream error words, the tensor-map
// encoder, settings) for the other C-ABI translation units.  Not installed; not part of the ABI.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "gsr.h"

namespace gsr {
namespace host {

gsr_status fail(cudaError_t e);          // records the code for gsr_last_cuda_error
gsr_status fail_encode(CUresult r);
gsr_status current_device(int* dev, int* num_sms);
gsr_status error_word(int dev, cudaStream_t stream, int** err);
// The stream's own workspace of at least `bytes` (grown after a wait for the stream).
gsr_status stream_scratch(int dev, cudaStream_t stream, size_t bytes, void** scratch);
gsr_status tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* encode);
uint64_t wait_timeout_ns();
uint32_t test_flags();

}  // namespace host
}  // namespace gsr
