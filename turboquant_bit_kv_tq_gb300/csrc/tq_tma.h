// The CUDA driver's tensor-map encoder, shared by the calls that use bulk tensor copies.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "tq_internal.h"

namespace tq {

// the encoder, or nullptr with the reason in `why`
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder(char* why, size_t why_len);

// the encoder wants a current context: binds the device's primary one to a
// host thread whose first call this is
tq_status bind_device_context();

}  // namespace tq
