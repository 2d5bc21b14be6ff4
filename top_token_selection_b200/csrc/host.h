// host.h -- host-side helpers of api.cu that the other C entry points share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/pivot.h"

namespace pivot {

// PIVOT_OK, or PIVOT_ERR_CUDA with the error's text for pivot_last_error_detail.
pivot_status_t status_of(cudaError_t e);

// SMs of the current device.
int sm_count();

// cuTensorMapEncodeTiled of the loaded driver (NULL if there is none).
using TensorMapEncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                       const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                       const cuuint32_t*, CUtensorMapInterleave,
                                       CUtensorMapSwizzle, CUtensorMapL2promotion,
                                       CUtensorMapFloatOOBfill);
TensorMapEncodeFn tensor_map_encode();

}  // namespace pivot
