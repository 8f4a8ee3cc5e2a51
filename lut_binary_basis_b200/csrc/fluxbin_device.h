// Device-side services of the library shared by its translation units
// (defined in fluxbin_api.cu).
#pragma once

#include <cuda_runtime.h>

namespace fluxbin {

// Records a failed CUDA call for fluxbin_last_error(), clears the CUDA error
// state and returns FLUXBIN_ERR_CUDA.
int report_cuda_failure(cudaError_t e);

// Address, on device `dev` (the current one), of the error word that
// fluxbin_device_status reads.
int device_error_word(int dev, unsigned int** out);

}  // namespace fluxbin
