// What the library's translation units share besides the C ABI.
#pragma once

#include <cuda_runtime.h>

#include "../../include/svdq.h"

namespace svdq {

// Record a failed CUDA call for svdq_last_error_string; returns SVDQ_ERR_CUDA.
svdq_status cuda_failure(cudaError_t e, const char* where);

// Read and clear the status word of the paged-cache kernels (each translation
// unit of kernels has its own word; svdq_get_status reads this one when the other is clear).
cudaError_t paged_status_take(unsigned int* v);

}  // namespace svdq
