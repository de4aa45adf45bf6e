// host.h -- what the library's translation units share on the host: the
// thread's last error and the current device's properties (gemm_epi.cu).
#pragma once

#include <cuda_runtime.h>

#include "gemm_epi.h"

namespace ge_host {

// Records the one-line reason gemm_epi_last_error() returns; returns `s`.
gemm_epi_status fail(gemm_epi_status s, const char* fmt, ...);
gemm_epi_status cuda_fail(cudaError_t e, const char* what);
void clear_error();

// The current device (0..127) and its SM count; GEMM_EPI_ERR_ARCH unless it
// is sm_103.
gemm_epi_status device_sms(int* dev, int* sms);

}  // namespace ge_host
