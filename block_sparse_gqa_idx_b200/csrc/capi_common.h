// capi_common.h -- what the C-ABI files (msa_capi.cu, chunk_capi.cu) share:
// pointer and status helpers and the CUDA error of the calling thread.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/msa.h"
#include "msa_internal.h"

constexpr size_t kStatusBytes = 256;  // status word + padding (keeps the rest 256-B aligned)

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline msa::DevStatus* status_of(void* ws) { return reinterpret_cast<msa::DevStatus*>(ws); }

// MSA_OK, or MSA_ERR_CUDA with the error kept for msa_last_error (msa_capi.cu).
msa_status msa_from_cuda(cudaError_t e);
