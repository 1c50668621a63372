// Argument checks shared by the C-ABI files.
#pragma once

#include "common.cuh"

namespace csa {

inline bool aligned16(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline bool act_ok(int f) { return f == CSA_F32 || f == CSA_BF16; }
inline bool kv_ok(int f) { return f == CSA_F32 || f == CSA_BF16 || f == CSA_FP8_S64; }

inline int cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return CSA_OK;
    if (e == cudaErrorInvalidValue) return CSA_ERR_UNSUPPORTED;
    return CSA_ERR_CUDA;
}

}  // namespace csa
