// cuda_call.h -- runtime calls of the block operators' entry points.
#pragma once
#include <cuda_runtime_api.h>

namespace mlpc {

// An error is reported by the call that had it, and not left with the runtime for a later one.
inline bool succeeded(cudaError_t e)
{
    if (e != cudaSuccess)
        cudaGetLastError();
    return e == cudaSuccess;
}

}  // namespace mlpc
