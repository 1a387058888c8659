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

// A handle's device, for the length of a call: the caller's current device is the same afterwards.
class OnDevice {
public:
    explicit OnDevice(int device) : ok_(succeeded(cudaGetDevice(&before_)) && succeeded(cudaSetDevice(device))), changed_(ok_ && device != before_) {}
    ~OnDevice()
    {
        if (changed_)
            succeeded(cudaSetDevice(before_));
    }
    OnDevice(const OnDevice &) = delete;
    OnDevice &operator=(const OnDevice &) = delete;
    explicit operator bool() const { return ok_; }

private:
    int before_ = 0;
    bool ok_, changed_;
};

}  // namespace mlpc
