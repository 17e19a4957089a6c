// The number of the capture that a stream is part of.
#include <cuda_runtime.h>

#include <cstdint>

// For the binding: the number of the capture that the stream is part of, 0 if it is not being captured.
extern "C" uint64_t ss__capture_id(void* stream) {
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &status, &id, nullptr, nullptr, nullptr, nullptr) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return status == cudaStreamCaptureStatusActive ? id : 0;
}
