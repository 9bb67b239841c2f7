// Branches of the graph that a stream captures, made on that stream by its dependencies.  A stream
// of the library's that took part in a capture would be unusable to every other call until the
// capture ends.
#pragma once

#include <cuda_runtime_api.h>

#include <algorithm>
#include <memory>
#include <new>

namespace cpring {

// What a capturing stream's next launch would depend on.
class CaptureTail {
 public:
  cudaError_t read(cudaStream_t stream) {
    cudaStreamCaptureStatus status;
    const cudaGraphNode_t* n = nullptr;
    const cudaGraphEdgeData* e = nullptr;
    size_t count = 0;
    const cudaError_t err =
        cudaStreamGetCaptureInfo(stream, &status, nullptr, nullptr, &n, &e, &count);
    if (err != cudaSuccess) return err;
    nodes_.reset(new (std::nothrow) cudaGraphNode_t[count + 1]);
    edges_.reset(new (std::nothrow) cudaGraphEdgeData[count + 1]());
    count_ = 0;
    if (!nodes_ || !edges_) return cudaErrorMemoryAllocation;
    std::copy(n, n + count, nodes_.get());
    if (e) std::copy(e, e + count, edges_.get());
    count_ = count;
    return cudaSuccess;
  }
  // Makes the stream's next launch depend on this instead (cudaStreamSetCaptureDependencies) or as
  // well (cudaStreamAddCaptureDependencies).
  cudaError_t put(cudaStream_t stream, unsigned flags) const {
    return cudaStreamUpdateCaptureDependencies(stream, nodes_.get(), edges_.get(), count_, flags);
  }

 private:
  std::unique_ptr<cudaGraphNode_t[]> nodes_;
  std::unique_ptr<cudaGraphEdgeData[]> edges_;
  size_t count_ = 0;
};

}  // namespace cpring
