// Two launches that read nothing of each other's, side by side behind a stream's work: the second
// on a stream of the library's (one per device, made on first use and kept for the process's
// life), so that its blocks take the multiprocessors that the first's last blocks leave idle.
//
// A stream that captures a graph gets both as branches of the graph, by its dependencies: drawing
// the library's stream into the capture would make it unusable to every other call until the
// capture ends.
#include <cuda_runtime_api.h>

#include <mutex>

#include "capture.h"
#include "internal.h"

namespace cpring {
namespace {

struct SideStream {
  std::mutex mu;
  cudaStream_t s = nullptr;
};
constexpr int kMaxDevices = 64;
SideStream g_side[kMaxDevices];

cudaStream_t side_stream() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  SideStream& b = g_side[dev];
  std::lock_guard<std::mutex> lock(b.mu);
  if (!b.s && cudaStreamCreateWithFlags(&b.s, cudaStreamNonBlocking) != cudaSuccess) b.s = nullptr;
  return b.s;
}

}  // namespace

cudaError_t launch_beside(cudaStream_t stream, LaunchFn first, void* what1, LaunchFn second,
                          void* what2) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(stream, &status);
  if (e != cudaSuccess) return e;
  if (status != cudaStreamCaptureStatusNone) {
    CaptureTail before, after;
    if ((e = before.read(stream)) != cudaSuccess) return e;
    if ((e = first(what1, stream)) != cudaSuccess) return e;
    if ((e = after.read(stream)) != cudaSuccess) return e;
    if ((e = before.put(stream, cudaStreamSetCaptureDependencies)) != cudaSuccess) return e;
    if ((e = second(what2, stream)) != cudaSuccess) return e;
    return after.put(stream, cudaStreamAddCaptureDependencies);
  }
  const cudaStream_t side = side_stream();
  if (!side) {
    e = first(what1, stream);
    return e == cudaSuccess ? second(what2, stream) : e;
  }
  cudaEvent_t ready = nullptr, done = nullptr;
  if (cudaEventCreateWithFlags(&ready, cudaEventDisableTiming) != cudaSuccess)
    return cudaErrorUnknown;
  if (cudaEventCreateWithFlags(&done, cudaEventDisableTiming) != cudaSuccess) {
    cudaEventDestroy(ready);
    return cudaErrorUnknown;
  }
  e = cudaEventRecord(ready, stream);
  if (e == cudaSuccess) e = first(what1, stream);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(side, ready, 0);
  if (e == cudaSuccess) e = second(what2, side);
  if (e == cudaSuccess) e = cudaEventRecord(done, side);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(stream, done, 0);
  // (destroying a recorded event releases it once the work it marks is done)
  cudaEventDestroy(ready);
  cudaEventDestroy(done);
  return e;
}

}  // namespace cpring
