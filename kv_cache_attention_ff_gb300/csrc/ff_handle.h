// What the host sides of the handles (ff_bank.cpp, ff_kv8.cpp, ff_paged.cpp) share: the error word, and those of
// the caches the current device, argument checks and the order of a handle's calls across streams.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "ff.h"

namespace ff {

// Makes a device current for the scope of a call.
class DeviceScope {
 public:
  explicit DeviceScope(int device) {
    ok_ = cudaGetDevice(&before_) == cudaSuccess && (before_ == device || cudaSetDevice(device) == cudaSuccess);
    changed_ = ok_ && before_ != device;
  }
  ~DeviceScope() {
    if (changed_) cudaSetDevice(before_);
  }
  bool ok() const { return ok_; }

 private:
  int before_ = 0;
  bool ok_ = false, changed_ = false;
};

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

inline bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

// Waits for the current device, takes its error word and leaves 0 there; and clears `also` (or null) if `with` says so of the
// word.  A memset may run on when it returns, and the streams of later calls need not wait for the legacy stream that it is
// on: the second wait keeps it from clearing what they count or report.
inline int take_error(unsigned int* err, unsigned int* word, unsigned int with = 0, void* also = nullptr, size_t also_bytes = 0) {
  if (cudaDeviceSynchronize() != cudaSuccess) return FF_ERR_CUDA;
  *word = 0;
  if (cudaMemcpy(word, err, sizeof(*word), cudaMemcpyDeviceToHost) != cudaSuccess) return FF_ERR_CUDA;
  if (!*word) return FF_OK;
  if (cudaMemset(err, 0, sizeof(*word)) != cudaSuccess || ((*word & with) && cudaMemset(also, 0, also_bytes) != cudaSuccess) ||
      cudaDeviceSynchronize() != cudaSuccess)
    return FF_ERR_CUDA;
  return FF_OK;
}

// What enter() found out about a call's stream.
struct CallEntry {
  bool capturing = false;
  unsigned long long stream = 0;
};

// Order of a handle's calls across streams: each comes after the latest one that was not captured.
struct CallOrder {
  cudaEvent_t ev = nullptr;
  unsigned long long last = 0;  // that call's stream's id: handles are used again, and one stands for each thread's own stream
  bool used = false;

  // Before a call's first launch: the stream belongs to the handle's device, and
  // work of other streams on the handle comes first.  A captured call takes no
  // part in that ordering (events from outside a capture cannot enter it).
  int enter(int device, cudaStream_t s, CallEntry* at) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &st) != cudaSuccess) {
      cudaGetLastError();
      return FF_ERR_CUDA;
    }
    at->capturing = st != cudaStreamCaptureStatusNone;
    if (at->capturing) return FF_OK;  // nor may a capturing stream be asked for its device
    int dev = -1;
    if (cudaStreamGetDevice(s, &dev) != cudaSuccess) {
      cudaGetLastError();
      return FF_ERR_ARG;
    }
    if (dev != device) return FF_ERR_ARG;
    if (cudaStreamGetId(s, &at->stream) != cudaSuccess) return FF_ERR_CUDA;
    if (used && last != at->stream && cudaStreamWaitEvent(s, ev, 0) != cudaSuccess) return FF_ERR_CUDA;
    return FF_OK;
  }

  int leave(cudaStream_t s, const CallEntry& at, cudaError_t launched) {
    if (!at.capturing) {
      if (cudaEventRecord(ev, s) != cudaSuccess) return FF_ERR_CUDA;
      last = at.stream;
      used = true;
    }
    return launched == cudaSuccess ? FF_OK : FF_ERR_CUDA;
  }
};

}  // namespace ff
