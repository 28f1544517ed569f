// A CUDA runtime without a GPU under the host sides of the library: device memory is the host's, and the calls that matter
// are written down in their order.  "memset" may still run on the device when it returns; "wait" waits for the device.
#include <cstdlib>
#include <cstring>
#include <string>

#include <cuda.h>
#include <cuda_runtime_api.h>

#include "ff_kv8.h"

static std::string text;
static unsigned word = 0;

static CUresult encode(...) { return CUDA_SUCCESS; }

extern "C" {

void fake_clear() { text.clear(); }
const char* fake_log() { return text.c_str(); }
// What the next 4 bytes read from the device are.
void fake_word(unsigned x) { word = x; }

cudaError_t cudaGetDeviceCount(int* n) { *n = 1; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr what, int) {
  *v = what == cudaDevAttrComputeCapabilityMajor ? 10 : what == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
  return cudaSuccess;
}
cudaError_t cudaGetDeviceProperties(cudaDeviceProp* p, int) {
  p->major = 10;
  p->minor = 3;
  p->multiProcessorCount = 152;
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t n) {
  *p = std::aligned_alloc(1024, (n + 1023) / 1024 * 1024);
  return *p ? cudaSuccess : cudaErrorMemoryAllocation;
}
cudaError_t cudaFree(void* p) { std::free(p); return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { text += "wait "; return cudaSuccess; }
cudaError_t cudaMemset(void* p, int x, size_t n) {
  std::memset(p, x, n);
  text += "memset ";
  return cudaSuccess;
}
cudaError_t cudaMemcpy(void* to, const void* from, size_t n, cudaMemcpyKind kind) {
  if (kind == cudaMemcpyDeviceToHost && n == sizeof(word)) {
    std::memcpy(to, &word, n);
    word = 0;
  } else {
    std::memcpy(to, from, n);
  }
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* found) {
  *fn = reinterpret_cast<void*>(encode);
  *found = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

}  // extern "C"

namespace ff {
Kv8TokenPlan kv8_token_plan(int, int, int, int) { return {1, 1, 1}; }
Kv8TokenPlan kv8_weigh_plan(int, int, int) { return {1, 1, 1}; }
int paged_token_blocks(int sms) { return 2 * sms; }
}  // namespace ff
