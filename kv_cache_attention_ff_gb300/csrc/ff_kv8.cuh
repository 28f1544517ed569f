// Device helpers of the 8-bit cache: e4m3 conversions and block scales.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ff_kv8.h"

namespace ff {

// The kernels here are launched so that one may start before the one ahead of it on
// the stream has ended (launch_kernel): grid_wait() stands before the first
// access to memory that another kernel may write or read, and returns when all
// earlier work is complete.  What it hides is the launch itself, some 2 us.
// Memory that those kernels write is read with plain or __ldcg loads: __ldg and
// ld.global.nc take it as constant while the kernel runs, and may be moved
// before the wait.
__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.launch_dependents;\n griddepcontrol.wait;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, int cluster,
                          const A&... args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// Rows held by sequence b, whatever the array says.
__device__ __forceinline__ int kv8_length(const Kv8Layer& c, int b) { return clampi(c.lengths[b], 0, c.capacity); }

__device__ __forceinline__ size_t kv8_tile(const Kv8Layer& c, int b, int block, int h) {
  return (static_cast<size_t>(b) * c.blocks + block) * c.kv_heads + h;
}

// Two e4m3 codes (low byte first) as f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(codes));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  const uint32_t h = e4m3x2_to_f16x2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Nearest e4m3 codes (ties to even) of (lo, hi): magnitudes above 448 and
// infinities become 448, NaN stays NaN.  Low byte first.
__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b16 h;\n cvt.rn.satfinite.e4m3x2.f32 h, %2, %1;\n cvt.u32.u16 %0, h;\n}\n"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// Smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8), for the bits of a finite
// fp32 amax >= 0, within the exponent bounds.
__device__ __forceinline__ int kv8_exponent(uint32_t amax_bits) {
  const int k = static_cast<int>(amax_bits >> 23) - 127;
  const int e = (amax_bits & 0x7fffffu) > 0x600000u ? k - 7 : k - 8;
  return clampi(e, kKv8EMin, kKv8EMax);
}

// 2^e for a normal result.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ int exponent_of(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 0xffu) - 127; }

// 1 / x of a softmax sum (2^-23 relative); 0 where nothing has been summed, and for NaN (whose outputs are NaN
// already).  Results of key ranges are kept divided by their sums: undivided ones may pass the fp32 range with
// the largest scales.
__device__ __forceinline__ float inverse_sum(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return x > 0.f ? r : 0.f;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Largest finite magnitude among the two bf16 values of w, as bf16 bits.
__device__ __forceinline__ uint32_t bf16x2_finite_max(uint32_t w) {
  uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  lo = lo >= 0x7f80u ? 0u : lo;
  hi = hi >= 0x7f80u ? 0u : hi;
  return max(lo, hi);
}

}  // namespace ff
