// Attention of more rows than the token form takes: a warp per (new row, query head).  Each lane has a key's score,
// then some features of the output.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "ff_paged.cuh"

namespace ff {
namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int PER = D / 32;
  __shared__ float sq[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = p.kv_heads * p.group;
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + warp;
  grid_wait();
  const int i = static_cast<int>(unit / heads), j = static_cast<int>(unit % heads);
  const PagedState& s = p.s;
  if (i >= p.n || i >= s.first[s.requests]) return;
  const int r = last_at_most(s.first, s.requests, i);
  const int place = i - s.first[r], news = s.news[r];
  if (place >= news || news > p.most || news <= kPagedTokenRows / p.group) return;
  const int seen = clampi(s.lengths[r], 0, s.capacity) - news + place + 1;
  const size_t at = static_cast<size_t>(i) * heads + j;
  for (int f = lane; f < D; f += 32) sq[warp][f] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[at * D + f]);
  __syncwarp();
  const int h = j / p.group;
  auto row_of = [&](int key) {
    const size_t page = page_at(s, r, key >> s.shift);
    return (((page * p.kv_heads + h) << s.shift) + (key & ((1 << s.shift) - 1))) * D;
  };
  float m = -CUDART_INF_F, l = 0.f, o[PER] = {};
  for (int key0 = 0; key0 < seen; key0 += 32) {
    const int key = key0 + lane;
    float x = -CUDART_INF_F;
    size_t at_key = 0;
    if (key < seen) {
      at_key = row_of(key);
      const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k_pool) + at_key;
      x = 0.f;
      for (int f = 0; f < D; ++f) x = __fmaf_rn(sq[warp][f], __bfloat162float(k[f]), x);
      x *= p.scale_log2;
    }
    float top = x;
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    top = fmaxf(top, m);
    const float z = top == -CUDART_INF_F ? 0.f : top;
    const float before = exp2f(m - z), w = exp2f(x - z);
    m = top;
    float sum = w;
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = __fmaf_rn(l, before, sum);
    for (int f = 0; f < PER; ++f) o[f] *= before;
    for (int k = 0; k < 32 && key0 + k < seen; ++k) {
      const float pk = __shfl_sync(0xffffffffu, w, k);
      const size_t from = __shfl_sync(0xffffffffu, at_key, k);
      for (int f = 0; f < PER; ++f)
        o[f] = __fmaf_rn(pk, __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_pool)[from + f * 32 + lane]), o[f]);
    }
  }
  for (int f = 0; f < PER; ++f) static_cast<__nv_bfloat16*>(p.out)[at * D + f * 32 + lane] = __float2bfloat16(o[f] / l);
  if (lane == 0 && p.lse) p.lse[at] = (m + log2f(l)) * CUDART_LN2_F;
}

}  // namespace

cudaError_t launch_paged_attn(int head_dim, const PagedAttnParams& p, cudaStream_t s) {
  const long long units = static_cast<long long>(p.n) * p.kv_heads * p.group;
  const unsigned grid = static_cast<unsigned>((units + kWarps - 1) / kWarps);
  return launch_kernel(head_dim == 128 ? paged_attn_kernel<128> : paged_attn_kernel<64>, grid, 32 * kWarps, 0, s, 1, p);
}

}  // namespace ff
