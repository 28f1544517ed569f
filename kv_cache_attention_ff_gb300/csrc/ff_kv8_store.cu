// Rows into and out of the 8-bit cache: append (quantising), load
// (dequantising) and eviction by accumulated attention weight.
//
// A block's scale is s = 2^e, e the smallest integer with amax <= 448 * 2^e.
// A power of two costs e4m3 no precision (its relative step does not depend on
// the scale) and makes x / s exact, so a stored value is rounded once, and
// values that move to a block of another scale (a grown block, an eviction)
// are rounded again only where they leave e4m3's normal range.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "ff_kv8.cuh"

namespace ff {
namespace {

constexpr int kTileThreads = 128;

// Largest of the threads' values (bits of non-negative fp32 numbers), for all of them.
__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t* sh) {
  x = __reduce_max_sync(0xffffffffu, x);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  uint32_t m = sh[0];
#pragma unroll
  for (int w = 1; w < kTileThreads / 32; ++w) m = max(m, sh[w]);
  return m;
}

// 16 e4m3 codes of 16 fp32 values times `f`.
__device__ __forceinline__ uint4 codes16(const float* x, float f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = float2_to_e4m3x2(x[4 * i] * f, x[4 * i + 1] * f) |
           (float2_to_e4m3x2(x[4 * i + 2] * f, x[4 * i + 3] * f) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void values16(const uint4& c, float* x) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = e4m3x2_to_float2(w[i] & 0xffffu), b = e4m3x2_to_float2(w[i] >> 16);
    x[4 * i] = a.x;
    x[4 * i + 1] = a.y;
    x[4 * i + 2] = b.x;
    x[4 * i + 3] = b.y;
  }
}

// ------------------------------------------------------------------- append
//
// One thread block per (touched token block, kv head, K or V): it reads its new
// rows once, keeps them in registers while the block's largest magnitude is
// found, and writes their codes.  Traffic is the floor (2 bytes read and 1
// written per value); only the first block of a run that starts inside a block
// reads codes back, and rewrites them when the scale grew.
template <int D>
__global__ void __launch_bounds__(kTileThreads) kv8_append_kernel(const __grid_constant__ Kv8AppendParams p) {
  constexpr int UPR = D / 16;                           // 16-value units per row
  constexpr int NU = kKv8Block * UPR / kTileThreads;    // units per thread
  __shared__ uint32_t sh[kTileThreads / 32];
  const int b = blockIdx.z, h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int held = kv8_length(p.c, b);
  const int start = p.start ? clampi(p.start[b], 0, held) : held;
  const int want = p.counts ? clampi(p.counts[b], 0, p.n) : p.n;
  const int count = min(want, p.c.capacity - start);
  const int end = start + count;
  const int t = start / kKv8Block + blockIdx.x;
  const int row0 = t * kKv8Block;
  if (row0 < end && count > 0) {
    const int rows_before = max(start - row0, 0);  // rows of the block that stay (first block only)
    const size_t tile = kv8_tile(p.c, b, t, h);
    uint8_t* dst = (is_v ? p.c.v8 : p.c.k8) + tile * (kKv8Block * D);
    float* scale = (is_v ? p.c.vs : p.c.ks) + tile;
    const uint4* src = static_cast<const uint4*>(is_v ? p.v : p.k);
    uint4 x[NU][2];
    uint32_t amax = 0;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int unit = u * kTileThreads + threadIdx.x;
      const int row = row0 + unit / UPR;
      x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
      if (row >= start && row < end) {
        const size_t at =
            ((static_cast<size_t>(b) * p.n + (row - start)) * p.c.kv_heads + h) * (D / 8) + (unit % UPR) * 2;
        x[u][0] = __ldcs(src + at);
        x[u][1] = __ldcs(src + at + 1);
      }
    }
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        amax = max(amax, max(max(bf16x2_finite_max(x[u][i].x), bf16x2_finite_max(x[u][i].y)),
                             max(bf16x2_finite_max(x[u][i].z), bf16x2_finite_max(x[u][i].w))));
    const float old_scale = rows_before ? *scale : 0.f;
    int e = kv8_exponent(block_max(amax, sh) << 16);
    if (rows_before) e = max(e, clampi(exponent_of(old_scale), kKv8EMin, kKv8EMax));
    const float new_scale = pow2i(e), inv = pow2i(-e);
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int unit = u * kTileThreads + threadIdx.x;
      const int row = row0 + unit / UPR;
      uint4* d4 = reinterpret_cast<uint4*>(dst) + unit;
      if (row >= start && row < end) {
        float f[16];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w[4] = {x[u][i].x, x[u][i].y, x[u][i].z, x[u][i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[8 * i + 2 * k] = bf16_lo(w[k]);
            f[8 * i + 2 * k + 1] = bf16_hi(w[k]);
          }
        }
        *d4 = codes16(f, inv);
      } else if (row < start && old_scale != new_scale) {
        float f[16];
        values16(*d4, f);
        *d4 = codes16(f, old_scale * inv);
      }
    }
    __syncthreads();  // every thread has read the old scale
    if (threadIdx.x == 0) *scale = new_scale;
  }
  // The last block of a sequence sets its length: all of them have read the old one by then.
  if (threadIdx.x == 0) {
    const unsigned total = gridDim.x * gridDim.y;
    __threadfence();
    if (atomicAdd(p.c.done + b, 1u) == total - 1) {
      p.c.done[b] = 0;
      p.c.lengths[b] = end;
      if (count < want) atomicOr(p.err, kErrCapacity);
    }
  }
}

// --------------------------------------------------------------------- load

template <int D>
__global__ void __launch_bounds__(256) kv8_load_kernel(const __grid_constant__ Kv8LoadParams p) {
  constexpr int UPR = D / 16;
  const int b = blockIdx.y;
  const int units = p.n * p.c.kv_heads * UPR;
  const int unit = blockIdx.x * 256 + threadIdx.x;
  if (unit >= units) return;
  const int part = unit % UPR, h = (unit / UPR) % p.c.kv_heads, i = unit / (UPR * p.c.kv_heads);
  const int start = p.start ? p.start[b] : 0;
  const long long row = static_cast<long long>(start) + i;
  const bool held = row >= 0 && row < kv8_length(p.c, b);
  const size_t tile = held ? kv8_tile(p.c, b, static_cast<int>(row) / kKv8Block, h) : 0;
  const size_t at = tile * (kKv8Block * UPR) + (held ? static_cast<int>(row) % kKv8Block : 0) * UPR + part;
  const size_t to = (static_cast<size_t>(b) * units + unit) * 2;
  uint4 c[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  float s[2] = {0.f, 0.f};
  if (held) {
    c[0] = __ldg(reinterpret_cast<const uint4*>(p.c.k8) + at);
    c[1] = __ldg(reinterpret_cast<const uint4*>(p.c.v8) + at);
    s[0] = p.c.ks[tile];
    s[1] = p.c.vs[tile];
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float x[16];
    values16(c[j], x);
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // exact: four significant bits times a power of two that keeps them normal bf16 numbers
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * k] * s[j], x[2 * k + 1] * s[j]);
      w[k] = *reinterpret_cast<const uint32_t*>(&v);
    }
    uint4* dst = static_cast<uint4*>(j ? p.v : p.k) + to;
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// ------------------------------------------------------------------ eviction
//
// Selection, one cluster of thread blocks per (sequence, kv head): a radix
// select (11, 11 and 10 bits, most significant first) over the weights'
// order-preserving integer keys finds the budget-th largest key T and how many
// rows equal to T still fit; then one ordered pass takes the rows above T, the
// first rows equal to T and the recent rows.  Each block of the cluster keeps its
// share of the keys in shared memory, so the weights are read from memory once
// (as far as they fit: 16384 keys a block), and the blocks' histograms and counts
// are added through distributed shared memory.  The work per key is a few
// instructions; what bounds it is the chain of passes, some 2 us each, which is
// why the digits are wide.

constexpr int kSelThreads = 512;
constexpr int kSelKeys = 16384;  // keys a block keeps in shared memory
constexpr int kSelBins = 2048;
constexpr int kSelShare = 4096;  // keys per block that a cluster is sized for

// Order-preserving key of a weight: larger weight, larger key; -0 equals 0, NaN below every number.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum over the threads before this one, and over all.
__device__ __forceinline__ unsigned sel_scan(unsigned x, unsigned* all, unsigned* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned run = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = run;
  __syncthreads();
  unsigned base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    if (w < warp) base += sh[w];
    total += sh[w];
  }
  *all = total;
  return base + run - x;
}

__global__ void __launch_bounds__(kSelThreads) kv8_select_kernel(const __grid_constant__ Kv8EvictParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t keys[];  // [kSelKeys]
  __shared__ unsigned hist[kSelBins];
  __shared__ unsigned sh[kSelThreads / 32];
  __shared__ unsigned found[2];   // the digit's bin, and rows still needed in it
  __shared__ unsigned counts[2];  // this block's rows above T or recent, and equal to T
  const cg::cluster_group cluster = cg::this_cluster();
  const int n_rank = cluster.num_blocks(), rank = cluster.block_rank();
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31;
  const int len = kv8_length(p.src, b);
  const size_t row = static_cast<size_t>(b) * p.src.kv_heads + h;
  const float* w = p.weights + row * p.src.capacity;
  int* kept = p.kept + row * p.n_keep;
  float* wout = p.weights_out + row * p.dst.capacity;
  const int count = min(len, p.n_keep);
  // what lies behind the kept rows
  for (int j = count + rank * kSelThreads + tid; j < p.n_keep; j += n_rank * kSelThreads) kept[j] = -1;
  for (int j = count + rank * kSelThreads + tid; j < p.dst.capacity; j += n_rank * kSelThreads) wout[j] = 0.f;
  if (len <= p.n_keep) {  // all of them (the whole cluster leaves here)
    for (int j = rank * kSelThreads + tid; j < len; j += n_rank * kSelThreads) {
      kept[j] = j;
      wout[j] = w[j];
    }
    return;
  }
  // a thread's rows are consecutive, an odd number of them (shared memory banks)
  const int per = ((len + n_rank * kSelThreads - 1) / (n_rank * kSelThreads)) | 1;
  const int share = per * kSelThreads;
  const int j0 = rank * share, j1 = min(len, j0 + share);
  const int old = len - p.n_recent;  // rows before the recent ones
  unsigned need = p.n_keep - p.n_recent;
  for (int j = j0 + tid; j < j1; j += kSelThreads)
    if (j - j0 < kSelKeys) keys[j - j0] = weight_key(w[j]);
  auto key_of = [&](int j) { return j - j0 < kSelKeys ? keys[j - j0] : weight_key(w[j]); };

  uint32_t prefix = 0, mask = 0;
  const bool any = need > 0;
  if (any) {
    for (int digit = 0; digit < 3; ++digit) {
      const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bits = digit < 2 ? 11 : 10;
      for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const int end = min(j1, old);
      for (int i = j0; i < end; i += kSelThreads) {
        const int j = i + tid;
        const uint32_t key = j < end ? key_of(j) : 0u;
        const bool in = j < end && (key & mask) == prefix;
        const unsigned bin = in ? (key >> shift) & ((1u << bits) - 1u) : kSelBins;
        // one addition per distinct bin of the warp: weights repeat
        const unsigned same = __match_any_sync(0xffffffffu, bin);
        if (in && lane == __ffs(same) - 1) atomicAdd(&hist[bin], __popc(same));
      }
      cluster.sync();
      // bins from the top: thread t adds up bins 2047 - 4 t .. 2044 - 4 t of all blocks
      constexpr int BPT = kSelBins / kSelThreads;
      unsigned c[BPT] = {}, sum = 0;
      for (int r = 0; r < n_rank; ++r) {
        const uint4 v = reinterpret_cast<const uint4*>(cluster.map_shared_rank(hist, r))[kSelThreads - 1 - tid];
        c[0] += v.w;
        c[1] += v.z;
        c[2] += v.y;
        c[3] += v.x;
      }
#pragma unroll
      for (int k = 0; k < BPT; ++k) sum += c[k];
      unsigned all;
      unsigned above = sel_scan(sum, &all, sh);
      if (above < need && need <= above + sum) {
#pragma unroll
        for (int k = 0; k < BPT; ++k) {
          if (above < need && need <= above + c[k]) {
            found[0] = kSelBins - 1 - BPT * tid - k;
            found[1] = need - above;
          }
          above += c[k];
        }
      }
      cluster.sync();  // every block has read the histograms; `found` is this block's own
      prefix |= found[0] << shift;
      need = found[1];
      mask |= ((1u << bits) - 1u) << shift;
    }
  }
  // prefix is T, `need` the rows equal to T that stay
  const int a0 = j0 + tid * per, a1 = min(j1, a0 + per);
  unsigned sure = 0, eq = 0;
  for (int j = a0; j < a1; ++j) {
    const uint32_t key = key_of(j);
    const bool before = j < old && any;
    sure += (before && key > prefix) || j >= old;
    eq += before && key == prefix;
  }
  unsigned all_sure, all_eq;
  unsigned at = sel_scan(sure, &all_sure, sh);
  unsigned eq_before = sel_scan(eq, &all_eq, sh);
  if (tid == 0) {
    counts[0] = all_sure;
    counts[1] = all_eq;
  }
  cluster.sync();
  unsigned other_eq = 0;
  for (int r = 0; r < rank; ++r) {
    const unsigned* o = cluster.map_shared_rank(counts, r);
    at += o[0];
    other_eq += o[1];
  }
  eq_before += other_eq;
  at += min(eq_before, need);  // equal rows that stay before this thread's
  for (int j = a0; j < a1; ++j) {
    const uint32_t key = key_of(j);
    const bool before = j < old && any;
    bool keep = (before && key > prefix) || j >= old;
    if (before && key == prefix) keep = eq_before++ < need;
    if (keep) {
      kept[at] = j;
      wout[at] = w[j];
      ++at;
    }
  }
  cluster.sync();  // no block leaves while its counts are read
}

// Moves the kept rows, one thread block per (destination block, kv head, K or V).
template <int D>
__global__ void __launch_bounds__(kTileThreads) kv8_move_kernel(const __grid_constant__ Kv8EvictParams p) {
  constexpr int UPR = D / 16;
  constexpr int NU = kKv8Block * UPR / kTileThreads;
  __shared__ uint32_t sh[kTileThreads / 32];
  const int b = blockIdx.z, h = blockIdx.y >> 1, t = blockIdx.x;
  const bool is_v = blockIdx.y & 1;
  const int count = min(kv8_length(p.src, b), p.n_keep);
  if (t == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.dst.lengths[b] = count;
  const int row0 = t * kKv8Block;
  if (row0 >= count) return;
  const int* kept = p.kept + (static_cast<size_t>(b) * p.src.kv_heads + h) * p.n_keep;
  const uint4* src = reinterpret_cast<const uint4*>(is_v ? p.src.v8 : p.src.k8);
  const float* scales = is_v ? p.src.vs : p.src.ks;
  uint4 c[NU];
  float s[NU];
  uint32_t amax = 0;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int unit = u * kTileThreads + threadIdx.x;
    const int row = row0 + unit / UPR;
    c[u] = make_uint4(0, 0, 0, 0);
    s[u] = 0.f;
    if (row < count) {
      const int from = kept[row];
      const size_t tile = kv8_tile(p.src, b, from / kKv8Block, h);
      c[u] = __ldg(src + (tile * kKv8Block + from % kKv8Block) * UPR + unit % UPR);
      s[u] = scales[tile];
    }
  }
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    // magnitudes of e4m3 codes are ordered as their low seven bits; 0x7f is NaN
    uint32_t m = 0;
    const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t v = (w[i / 4] >> (8 * (i % 4))) & 0x7fu;
      m = max(m, v == 0x7fu ? 0u : v);
    }
    amax = max(amax, __float_as_uint(e4m3x2_to_float2(m).x * s[u]));
  }
  const int e = kv8_exponent(block_max(amax, sh));
  const float inv = pow2i(-e);
  const size_t tile = kv8_tile(p.dst, b, t, h);
  uint4* dst = reinterpret_cast<uint4*>((is_v ? p.dst.v8 : p.dst.k8) + tile * (kKv8Block * D));
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int unit = u * kTileThreads + threadIdx.x;
    if (row0 + unit / UPR >= count) continue;
    float x[16];
    values16(c[u], x);
    dst[unit] = codes16(x, s[u] * inv);
  }
  if (threadIdx.x == 0) (is_v ? p.dst.vs : p.dst.ks)[tile] = pow2i(e);
}

}  // namespace

cudaError_t kv8_store_configure() {
  return cudaFuncSetAttribute(kv8_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kSelKeys * sizeof(uint32_t));
}

cudaError_t launch_kv8_append(int head_dim, const Kv8AppendParams& p, cudaStream_t s) {
  // rows start .. start + n - 1 touch at most (n + 126) / 64 blocks
  const dim3 grid((p.n + 2 * kKv8Block - 2) / kKv8Block, 2 * p.c.kv_heads, p.c.batch);
  if (head_dim == 128)
    kv8_append_kernel<128><<<grid, kTileThreads, 0, s>>>(p);
  else
    kv8_append_kernel<64><<<grid, kTileThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv8_load(int head_dim, const Kv8LoadParams& p, cudaStream_t s) {
  const int units = p.n * p.c.kv_heads * (head_dim / 16);
  const dim3 grid((units + 255) / 256, p.c.batch);
  if (head_dim == 128)
    kv8_load_kernel<128><<<grid, 256, 0, s>>>(p);
  else
    kv8_load_kernel<64><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv8_evict(int head_dim, const Kv8EvictParams& p, cudaStream_t s) {
  // blocks per cluster: 4096 rows each, at most 8
  int ranks = 1;
  while (ranks < 8 && static_cast<long long>(ranks) * kSelShare < p.src.capacity) ranks *= 2;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(ranks), 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ranks, p.src.kv_heads, p.src.batch);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = kSelKeys * sizeof(uint32_t);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_select_kernel, p);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.n_keep + kKv8Block - 1) / kKv8Block, 2 * p.src.kv_heads, p.src.batch);
  if (head_dim == 128)
    kv8_move_kernel<128><<<grid, kTileThreads, 0, s>>>(p);
  else
    kv8_move_kernel<64><<<grid, kTileThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ff
