// Rows into and out of the 8-bit cache: append (quantising), load
// (dequantising) and eviction by accumulated attention weight.
//
// A block's scale is s = 2^e, e the smallest integer with amax <= 448 * 2^e.
// A power of two costs e4m3 no precision (its relative step does not depend on
// the scale) and makes x / s exact, so a stored value is rounded once, and
// values that move to a block of another scale (a grown block, an eviction)
// are rounded again only where they leave e4m3's normal range.
#include <algorithm>

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

// N e4m3 codes (4 to a word) of N fp32 values times `f`, and back.
template <int N>
__device__ __forceinline__ void to_codes(const float* x, float f, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    w[i] = float2_to_e4m3x2(x[4 * i] * f, x[4 * i + 1] * f) |
           (float2_to_e4m3x2(x[4 * i + 2] * f, x[4 * i + 3] * f) << 16);
}
template <int N>
__device__ __forceinline__ void to_values(const uint32_t* w, float* x) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
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
// reads codes back, and rewrites them when the scale grew.  4680 rows of 40 heads at
// d 128 (144 MB): 24 us, 6.0 TB/s of the 6.8 that a copy reaches; one row of 32 sequences
// and 8 heads: 4 us, a chain of dependent loads (length, rows, old scale) and the launch.
template <int D>
__global__ void __launch_bounds__(kTileThreads) kv8_append_kernel(const __grid_constant__ Kv8AppendParams p) {
  constexpr int UPR = D / 8;                            // 8-value units per row (16 bytes in, 8 out)
  constexpr int NU = kKv8Block * UPR / kTileThreads;    // units per thread
  __shared__ uint32_t sh[kTileThreads / 32];
  const int b = blockIdx.z, h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  grid_wait();
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
    uint4 x[NU];
    uint32_t amax = 0;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int unit = u * kTileThreads + threadIdx.x;
      const int row = row0 + unit / UPR;
      x[u] = make_uint4(0, 0, 0, 0);
      if (row >= start && row < end)
        x[u] = __ldcs(src + ((static_cast<size_t>(b) * p.n + (row - start)) * p.c.kv_heads + h) * UPR + unit % UPR);
    }
    // pairs at once; values that are not finite, which do not count, are rare
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      constexpr uint32_t m = 0x7fff7fffu;
      amax = __vmaxu2(__vmaxu2(amax, __vmaxu2(x[u].x & m, x[u].y & m)), __vmaxu2(x[u].z & m, x[u].w & m));
    }
    amax = max(amax >> 16, amax & 0xffffu);
    if (amax >= 0x7f80u) {
      amax = 0;
#pragma unroll
      for (int u = 0; u < NU; ++u)
        amax = max(amax, max(max(bf16x2_finite_max(x[u].x), bf16x2_finite_max(x[u].y)),
                             max(bf16x2_finite_max(x[u].z), bf16x2_finite_max(x[u].w))));
    }
    const float old_scale = rows_before ? *scale : 0.f;
    int e = kv8_exponent(block_max(amax, sh) << 16);
    if (rows_before) e = max(e, clampi(exponent_of(old_scale), kKv8EMin, kKv8EMax));
    const float new_scale = pow2i(e), inv = pow2i(-e);
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int unit = u * kTileThreads + threadIdx.x;
      const int row = row0 + unit / UPR;
      uint2* to = reinterpret_cast<uint2*>(dst) + unit;
      uint32_t w[2];
      float f[8];
      if (row >= start && row < end) {
        const uint32_t v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[2 * k] = bf16_lo(v[k]);
          f[2 * k + 1] = bf16_hi(v[k]);
        }
        to_codes<8>(f, inv, w);
        *to = make_uint2(w[0], w[1]);
      } else if (row < start && old_scale != new_scale) {
        const uint2 c = *to;
        w[0] = c.x;
        w[1] = c.y;
        to_values<8>(w, f);
        to_codes<8>(f, old_scale * inv, w);
        *to = make_uint2(w[0], w[1]);
      }
    }
    __syncthreads();  // every thread has read the old scale
    if (threadIdx.x == 0) *scale = new_scale;
  }
  // The last block of a sequence sets its length: all of them have read the old one by then,
  // with every thread, also of a block that found nothing to do.
  __syncthreads();
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

// Thread blocks of 32 rows of one kv head; a thread takes 8 values of one or two
// rows, in K and V: 8 bytes in and 16 out for each, so that both sides of a
// warp are whole lines.  15600 rows of 12 heads at d 128 (144 MB): 20 us, 7.1 TB/s (a
// part of the rows still lies in L2).
constexpr int kLoadThreads = 256;
constexpr int kLoadRows = 32;

template <int D>
__global__ void __launch_bounds__(kLoadThreads) kv8_load_kernel(const __grid_constant__ Kv8LoadParams p) {
  constexpr int UPR = D / 8;                          // 8-value units per row
  constexpr int ROWS = kLoadThreads / UPR;            // rows of a pass
  constexpr int NU = kLoadRows / ROWS;
  const int b = blockIdx.z, h = blockIdx.y;
  const int part = threadIdx.x % UPR, i0 = blockIdx.x * kLoadRows + threadIdx.x / UPR;
  grid_wait();
  const int len = kv8_length(p.c, b);
  const long long row0 = static_cast<long long>(p.start ? p.start[b] : 0) + i0;
  uint2 c[NU][2];
  float s[NU][2];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const long long row = row0 + u * ROWS;
    c[u][0] = c[u][1] = make_uint2(0, 0);
    s[u][0] = s[u][1] = 0.f;
    if (i0 + u * ROWS < p.n && row >= 0 && row < len) {
      const int r = static_cast<int>(row);
      const size_t tile = kv8_tile(p.c, b, r / kKv8Block, h);
      const size_t at = (tile * kKv8Block + r % kKv8Block) * UPR + part;
      c[u][0] = __ldcg(reinterpret_cast<const uint2*>(p.c.k8) + at);
      c[u][1] = __ldcg(reinterpret_cast<const uint2*>(p.c.v8) + at);
      s[u][0] = __ldcg(p.c.ks + tile);
      s[u][1] = __ldcg(p.c.vs + tile);
    }
  }
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int i = i0 + u * ROWS;
    if (i >= p.n) break;
    const size_t to = ((static_cast<size_t>(b) * p.n + i) * p.c.kv_heads + h) * UPR + part;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t w[2] = {c[u][j].x, c[u][j].y};
      float x[8];
      to_values<8>(w, x);
      uint32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // exact: four significant bits times a power of two that keeps them normal bf16 numbers
        const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * k] * s[u][j], x[2 * k + 1] * s[u][j]);
        v[k] = *reinterpret_cast<const uint32_t*>(&t);
      }
      __stcs(static_cast<uint4*>(j ? p.v : p.k) + to, make_uint4(v[0], v[1], v[2], v[3]));
    }
  }
}

// ------------------------------------------------------------------ eviction
//
// Selection, one cluster of thread blocks per (sequence, kv head): a radix
// select (8 bits a pass, most significant first) over the weights'
// order-preserving integer keys finds the budget-th largest key T and how many
// rows equal to T still fit; then one ordered pass takes the rows above T, the
// first rows equal to T and the recent rows.  Each block of the cluster keeps its
// share of the keys in shared memory, so the weights are read from memory once
// (as far as they fit: 16384 keys a block), and the blocks' histograms and counts
// are added through distributed shared memory.  What bounds it is the chain of
// steps: a pass over 3900 keys a block takes about 1 us, of which the keys are a
// sixth, the cluster's barrier and the loads of the others' histograms two thirds.
// (Passes of 11 bits are one fewer, but their histograms took 2 us each to add;
// increments of one, equal bins of a warp among them, are single instructions in
// shared memory, where collecting equal bins first took 2.7 us.)  12 heads of 31200
// rows take 16 us in all: three quarters of it the passes, the clusters' uneven
// start and the launch.

constexpr int kSelThreads = 512;
constexpr int kSelKeys = 16384;  // keys a block keeps in shared memory
constexpr int kSelBins = 256;
constexpr int kSelShare = 2048;  // keys per block that a cluster is sized for
constexpr int kSelRanks = 8;     // blocks of a cluster, at most

// Order-preserving key of a weight: larger weight, larger key; -0 equals 0, NaN below every number.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The weight of a key (of a number: NaN has no key of its own).
__device__ __forceinline__ float key_weight(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// Sums of x[0] and x[1] over the threads before this one, and over all, of the first
// WARPS warps (the others only come to the barrier).  `sh` is not in use by a scan before it.
template <int WARPS, int N>
__device__ __forceinline__ void sel_scan(unsigned (&x)[N], unsigned (&all)[N], unsigned (*sh)[kSelThreads / 32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned run[N];
#pragma unroll
  for (int i = 0; i < N; ++i) run[i] = x[i];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned y = __shfl_up_sync(0xffffffffu, run[i], o);
      if (lane >= o) run[i] += y;
    }
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < N; ++i) sh[i][warp] = run[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    unsigned base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const unsigned y = sh[i][w];
      base += w < warp ? y : 0u;
      total += y;
    }
    all[i] = total;
    x[i] = base + run[i] - x[i];
  }
}

__global__ void __launch_bounds__(kSelThreads) kv8_select_kernel(const __grid_constant__ Kv8EvictParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t keys[];  // [p.select_keys]
  __shared__ unsigned hist_all[4][kSelBins];  // one for each digit: a block may still read another's last one
  __shared__ unsigned sh[6][kSelThreads / 32];  // one row for each sum of a scan
  __shared__ unsigned found[4][2];  // each digit's bin, and rows still needed in it
  __shared__ unsigned counts[2];    // this block's rows above T or recent, and equal to T
  const cg::cluster_group cluster = cg::this_cluster();
  const int n_rank = cluster.num_blocks(), rank = cluster.block_rank();
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  grid_wait();
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
  const int in_smem = min(j1, j0 + p.select_keys);
#pragma unroll 8
  for (int j = j0 + tid; j < in_smem; j += kSelThreads) keys[j - j0] = weight_key(w[j]);
  for (int i = tid; i < 4 * kSelBins; i += kSelThreads) hist_all[0][i] = 0;
  __syncthreads();
  auto key_of = [&](int j) { return j < in_smem ? keys[j - j0] : weight_key(w[j]); };

  uint32_t prefix = 0, mask = 0;
  const bool any = need > 0;
  if (any) {
    for (int digit = 0; digit < 4; ++digit) {
      const int shift = 24 - 8 * digit;
      unsigned* hist = hist_all[digit];
      const int end = min(j1, old);
      const auto count = [&](uint32_t key) {
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      };
      const int near = min(end, in_smem);
#pragma unroll 8
      for (int j = j0 + tid; j < near; j += kSelThreads) count(keys[j - j0]);
      for (int j = near + tid; j < end; j += kSelThreads) count(weight_key(w[j]));
      cluster.sync();
      // bins from the top: thread t adds up bin 255 - t of all blocks
      unsigned v[kSelRanks];
#pragma unroll
      for (int r = 0; r < kSelRanks; ++r)
        v[r] = r < n_rank && tid < kSelBins ? cluster.map_shared_rank(hist, r)[kSelBins - 1 - tid] : 0u;
      unsigned sum = 0;
#pragma unroll
      for (int r = 0; r < kSelRanks; ++r) sum += v[r];
      unsigned above[1] = {sum}, all[1];
      sel_scan<kSelBins / 32>(above, all, sh + digit);
      if (above[0] < need && need <= above[0] + sum && tid < kSelBins) {
        found[digit][0] = kSelBins - 1 - tid;
        found[digit][1] = need - above[0];
      }
      __syncthreads();
      prefix |= found[digit][0] << shift;
      need = found[digit][1];
      mask |= 255u << shift;
    }
  }
  // prefix is T, `need` the rows equal to T that stay
  const int a0 = j0 + tid * per, a1 = min(j1, a0 + per);
  // A thread's rows in eights, whose keys are loaded at once: step(j, sure, eq) for each.
  const auto each_row = [&](auto step) {
    for (int j8 = a0; j8 < a1; j8 += 8) {
      uint32_t key[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) key[i] = j8 + i < a1 ? key_of(j8 + i) : 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = j8 + i;
        if (j >= a1) break;
        const bool before = j < old && any;
        step(j, key[i], (before && key[i] > prefix) || j >= old, before && key[i] == prefix);
      }
    }
  };
  unsigned mine[2] = {0, 0}, all[2];  // rows above T or recent, and equal to T
  each_row([&](int, uint32_t, bool sure, bool eq) {
    mine[0] += sure;
    mine[1] += eq;
  });
  sel_scan<kSelThreads / 32>(mine, all, sh + 4);
  if (tid == 0) {
    counts[0] = all[0];
    counts[1] = all[1];
  }
  cluster.sync();
  unsigned at = mine[0], eq_before = mine[1];
#pragma unroll
  for (int r = 0; r < kSelRanks; ++r)
    if (r < rank) {
      const unsigned* o = cluster.map_shared_rank(counts, r);
      at += o[0];
      eq_before += o[1];
    }
  // no block leaves while its counts are read: these have arrived when the barrier is told so
  asm volatile("barrier.cluster.arrive.relaxed;" : "+r"(at), "+r"(eq_before)::"memory");
  at += min(eq_before, need);  // equal rows that stay before this thread's
  each_row([&](int j, uint32_t key, bool sure, bool eq) {
    if (sure || (eq && eq_before++ < need)) {
      kept[at] = j;
      wout[at] = key ? key_weight(key) : w[j];
      ++at;
    }
  });
  asm volatile("barrier.cluster.wait;" ::: "memory");
}

// Moves the kept rows, one thread block per (destination block, kv head, K or V):
// 1 byte read and written per value, the rows gathered in pieces of 64 or 128 bytes.
// Half of 31200 rows of 12 heads at d 128 (96 MB): 19 us, 5.0 TB/s; the latency of
// index, row and write bounds it more than bandwidth does.
template <int D>
__global__ void __launch_bounds__(kTileThreads) kv8_move_kernel(const __grid_constant__ Kv8EvictParams p) {
  constexpr int UPR = D / 16;
  constexpr int NU = kKv8Block * UPR / kTileThreads;
  __shared__ uint32_t sh[kTileThreads / 32];
  const int b = blockIdx.z, h = blockIdx.y >> 1, t = blockIdx.x;
  const bool is_v = blockIdx.y & 1;
  grid_wait();
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
      c[u] = __ldcg(src + (tile * kKv8Block + from % kKv8Block) * UPR + unit % UPR);
      s[u] = scales[tile];
    }
  }
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    // magnitudes of e4m3 codes are ordered as their low seven bits; 0x7f is NaN, which is rare
    const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = __vmaxu2(__vmaxu2(m, w[i] & 0x007f007fu), (w[i] >> 8) & 0x007f007fu);
    m = max(m >> 16, m & 0xffffu);
    if (m == 0x7fu) {
      m = 0;
      for (int i = 0; i < 16; ++i) {
        const uint32_t v = (w[i / 4] >> (8 * (i % 4))) & 0x7fu;
        m = max(m, v == 0x7fu ? 0u : v);
      }
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
    if (s[u] * inv == 1.f) {  // the block's scale is the row's old one: its codes stay
      dst[unit] = c[u];
      continue;
    }
    uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
    float x[16];
    to_values<16>(w, x);
    // zeros may come from a block of any scale: the factor stays finite for them
    to_codes<16>(x, fminf(s[u] * inv, 0x1p100f), w);
    dst[unit] = make_uint4(w[0], w[1], w[2], w[3]);
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
  return launch_kernel(head_dim == 128 ? kv8_append_kernel<128> : kv8_append_kernel<64>, grid, kTileThreads, 0, s, 1, p);
}

cudaError_t launch_kv8_load(int head_dim, const Kv8LoadParams& p, cudaStream_t s) {
  const dim3 grid((p.n + kLoadRows - 1) / kLoadRows, p.c.kv_heads, p.c.batch);
  return launch_kernel(head_dim == 128 ? kv8_load_kernel<128> : kv8_load_kernel<64>, grid, kLoadThreads, 0, s, 1, p);
}

cudaError_t launch_kv8_evict(int head_dim, const Kv8EvictParams& p, int sms, cudaStream_t s) {
  // Blocks per cluster: 2048 rows each, at most 8 (12 heads of 3000 rows, evicted and read back: 17.7 us
  // with 4096 rows a block, 15.3 with 2048; 8 heads of 1500 rows 13.1 with one block, 15.1 with two), and
  // doubled while all heads' blocks are no more than the SMs, which ends at two for each SM at most (12 heads of
  // 31200 rows 65 us with four blocks, 61 with eight; 128 heads of 8190 rows 34.7 with two, 39.2 with one, which
  // is where a block an SM would end, and 40 heads of 31200 rows 168 with four and 183 with two; 512 heads of 8190
  // rows 95 with one, 125 with four: the clusters' barriers).
  const long long items = static_cast<long long>(p.src.kv_heads) * p.src.batch;
  int ranks = 1;
  while (ranks < kSelRanks && static_cast<long long>(ranks) * kSelShare < p.src.capacity && items * ranks <= sms)
    ranks *= 2;
  // no more shared memory than a full sequence's share takes: more blocks per SM
  const int per = ((p.src.capacity + ranks * kSelThreads - 1) / (ranks * kSelThreads)) | 1;
  Kv8EvictParams q = p;
  q.select_keys = std::min(kSelKeys, per * kSelThreads);
  const cudaError_t e = launch_kernel(kv8_select_kernel, dim3(ranks, p.src.kv_heads, p.src.batch), kSelThreads,
                                      q.select_keys * sizeof(uint32_t), s, ranks, q);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.n_keep + kKv8Block - 1) / kKv8Block, 2 * p.src.kv_heads, p.src.batch);
  return launch_kernel(head_dim == 128 ? kv8_move_kernel<128> : kv8_move_kernel<64>, grid, kTileThreads, 0, s, 1, p);
}

}  // namespace ff
