// The weight that every cached row received from many query rows, on tcgen05
// tensor cores: weights[j] = weights_in[j] + sum over query rows of
// 2^(score - lse2).
//
// The scores are taken transposed, S^T = K Q^T: a key is a row of the
// accumulator, so one thread owns a key and adds up its probabilities in a
// register, in a fixed order, and nothing is reduced between threads.  A CTA
// keeps 256 keys (converted to bf16 once, exactly) in shared memory and streams
// the query rows past them in tiles of 128:
//   warps 0-3  sums of keys 0..127     warps 8-11  query loaders
//   warps 4-7  sums of keys 128..255   warp  12    TMEM allocator and MMA issuer
// Each key tile's scores are double-buffered in tensor memory (4 x 128
// columns), so a tile's products run while the previous one's are summed.
// With few keys the query rows are cut into ranges as well, whose sums the last
// range to finish adds in order.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "ff_kv8.cuh"
#include "ff_ptx.cuh"

namespace ff {
namespace {

constexpr int kThreads = 416;

template <int D>
struct WeighCfg {
  static constexpr int BLK = 128 * 128;     // bytes of one [128 rows x 64 bf16] swizzled block
  static constexpr int TILE = 128 * D * 2;  // a tile of keys or of query rows
  static constexpr int NST = 4;
  static constexpr int OFF_Q = 2 * TILE;
  static constexpr int OFF_LSE = OFF_Q + NST * TILE;
  static constexpr int OFF_SEEN = OFF_LSE + NST * 512;
  static constexpr int OFF_BAR = OFF_SEEN + NST * 512;
  static constexpr int N_BARS = 2 * NST + 8 + 1;
  static constexpr int SMEM = OFF_BAR + 256 + 1024;
  static constexpr int CPT = 128 * D * 2 / 16 / 128;  // 16-byte chunks of a query tile per loader thread
  static_assert(N_BARS * 8 + 12 <= 256, "barrier area");
  static_assert(SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Offset of 16-byte chunk `ch` of row `row` in a tile of column blocks.
__device__ __forceinline__ uint32_t chunk_off(int row, int ch) {
  return (ch >> 3) * (128 * 128) + (row >> 3) * 1024 + (row & 7) * 128 + (((ch & 7) ^ (row & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_chunk_weigh_kernel(const __grid_constant__ Kv8ChunkWeighParams p) {
  using C = WeighCfg<D>;
  const int kt = blockIdx.x / p.splits, split = blockIdx.x - kt * p.splits;
  const int h = blockIdx.y, b = blockIdx.z;
  const int len = kv8_length(p.c, b);
  const int key0 = kt * 256;
  if (key0 >= len) return;
  const int count = p.counts ? clampi(p.counts[b], 0, p.n) : p.n;
  const int rows = count * p.group;
  // query tiles that see some key of the CTA
  const int first = p.causal ? clampi(key0 - (len - count), 0, count) * p.group / 128 : 0;
  const int n_tiles = max(0, (rows + 127) / 128 - first);
  const int n_split = max(1, min(p.splits, n_tiles));
  if (split >= n_split) return;
  const int t0 = first + static_cast<int>(static_cast<long long>(n_tiles) * split / n_split);
  const int n = first + static_cast<int>(static_cast<long long>(n_tiles) * (split + 1) / n_split) - t0;
  const bool two = len - key0 > 128;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::OFF_Q;
  float* sLse = reinterpret_cast<float*>(smem + C::OFF_LSE);
  int* sSeen = reinterpret_cast<int*>(smem + C::OFF_SEEN);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NST;
  uint64_t* s_full = empty + C::NST;  // [key tile][buffer]
  uint64_t* s_free = s_full + 4;
  uint64_t* fin = s_free + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + C::N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = abort_flag + 1;
  const int warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(full + s, 128);
      mbar_init(empty + s, 1 + (two ? 256 : 128));
    }
    for (int t = 0; t < 4; ++t) {
      mbar_init(s_full + t, 1);
      mbar_init(s_free + t, 128);
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    *last_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // keys to bf16; rows that are not held are zeros (they own no result)
  for (int u = threadIdx.x; u < 256 * (D / 16); u += kThreads) {
    const int row = u / (D / 16), ch = u % (D / 16);
    const int key = key0 + row;
    uint4 c = make_uint4(0, 0, 0, 0);
    if (key < len)
      c = __ldg(reinterpret_cast<const uint4*>(p.c.k8 + kv8_tile(p.c, b, key / kKv8Block, h) * (kKv8Block * D) +
                                               (key % kKv8Block) * D) + ch);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t f[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 lo = e4m3x2_to_float2(w[k] & 0xffffu), hi = e4m3x2_to_float2(w[k] >> 16);
      f[2 * k] = pack_bf16x2(lo.x, lo.y);
      f[2 * k + 1] = pack_bf16x2(hi.x, hi.y);
    }
    const uint32_t base = smem_u32(smem) + (row >> 7) * C::TILE;
    st_shared_v4(base + chunk_off(row & 127, 2 * ch), f[0], f[1], f[2], f[3]);
    st_shared_v4(base + chunk_off(row & 127, 2 * ch + 1), f[4], f[5], f[6], f[7]);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  uint32_t* err = p.err;

  float total = 0.f;
  if (warp == 12) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      constexpr uint32_t kIdesc = idesc_bf16(128, 128, 0);
      const uint32_t ka = smem_u32(smem), qa = smem_u32(sQ);
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        const int stage = i % C::NST, buf = i & 1;
        if (!(ok = mbar_wait(full + stage, (i / C::NST) & 1, abort_flag, err))) break;
        for (int t = 0; t < (two ? 2 : 1); ++t) {
          const int slot = t * 2 + buf;
          if (i >= 2 && !(ok = mbar_wait(s_free + slot, (i / 2 - 1) & 1, abort_flag, err))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::BLK + (kk & 3) * 32;
            mma_bf16_ss(tmem + slot * 128, smem_desc(ka + t * C::TILE + off, 16, 1024),
                        smem_desc(qa + stage * C::TILE + off, 16, 1024), kIdesc, kk > 0 ? 1u : 0u);
          }
          mma_commit(s_full + slot);
        }
        if (ok) mma_commit(empty + stage);
      }
      mma_commit(fin);
      mbar_wait(fin, 0, abort_flag, err);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ query loaders
    const int tid = threadIdx.x - 256;
    const int heads = p.c.kv_heads * p.group;
    const size_t base = static_cast<size_t>(b) * p.n * heads + h * p.group;
    float lse_next = 0.f;
    int seen_next = 0;
    auto publish = [&](int i) {  // tile i has arrived: its row sums too, then hand it over
      const int stage = i % C::NST;
      sLse[stage * 128 + tid] = lse_next;
      sSeen[stage * 128 + tid] = seen_next;
      fence_proxy_async_smem();
      mbar_arrive(full + stage);
    };
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int stage = i % C::NST;
      if (i >= C::NST && !(ok = mbar_wait(empty + stage, (i / C::NST - 1) & 1, abort_flag, err))) break;
      const int r0 = (t0 + i) * 128;
      const uint32_t dst = smem_u32(sQ) + stage * C::TILE;
#pragma unroll 4
      for (int k = 0; k < C::CPT; ++k) {
        const int u = k * 128 + tid;
        const int row = u / (D / 8), ch = u % (D / 8);
        const int r = min(r0 + row, rows - 1);
        const size_t at = base + static_cast<size_t>(r / p.group) * heads + r % p.group;
        cp_async16(dst + chunk_off(row, ch), static_cast<const uint4*>(p.q) + at * (D / 8) + ch,
                   r0 + row < rows ? 16 : 0);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (i > 0) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        publish(i - 1);
      }
      const int r = r0 + tid;
      lse_next = CUDART_INF_F;  // rows past the last: 2^(0 - inf) = 0
      seen_next = 0x7fffffff;
      if (r < rows) {
        lse_next = __ldg(p.lse2 + base + static_cast<size_t>(r / p.group) * heads + r % p.group);
        if (p.causal) seen_next = len - count + r / p.group + 1;
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (ok && n > 0) publish(n - 1);
  } else {
    // ------------------------------------------------------------ sums
    const int t = warp >> 2;
    const int key = key0 + threadIdx.x;  // threads 0..255: keys of both tiles
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    if (t == 0 || two) {
      const float f = p.scale_log2 * __ldg(p.c.ks + kv8_tile(p.c, b, min(key, len - 1) / kKv8Block, h));
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int stage = i % C::NST, slot = t * 2 + (i & 1);
        if (!(ok = mbar_wait(s_full + slot, (i / 2) & 1, abort_flag, err))) break;
        // the row sums were stored before the products were issued
        if (!(ok = mbar_wait(full + stage, (i / C::NST) & 1, abort_flag, err))) break;
        tc_fence_after();
        const uint32_t tS = tmem + lane_off + slot * 128;
        const float4* lse4 = reinterpret_cast<const float4*>(sLse + stage * 128);
        const int4* seen4 = reinterpret_cast<const int4*>(sSeen + stage * 128);
        // rows see more keys the later they come: the tile's first row tells whether any key is hidden
        const bool masked = sSeen[stage * 128] < key0 + t * 128 + 128;
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float s[32];
          tmem_ld32(tS + cc * 32, s);
          tmem_wait_ld();
          if (cc == 3) {
            tc_fence_before();
            mbar_arrive(s_free + slot);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 l = lse4[cc * 8 + k];
            float w[4];
            w[0] = ex2_approx(__fmaf_rn(s[4 * k], f, -l.x));
            w[1] = ex2_approx(__fmaf_rn(s[4 * k + 1], f, -l.y));
            w[2] = ex2_approx(__fmaf_rn(s[4 * k + 2], f, -l.z));
            w[3] = ex2_approx(__fmaf_rn(s[4 * k + 3], f, -l.w));
            if (masked) {
              const int4 e = seen4[cc * 8 + k];
              w[0] = key < e.x ? w[0] : 0.f;
              w[1] = key < e.y ? w[1] : 0.f;
              w[2] = key < e.z ? w[2] : 0.f;
              w[3] = key < e.w ? w[3] : 0.f;
            }
            const int a = (k & 1) * 4;
            add2(acc[a], acc[a + 1], w[0], w[1]);
            add2(acc[a + 2], acc[a + 3], w[2], w[3]);
          }
        }
        mbar_arrive(empty + stage);
      }
      total = ((acc[0] + acc[4]) + (acc[1] + acc[5])) + ((acc[2] + acc[6]) + (acc[3] + acc[7]));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  const int key = key0 + threadIdx.x;
  const size_t at = (static_cast<size_t>(b) * p.c.kv_heads + h) * p.c.capacity + key;
  const bool mine = threadIdx.x < 256 && key < len;
  if (n_split == 1) {
    if (mine) p.weights[at] = p.weights_in[at] + total;
    return;
  }
  const size_t item = (static_cast<size_t>(b) * p.c.kv_heads + h) * p.key_tiles + kt;
  float* part = p.part + item * p.splits * 256 + threadIdx.x;
  if (mine) part[split * 256] = total;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool last = atomicAdd(p.tickets + item, 1u) == static_cast<unsigned>(n_split - 1);
    if (last) p.tickets[item] = 0;
    *last_flag = last;
  }
  __syncthreads();
  if (!*last_flag) return;
  __threadfence();
  if (mine) {
    float sum = 0.f;
    for (int k = 0; k < n_split; ++k) sum += __ldcg(part + k * 256);
    p.weights[at] = p.weights_in[at] + sum;
  }
}

}  // namespace

cudaError_t kv8_chunk_weigh_configure(int head_dim) {
  return head_dim == 128 ? cudaFuncSetAttribute(kv8_chunk_weigh_kernel<128>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, WeighCfg<128>::SMEM)
                         : cudaFuncSetAttribute(kv8_chunk_weigh_kernel<64>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, WeighCfg<64>::SMEM);
}

cudaError_t launch_kv8_chunk_weigh(int head_dim, const Kv8ChunkWeighParams& p, cudaStream_t s) {
  const dim3 grid(p.key_tiles * p.splits, p.c.kv_heads, p.c.batch);
  if (head_dim == 128)
    kv8_chunk_weigh_kernel<128><<<grid, kThreads, WeighCfg<128>::SMEM, s>>>(p);
  else
    kv8_chunk_weigh_kernel<64><<<grid, kThreads, WeighCfg<64>::SMEM, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ff
