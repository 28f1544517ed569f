// The weight that every cached row received from many query rows, on tcgen05
// tensor cores: weights[j] = weights_in[j] + sum over query rows of
// 2^(score - lse2).
//
// The scores are taken transposed, S^T = K Q^T: a key is a row of the
// accumulator, so one thread owns a key and adds up its probabilities in a
// register, in a fixed order, and nothing is reduced between threads.  A CTA
// keeps 256 keys (converted to bf16 once, exactly) in shared memory and streams
// the query rows past them in tiles of 128, which a tensor map brings as they lie:
// `tg` heads of the group by `tt` tokens.
//   warps 0-3  sums of keys 0..127     warps 8-11  loaders (of the row sums; one thread of the tiles)
//   warps 4-7  sums of keys 128..255   warp  12    TMEM allocator and MMA issuer
// Each key tile's scores are double-buffered in tensor memory (4 x 128
// columns), so a tile's products run while the previous one's are summed.
// With few keys the query rows are cut into ranges as well, whose sums the last
// range to finish adds in order.
#include <type_traits>

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
  static_assert(N_BARS * 8 + 12 <= 256, "barrier area");
  static_assert(SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// (r0, r1) = (a0, a1) * b + (c0, c1) as one packed FMA.
__device__ __forceinline__ void fma2v(float& r0, float& r1, float a0, float a1, float b, float c0, float c1) {
  unsigned long long x, y, z, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b), "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c0), "f"(c1));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r0), "=f"(r1) : "l"(d));
}

// Offset of 16-byte chunk `ch` of row `row` in a tile of column blocks.
__device__ __forceinline__ uint32_t chunk_off(int row, int ch) {
  return (ch >> 3) * (128 * 128) + (row >> 3) * 1024 + (row & 7) * 128 + (((ch & 7) ^ (row & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_chunk_weigh_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ Kv8ChunkWeighParams p) {
  using C = WeighCfg<D>;
  const int kt = blockIdx.x / p.splits, split = blockIdx.x - kt * p.splits;
  const int h = blockIdx.y, b = blockIdx.z;
  grid_wait();
  const int len = kv8_length(p.c, b);
  const int key0 = kt * 256;
  if (key0 >= len) return;
  const int count = p.counts ? clampi(p.counts[b], 0, p.n) : p.n;
  // query tiles: (tokens, heads) of the group; of the first tokens, those that see some key of the CTA
  const int head_tiles = (p.group + p.tg - 1) / p.tg;
  const int first = p.causal ? clampi(key0 - (len - count), 0, count) / p.tt : 0;
  const int n_tiles = max(0, (count + p.tt - 1) / p.tt - first) * head_tiles;
  const int n_split = max(1, min(p.splits, n_tiles));
  if (split >= n_split) return;
  const int t0 = static_cast<int>(static_cast<long long>(n_tiles) * split / n_split);
  const int n = static_cast<int>(static_cast<long long>(n_tiles) * (split + 1) / n_split) - t0;
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
  if (threadIdx.x == 0) tma_prefetch_desc(&tmQ);
  // keys to bf16; rows that are not held are zeros (they own no result)
  {
    constexpr int UNITS = 256 * (D / 16), NU = (UNITS + kThreads - 1) / kThreads;
    uint4 c[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = i * kThreads + threadIdx.x;
      const int key = key0 + u / (D / 16);
      c[i] = make_uint4(0, 0, 0, 0);
      if (u < UNITS && key < len)
        c[i] = __ldcg(reinterpret_cast<const uint4*>(p.c.k8 + kv8_tile(p.c, b, key / kKv8Block, h) * (kKv8Block * D) +
                                                    (key % kKv8Block) * D) + u % (D / 16));
    }
    // the places of a tile that no box fills stay zeros
    if (p.tg * p.tt < 128)
      for (int i = threadIdx.x; i < C::NST * C::TILE / 16; i += kThreads)
        reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = i * kThreads + threadIdx.x;
      if (u >= UNITS) break;
      const int row = u / (D / 16), ch = u % (D / 16);
      const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
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
    // this thread's row of a tile: token r_token of it, head r_head of the group's part
    const int r_token = tid / p.tg, r_head = tid - r_token * p.tg;
    const uint32_t bytes = p.tg * p.tt * D * 2;
    auto row_of = [&](int i, float& nlse, int& seen) {
      const int tile = t0 + i;
      const int token = (first + tile / head_tiles) * p.tt + r_token, head = tile % head_tiles * p.tg + r_head;
      nlse = -CUDART_INF_F;  // nobody's row: 2^(0 - inf) = 0
      seen = 0;
      if (r_token < p.tt && token < count && head < p.group) {
        nlse = -__ldcg(p.lse2 + (static_cast<size_t>(b) * p.n + token) * heads + h * p.group + head);
        seen = p.causal ? len - count + token + 1 : 0x7fffffff;
      }
    };
    float nlse;
    int seen;
    if (n > 0) row_of(0, nlse, seen);
    for (int i = 0; i < n; ++i) {
      const int stage = i % C::NST;
      if (i >= C::NST && !mbar_wait(empty + stage, (i / C::NST - 1) & 1, abort_flag, err)) {
        // given up: no copy of this CTA may land after it has gone
        volatile int no_abort = 0;
        if (tid == 0)
          for (int k = max(0, i - C::NST); k < i; ++k) mbar_wait(full + k % C::NST, (k / C::NST) & 1, &no_abort, err);
        break;
      }
      sLse[stage * 128 + tid] = nlse;
      sSeen[stage * 128 + tid] = seen;
      if (tid == 0) {
        const int tile = t0 + i;
        mbar_expect_tx(full + stage, bytes);
#pragma unroll
        for (int kb = 0; kb < D / 64; ++kb)
          tma_load_3d(smem_u32(sQ) + stage * C::TILE + kb * C::BLK, &tmQ, kb * 64, h * p.group + tile % head_tiles * p.tg,
                      b * p.n + (first + tile / head_tiles) * p.tt, full + stage);
      } else {
        mbar_arrive(full + stage);
      }
      if (i + 1 < n) row_of(i + 1, nlse, seen);
    }
  } else {
    // ------------------------------------------------------------ sums
    const int t = warp >> 2;
    const int key = key0 + threadIdx.x;  // threads 0..255: keys of both tiles
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    if (t == 0 || two) {
      const float f = p.scale_log2 * __ldcg(p.c.ks + kv8_tile(p.c, b, min(key, len - 1) / kKv8Block, h));
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      bool ok = true;
      int token = (first + t0 / head_tiles) * p.tt, head_tile = t0 % head_tiles;  // of tile i
      for (int i = 0; i < n; ++i) {
        const int stage = i % C::NST, slot = t * 2 + (i & 1);
        if (!(ok = mbar_wait(s_full + slot, (i / 2) & 1, abort_flag, err))) break;
        // the row sums were stored before the products were issued
        if (!(ok = mbar_wait(full + stage, (i / C::NST) & 1, abort_flag, err))) break;
        tc_fence_after();
        const uint32_t tS = tmem + lane_off + slot * 128;
        const float4* lse4 = reinterpret_cast<const float4*>(sLse + stage * 128);
        const int4* seen4 = reinterpret_cast<const int4*>(sSeen + stage * 128);
        // Rows of other sequences or heads (past the counts), and keys that a row does not see, are
        // left out by choice, not by arithmetic: what they hold may be NaN.  Rows see more keys
        // the later they come: the tile's first token tells whether any key is hidden.
        const bool masked = token + p.tt > count || (head_tile + 1) * p.tg > p.group ||
                            (p.causal && len - count + token + 1 < key0 + t * 128 + 128);
        // two loops: choosing by element costs as much again as the sums
        auto add_tile = [&](auto hidden) {
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
              fma2v(w[0], w[1], s[4 * k], s[4 * k + 1], f, l.x, l.y);
              fma2v(w[2], w[3], s[4 * k + 2], s[4 * k + 3], f, l.z, l.w);
#pragma unroll
              for (int e = 0; e < 4; ++e) w[e] = ex2_approx(w[e]);
              if constexpr (decltype(hidden)::value) {
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
        };
        if (masked)
          add_tile(std::true_type{});
        else
          add_tile(std::false_type{});
        mbar_arrive(empty + stage);
        if (++head_tile == head_tiles) {
          head_tile = 0;
          token += p.tt;
        }
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

cudaError_t launch_kv8_chunk_weigh(int head_dim, const CUtensorMap& tq, const Kv8ChunkWeighParams& p, cudaStream_t s) {
  const dim3 grid(p.key_tiles * p.splits, p.c.kv_heads, p.c.batch);
  return head_dim == 128 ? launch_kernel(kv8_chunk_weigh_kernel<128>, grid, kThreads, WeighCfg<128>::SMEM, s, 1, tq, p)
                         : launch_kernel(kv8_chunk_weigh_kernel<64>, grid, kThreads, WeighCfg<64>::SMEM, s, 1, tq, p);
}

}  // namespace ff
