// The weight that every cached row received from many query rows, on tcgen05
// tensor cores: weights[j] = weights_in[j] + sum over query rows of
// 2^(score - lse2).
//
// The scores are taken transposed, S^T = K Q^T: a key is a row of the
// accumulator, so one thread owns a key and adds up its probabilities in a
// register, in a fixed order, and nothing is reduced between threads.  An item is
// 256 keys and a range of the query rows; the rows pass in tiles of 128, which a
// tensor map brings as they lie: `tg` heads of the group by `tt` tokens.
//   warps 0-3  sums of keys 0..127     warps 8-11  keys to bf16
//   warps 4-7  sums of keys 128..255   warp  12    TMEM allocator and MMA issuer
//   warp  13   query tiles and their row sums
// A CTA stays on its SM and takes every gridDim.x-th item: the next item's keys are
// loaded, converted and stored beside this one's products (a call with a CTA for
// each item took 209 us where this takes 199 at 1560 queries, 220 where it takes 169
// at 26).  Each key tile's scores are double-buffered in tensor memory (4 x 128
// columns), so a tile's products run while the previous one's are summed.
// 1560 queries over 12480 keys, 12 heads, d 128 (60 GFLOP): 66 us, 0.9 PFLOP/s.  A tile
// takes some 2700 clocks: the sums 2400 (exponentials 1064 of them), the products 1360.
// Sixteen warps of sums (by halves of the columns, or every other tile each) gained 1 %
// there and up to 5 % at d 64 with many rows, and lost 4 to 10 % with few; one read of
// a row's sum for two keys, and one arrival a warp in place of each thread's, nothing.
// With few items the query rows are cut into ranges, whose sums the last
// range to finish adds in order.
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>
#include <math_constants.h>

#include "ff_kv8.cuh"
#include "ff_ptx.cuh"

namespace ff {
namespace {

constexpr int kThreads = 448;

template <int D>
struct WeighCfg {
  static constexpr int BLK = 128 * 128;     // bytes of one [128 rows x 64 bf16] swizzled block
  static constexpr int TILE = 128 * D * 2;  // a tile of keys or of query rows
  static constexpr int NST = D == 128 ? 3 : 5;
  static constexpr int OFF_Q = 4 * TILE;  // two items' keys come first
  static constexpr int OFF_LSE = OFF_Q + NST * TILE;
  static constexpr int OFF_BAR = OFF_LSE + NST * 512;
  static constexpr int N_BARS = 2 * NST + 4 + 8 + 1;
  static constexpr int SMEM = OFF_BAR + 256 + 1024;
  static_assert(N_BARS * 8 + 8 <= 256, "barrier area");
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

// A CTA's list of items, every gridDim.x-th, and the item that it stands at: 256
// keys of (b, h) and a range of the query tiles.  Each role of the CTA walks the list
// by itself.  The item's number [b][h][kt][split] is kept digit by digit: a step
// adds gridDim.x's digits (divisions took 1400 clocks an item).
struct ItemWalk {
  int split, kt, h, b;
  int d_split, d_kt, d_h, d_b;
  bool fresh;  // the first item is still to come
  // of the item
  int len, count;
  int first;   // tokens before first * tt see none of the keys
  int n_split;
  int t0, n;   // tiles t0 .. t0 + n - 1 of those from `first` on

  __device__ __forceinline__ static void digits(const Kv8ChunkWeighParams& p, int x, int& split, int& kt, int& h, int& b) {
    int q = x / p.splits;
    split = x - q * p.splits;
    x = q / p.key_tiles;
    kt = q - x * p.key_tiles;
    b = x / p.c.kv_heads;
    h = x - b * p.c.kv_heads;
  }
  __device__ __forceinline__ explicit ItemWalk(const Kv8ChunkWeighParams& p) : fresh(true) {
    digits(p, blockIdx.x, split, kt, h, b);
    digits(p, gridDim.x, d_split, d_kt, d_h, d_b);
  }
  // To the next item that has something to do; false: there is none.
  __device__ __forceinline__ bool next(const Kv8ChunkWeighParams& p) {
    for (;;) {
      if (!fresh) {
        split += d_split;
        kt += d_kt;
        h += d_h;
        b += d_b;
        if (split >= p.splits) split -= p.splits, ++kt;
        if (kt >= p.key_tiles) kt -= p.key_tiles, ++h;
        if (h >= p.c.kv_heads) h -= p.c.kv_heads, ++b;
      }
      fresh = false;
      if (b >= p.c.batch) return false;
      len = kv8_length(p.c, b);
      const int key0 = kt * 256;
      if (key0 >= len) continue;
      count = p.counts ? clampi(p.counts[b], 0, p.n) : p.n;
      const int hidden = p.causal ? clampi(key0 - (len - count), 0, count) : 0;
      first = hidden ? hidden / p.tt : 0;
      const int n_tiles = max(0, (count + p.tt - 1) / p.tt - first) * p.head_tiles;
      n_split = max(1, min(p.splits, n_tiles));
      if (split >= n_split) continue;
      t0 = 0;
      n = n_tiles;
      if (n_split > 1) {
        const int each = n_tiles / n_split, more = n_tiles - each * n_split;
        t0 = split * each + min(split, more);
        n = each + (split < more);
      }
      return true;
    }
  }
  // First token, and first head of the group, of the item's tile i.
  __device__ __forceinline__ void tile(const Kv8ChunkWeighParams& p, int i, int& token0, int& head0) const {
    const int k = t0 + i, q = p.head_tiles == 1 ? k : k / p.head_tiles;
    token0 = (first + q) * p.tt;
    head0 = (k - q * p.head_tiles) * p.tg;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_chunk_weigh_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ Kv8ChunkWeighParams p) {
  using C = WeighCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::OFF_Q;
  float* sLse = reinterpret_cast<float*>(smem + C::OFF_LSE);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NST;
  uint64_t* k_full = empty + C::NST;
  uint64_t* k_empty = k_full + 2;
  uint64_t* s_full = k_empty + 2;  // [key tile][buffer]
  uint64_t* s_free = s_full + 4;
  uint64_t* fin = s_free + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + C::N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(full + s, 32);
      mbar_init(empty + s, 1 + 256);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(k_full + t, 128);
      mbar_init(k_empty + t, 1);
    }
    for (int t = 0; t < 4; ++t) {
      mbar_init(s_full + t, 1);
      mbar_init(s_free + t, 128);
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // the places of a tile that no box fills stay zeros
  if (p.tg * p.tt < 128) {
    for (int i = threadIdx.x; i < C::NST * C::TILE / 16; i += kThreads)
      reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  uint32_t* err = p.err;
  grid_wait();

  ItemWalk w(p);
  if (warp == 12) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      constexpr uint32_t kIdesc = idesc_bf16(128, 128, 0);
      const uint32_t qa = smem_u32(sQ);
      bool ok = true;
      uint32_t it = 0, tile = 0;  // items with tiles, and tiles, of all so far
      while (ok && w.next(p)) {
        if (w.n == 0) continue;
        const uint32_t ka = smem_u32(smem) + (it & 1) * (2 * C::TILE);
        if (!(ok = mbar_wait(k_full + (it & 1), (it >> 1) & 1, abort_flag, err))) break;
        for (int i = 0; i < w.n && ok; ++i, ++tile) {
          const uint32_t stage = tile % C::NST, buf = tile & 1;
          if (!(ok = mbar_wait(full + stage, (tile / C::NST) & 1, abort_flag, err))) break;
          for (int t = 0; t < 2; ++t) {
            const int slot = t * 2 + buf;
            if (tile >= 2 && !(ok = mbar_wait(s_free + slot, (tile / 2 - 1) & 1, abort_flag, err))) break;
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
        mma_commit(k_empty + (it & 1));
        ++it;
      }
      mma_commit(fin);
      mbar_wait(fin, 0, abort_flag, err);
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------ query tiles and their row sums
    const int heads = p.c.kv_heads * p.group;
    const uint32_t bytes = p.tg * p.tt * D * 2;
    int r_token[4], r_head[4];  // this lane's four rows of a tile: token of it, head of the group's part
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r_token[e] = (lane * 4 + e) / p.tg;
      r_head[e] = lane * 4 + e - r_token[e] * p.tg;
    }
    uint32_t tile = 0;
    bool ok = true;
    while (ok && w.next(p)) {
      // four loads in flight; places without a row take another's address
      auto load_rows = [&](int i, float (&v)[4]) {
        int token0, head0;
        w.tile(p, i, token0, head0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int token = min(token0 + r_token[e], w.count - 1), head = min(head0 + r_head[e], p.group - 1);
          v[e] = __ldcg(p.lse2 + (static_cast<size_t>(w.b) * p.n + token) * heads + w.h * p.group + head);
        }
      };
      float v[4] = {};
      if (w.n > 0) load_rows(0, v);
      for (int i = 0; i < w.n; ++i, ++tile) {
        const uint32_t stage = tile % C::NST;
        if (tile >= C::NST && !(ok = mbar_wait(empty + stage, (tile / C::NST - 1) & 1, abort_flag, err))) {
          // given up: no copy of this CTA may land after it has gone
          volatile int no_abort = 0;
          if (lane == 0)
            for (uint32_t k = tile - C::NST; k < tile; ++k)
              mbar_wait(full + k % C::NST, (k / C::NST) & 1, &no_abort, err);
          break;
        }
        int token0, head0;
        w.tile(p, i, token0, head0);
        float nlse[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)  // nobody's row: 2^(0 - inf) = 0
          nlse[e] = r_token[e] < p.tt && token0 + r_token[e] < w.count && head0 + r_head[e] < p.group ? -v[e] : -CUDART_INF_F;
        reinterpret_cast<float4*>(sLse + stage * 128)[lane] = make_float4(nlse[0], nlse[1], nlse[2], nlse[3]);
        if (lane == 0) {
          mbar_expect_tx(full + stage, bytes);
#pragma unroll
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(smem_u32(sQ) + stage * C::TILE + kb * C::BLK, &tmQ, kb * 64,
                        w.h * p.group + head0, w.b * p.n + token0, full + stage);
        } else {
          mbar_arrive(full + stage);
        }
        if (i + 1 < w.n) load_rows(i + 1, v);
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ keys, to bf16 (exactly)
    constexpr int CPR = D / 16, NU = 256 * CPR / 128;  // 16-byte chunks per row and thread
    const int tid = threadIdx.x - 256;
    uint4 c[NU];
    // keys that are not held are zeros (they own no result)
    auto load = [&]() {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int u = i * 128 + tid, key = w.kt * 256 + u / CPR;
        c[i] = make_uint4(0, 0, 0, 0);
        if (key < w.len)
          c[i] = __ldcg(reinterpret_cast<const uint4*>(p.c.k8 + kv8_tile(p.c, w.b, key / kKv8Block, w.h) * (kKv8Block * D) +
                                                      (key % kKv8Block) * D) + u % CPR);
      }
    };
    auto next = [&]() {
      while (w.next(p))
        if (w.n > 0) return true;
      return false;
    };
    bool more = next();
    if (more) load();
    for (uint32_t it = 0; more; ++it) {
      if (it >= 2 && !mbar_wait(k_empty + (it & 1), ((it >> 1) - 1) & 1, abort_flag, err)) break;
      const uint32_t base = smem_u32(smem) + (it & 1) * (2 * C::TILE);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int u = i * 128 + tid, row = u / CPR, ch = u % CPR;
        const uint32_t x[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
        uint32_t f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = e4m3x2_to_float2(x[k] & 0xffffu), hi = e4m3x2_to_float2(x[k] >> 16);
          f[2 * k] = pack_bf16x2(lo.x, lo.y);
          f[2 * k + 1] = pack_bf16x2(hi.x, hi.y);
        }
        const uint32_t to = base + (row >> 7) * C::TILE;
        st_shared_v4(to + chunk_off(row & 127, 2 * ch), f[0], f[1], f[2], f[3]);
        st_shared_v4(to + chunk_off(row & 127, 2 * ch + 1), f[4], f[5], f[6], f[7]);
      }
      fence_proxy_async_smem();
      mbar_arrive(k_full + (it & 1));
      more = next();
      if (more) load();
    }
  } else {
    // ------------------------------------------------------------ sums
    const int t = warp >> 2;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t tile = 0;
    bool ok = true;
    while (w.next(p)) {
      const int key = w.kt * 256 + threadIdx.x;  // threads 0..255: keys of both tiles
      const bool mine = key < w.len;
      const size_t item = (static_cast<size_t>(w.b) * p.c.kv_heads + w.h) * p.key_tiles + w.kt;
      const size_t to = (static_cast<size_t>(w.b) * p.c.kv_heads + w.h) * p.c.capacity + key;
      const float f = p.scale_log2 * __ldcg(p.c.ks + kv8_tile(p.c, w.b, min(key, w.len - 1) / kKv8Block, w.h));
      const float before = mine ? p.weights_in[to] : 0.f;
      const int past = w.len - w.count;  // keys that the first query sees besides its own
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      // tile i: tokens from token0, heads of the group from head0
      int token0, head0;
      w.tile(p, 0, token0, head0);
      for (int i = 0; i < w.n && ok; ++i, ++tile) {
        const uint32_t stage = tile % C::NST;
        const int slot = t * 2 + (tile & 1);
        if (!(ok = mbar_wait(s_full + slot, (tile / 2) & 1, abort_flag, err))) break;
        // the row sums were stored before the products were issued
        if (!(ok = mbar_wait(full + stage, (tile / C::NST) & 1, abort_flag, err))) break;
        tc_fence_after();
        const uint32_t tS = tmem + lane_off + slot * 128;
        const float4* lse4 = reinterpret_cast<const float4*>(sLse + stage * 128);
        // Rows of other sequences or heads (from row_end on), and keys that a row does not see (rows before
        // row_begin), are left out by choice, not by arithmetic: what they hold may be NaN.
        const int row_end = min(min(p.tt, w.count - token0) * p.tg, p.group - head0 + (p.tt - 1) * p.tg);
        const bool masked = row_end < p.tt * p.tg || (p.causal && w.kt * 256 + t * 128 + 127 > past + token0);
        const int row_begin = p.causal ? clampi(key - past - token0, 0, 128) * p.tg : 0;
        // two loops: choosing by element costs as much again as the sums
        auto add_tile = [&](auto hidden) {
          constexpr bool kHidden = decltype(hidden)::value;
          float s[2][32];  // a quarter of the columns is loaded while the one before it is added
          tmem_ld32(tS, s[0]);
          tmem_wait_ld();
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            if (cc < 3) {
              tmem_ld32(tS + (cc + 1) * 32, s[(cc + 1) & 1]);
            } else {
              tc_fence_before();
              mbar_arrive(s_free + slot);
            }
            if (!kHidden || cc * 32 < row_end) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 l = lse4[cc * 8 + k];
                const float* x = s[cc & 1] + 4 * k;
                float v[4];
                fma2v(v[0], v[1], x[0], x[1], f, l.x, l.y);
                fma2v(v[2], v[3], x[2], x[3], f, l.z, l.w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  v[e] = ex2_approx(v[e]);
                  if constexpr (kHidden) {
                    const int row = cc * 32 + 4 * k + e;
                    v[e] = row >= row_begin && row < row_end ? v[e] : 0.f;
                  }
                }
                const int a = (k & 1) * 4;
                add2(acc[a], acc[a + 1], v[0], v[1]);
                add2(acc[a + 2], acc[a + 3], v[2], v[3]);
              }
            }
            if (cc < 3) tmem_wait_ld();
          }
        };
        if (masked)
          add_tile(std::true_type{});
        else
          add_tile(std::false_type{});
        mbar_arrive(empty + stage);
        head0 += p.tg;
        if (head0 >= p.group) {
          head0 = 0;
          token0 += p.tt;
        }
      }
      const float total = ((acc[0] + acc[4]) + (acc[1] + acc[5])) + ((acc[2] + acc[6]) + (acc[3] + acc[7]));
      if (w.n_split == 1) {
        if (mine) p.weights[to] = before + total;
        continue;
      }
      // the last range of a warp's 32 keys to finish adds them all, in order (after a wait that ran out too: the
      // tickets have to come back to 0)
      float* part = p.part + item * p.splits * 256 + threadIdx.x;
      if (mine) part[w.split * 256] = total;
      __threadfence();
      __syncwarp();
      unsigned ticket = 0;
      if (lane == 0) ticket = atomicAdd(p.tickets + item * 8 + warp, 1u);
      if (__shfl_sync(0xffffffffu, ticket, 0) != static_cast<unsigned>(w.n_split - 1)) continue;
      if (lane == 0) p.tickets[item * 8 + warp] = 0;
      __threadfence();
      if (mine) {
        float sum = 0.f;
        for (int k = 0; k < w.n_split; ++k) sum += __ldcg(part + k * 256);
        p.weights[to] = before + sum;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t kv8_chunk_weigh_configure(int head_dim) {
  return head_dim == 128 ? cudaFuncSetAttribute(kv8_chunk_weigh_kernel<128>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, WeighCfg<128>::SMEM)
                         : cudaFuncSetAttribute(kv8_chunk_weigh_kernel<64>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, WeighCfg<64>::SMEM);
}

cudaError_t launch_kv8_chunk_weigh(int head_dim, const CUtensorMap& tq, const Kv8ChunkWeighParams& p, int sms,
                                   cudaStream_t s) {
  const dim3 grid(std::min(p.items, sms));
  return head_dim == 128 ? launch_kernel(kv8_chunk_weigh_kernel<128>, grid, kThreads, WeighCfg<128>::SMEM, s, 1, tq, p)
                         : launch_kernel(kv8_chunk_weigh_kernel<64>, grid, kThreads, WeighCfg<64>::SMEM, s, 1, tq, p);
}

}  // namespace ff
