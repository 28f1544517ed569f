// Attention of many query rows over the 8-bit cache on tcgen05 tensor cores.
//
// A unit is one (sequence, kv head) and 256 of its query rows (row r = token
// r / group, head r mod group), a CTA one unit or one key range of it:
//   warps 0-3          softmax of rows 0..127: one thread per row
//   warps 4-7          softmax of rows 128..255
//   warps 8-11, 13-15  producers: codes from global memory, to f16, to shared memory
//   warp  12           TMEM allocator and single-thread MMA issuer
// Tensor memory (512 columns): S0 | S1 | O0 | O1.  Per key tile j of 128 keys the
// MMA thread issues S0 = Q0 K_j^T, O0 += P0 V_{j-1}, S1 = Q1 K_j^T,
// O1 += P1 V_{j-1}: the tensor pipe works on one query tile's products while
// the other's scores become probabilities.  Where one tile of 128 holds all
// query rows (ONE), both groups have its rows and take every other key tile; their
// maxima, sums and outputs meet at the end.
//
// Codes become f16 exactly, on the way into shared memory (kind::f16 wants both
// operands of one type, and e4m3 queries or probabilities would cost the
// result its precision).  Scales never touch an operand: K's multiplies the
// scores, V's enters as an exponent of the probabilities, which are
// 2^(s - m + kOff + ev - R) in f16 (11 bits) with 2^ev the V block's scale, m the
// running maximum of the scores (for the sum) and 2^(m + R) the unit of the
// row's output.  Both belong to the row, and follow what it sees: the unit is the
// running maximum of probability times scale, so a large block that a row does
// not see, or gives no weight, costs it nothing.  m rises by more than 2^4 at a
// time (R then falls as much: the output stays as it is), the unit by more than
// 2^2, and only that rescales the output.  f16 holds 11 bits of what lies down to
// 2^-19 below the unit; anything is rounded by at most 2^-30 of the unit times
// its code.  Queries are scaled per row by a power of two (exact).
//
// 4680 queries over 31200 keys, 12 heads, d 128 (897 GFLOP): 602 to 612 us at 2070 MHz, 625
// to 636 in series long enough for the power cap (1960 to 2020 MHz): 1.41 to 1.49 PFLOP/s,
// 0.76 to 0.80 of a large product's rate.  A pair of query tiles and a key tile
// takes some 3600 clocks, 2048 of them products; the rest is the chain of scores,
// probabilities and products, and the f16 tiles' way through shared memory, whose
// bandwidth the operands share.  Cutting all units into equal runs of key tiles
// measured 690 us, codes copied by TMA and expanded in place 733, and issuing
// S0, S1, PV0, PV1 702.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "ff_kv8.cuh"
#include "ff_ptx.cuh"

namespace ff {
namespace {

constexpr int kThreads = 512;
constexpr float kOff = 5.f;   // 2^(4 + 5 + 2) < 65504: stale maximum, offset, stale unit
constexpr float kMaxDrift = 2.f;
constexpr float kNoUnit = -200.f;  // of a row that has seen nothing: below every scale's exponent
constexpr int kPrefetchTiles = 6;
constexpr int kProducers = 224;

template <int D>
struct ChunkCfg {
  static constexpr int KB = D / 64;              // 128-byte column blocks per f16 row
  static constexpr int BLK = 128 * 128;          // bytes of one [128 rows x 64 f16] swizzled block
  static constexpr int Q_BYTES = 128 * D * 2;
  static constexpr int KV_BYTES = 128 * D * 2;
  static constexpr int P_BYTES = 128 * 128 * 2;
  static constexpr int NST = (D == 128) ? 3 : 4;
  static constexpr int OFF_P = 2 * Q_BYTES;
  static constexpr int OFF_KV = OFF_P + 2 * P_BYTES;
  static constexpr int OFF_BAR = OFF_KV + NST * KV_BYTES;
  static constexpr int N_BARS = 2 + 2 * NST + 8 + 1;
  static constexpr int SMEM = OFF_BAR + 256 + 1024;
  static_assert(N_BARS * 8 + 8 <= 256, "barrier area");
  static_assert(SMEM <= 232448, "shared memory");
  static constexpr int TMEM_S = 0;
  static constexpr int TMEM_O = 256;
};

// f16 operands, fp32 accumulator (format fields 0), A K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Fetch `bytes` (a multiple of 16) at a 16-byte aligned address into L2.
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// 16 bytes that this CTA reads once: not kept in L1.
__device__ __forceinline__ uint4 ldg_stream(const uint8_t* src) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(src));
  return v;
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ float4 ld_shared_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void st_shared_f4(uint32_t a, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// What a CTA (or a row of the merge) works on, from the lengths on the device.
struct Work {
  int b, h, row0, nrow;   // query rows row0 .. row0 + nrow - 1 of (b, h); nrow 0: nothing to do
  int len, count, n_keys; // rows held, valid queries, keys that some row sees
  int n_kv, n_split;      // key tiles, key ranges
};

__device__ __forceinline__ int seen_by(const Work& w, int causal, int group, int row) {
  return causal ? max(0, w.len - w.count + row / group + 1) : w.len;
}

__device__ __forceinline__ Work work_of(const Kv8ChunkParams& p, int unit, int splits) {
  Work w;
  const int bh = unit / p.row_blocks;
  // the rows that see most come first
  const int rb = p.row_blocks - 1 - (unit - bh * p.row_blocks);
  w.b = bh / p.c.kv_heads;
  w.h = bh - w.b * p.c.kv_heads;
  w.len = kv8_length(p.c, w.b);
  w.count = p.counts ? clampi(p.counts[w.b], 0, p.n) : p.n;
  w.row0 = rb * 256;
  w.nrow = clampi(w.count * p.group - w.row0, 0, 256);
  w.n_keys = w.nrow ? min(w.len, seen_by(w, p.causal, p.group, w.row0 + w.nrow - 1)) : 0;
  w.n_kv = (w.n_keys + 127) / 128;
  w.n_split = max(1, min(splits, w.n_kv));
  return w;
}

// Index of query row `row` of (b, h) in [batch, n, heads].
__device__ __forceinline__ size_t query_at(const Kv8ChunkParams& p, const Work& w, int row) {
  return (static_cast<size_t>(w.b) * p.n + row / p.group) * (p.c.kv_heads * p.group) + w.h * p.group + row % p.group;
}

// The places of rows row, row + step, .. of a unit in [batch, n, heads], one after the other.
struct RowWalk {
  size_t at;
  int g, group, heads, dq, dr;
  __device__ __forceinline__ RowWalk(const Kv8ChunkParams& p, const Work& w, int row, int step) {
    group = p.group;
    heads = p.c.kv_heads * p.group;
    const int token = row / group;
    g = row - token * group;
    at = (static_cast<size_t>(w.b) * p.n + token) * heads + w.h * group + g;
    dq = step / group * heads;
    dr = step % group;
  }
  __device__ __forceinline__ void next() {
    at += dq + dr;
    g += dr;
    if (g >= group) {
      g -= group;
      at += heads - group;
    }
  }
};

// Producer threads (7 warps): each takes 16-byte chunks (16 codes) of every tile
// from global memory to f16 in the ring.  A chunk's registers are refilled from
// the ring's next tile as soon as they are read: 16 KB of loads in flight, which
// pass through the 28 KB of L1 that the shared memory leaves (two tiles in
// flight do not fit there and measured 25 % slower; a copy into shared memory first
// adds its latency to every slot's refill and measured 10 % slower).
template <int D, int LAG>
__device__ __forceinline__ void produce(const Kv8ChunkParams& p, const Work& w, int kv0, int n, int tid, uint32_t ring,
                                        uint64_t* kv_full, uint64_t* kv_empty, volatile int* abort_flag,
                                        uint32_t* err) {
  using C = ChunkCfg<D>;
  constexpr int PER_ROW = D / 16;
  constexpr int NU = (128 * PER_ROW + kProducers - 1) / kProducers;  // chunks of a tile per thread, at most
  constexpr int ROWS = kProducers / PER_ROW;                         // rows that one pass of the threads covers
  static_assert(ROWS % 4 == 0, "a thread's rows agree in their place of 8 but for its top bit");
  // The 16 codes are two 16-byte chunks of the f16 row.  Threads of the second
  // 64-feature column block take the neighbouring row, which keeps the banks of a
  // store apart (a row's chunks are xored with its place of 8).
  const int ch = tid % PER_ROW, row0 = (tid / PER_ROW) ^ (ch >> 2);
  const uint32_t to_even = (ch >> 2) * C::BLK + row0 * 128 + ((((ch & 3) * 2) ^ (row0 & 7)) << 4);
  const uint32_t to_odd = ROWS % 8 ? to_even ^ 64 : to_even;         // passes with an odd number
  const size_t step = static_cast<size_t>(p.c.kv_heads) * (kKv8Block * D);  // from a block to the next
  const size_t first = kv8_tile(p.c, w.b, 0, w.h) * (kKv8Block * D) + row0 * D + ch * 16;
  // ring order: K_0 .. K_{LAG-1}, then (K_j, V_{j-LAG}) for j >= LAG, then the last V
  const int lead = LAG == 1 ? 1 : min(n, LAG);
  auto is_v = [&](int li) { return li >= lead && (((li - lead) & 1) || li >= 2 * n - lead); };
  auto tile_of = [&](int li) {
    return li >= 2 * n - lead ? li - n : li < lead ? li : is_v(li) ? (li - lead) / 2 : (li + lead) / 2;
  };
  uint4 x[NU];
  const uint8_t* src = nullptr;  // the thread's first chunk of the tile to load
  int held = 0;                  // rows of that tile that are held
  auto aim = [&](int li) {
    held = 0;
    if (li >= 2 * n) return;
    const int j = kv0 + tile_of(li);
    held = min(128, w.len - j * 128);
    src = (is_v(li) ? p.c.v8 : p.c.k8) + first + static_cast<size_t>(2 * j) * step;
  };
  // rows that are not held are zeros: what lies there may be NaN
  auto load = [&](int i) {
    const int row = i * ROWS + row0;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < held) v = ldg_stream(src + i * ROWS * D + (row >= kKv8Block ? step - kKv8Block * D : 0));
    return v;
  };
  aim(0);
#pragma unroll
  for (int i = 0; i < NU; ++i) x[i] = load(i);
  for (int li = 0; li < 2 * n; ++li) {
    const int stage = li % C::NST;
    const uint32_t use = li / C::NST;
    aim(li + 1);
    if (use > 0 && !mbar_wait(kv_empty + stage, (use - 1) & 1, abort_flag, err)) return;
    const uint32_t slot = ring + stage * C::KV_BYTES;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t c[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t f[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[2 * q] = e4m3x2_to_f16x2(c[q] & 0xffffu);
        f[2 * q + 1] = e4m3x2_to_f16x2(c[q] >> 16);
      }
      x[i] = load(i);
      if (i * ROWS + row0 < 128) {
        const uint32_t at = slot + (i & 1 ? to_odd : to_even);
        st_shared_v4(at + i * ROWS * 128, f[0], f[1], f[2], f[3]);
        st_shared_v4((at ^ 16) + i * ROWS * 128, f[4], f[5], f[6], f[7]);
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(kv_full + stage);
  }
}

template <int D, bool ONE>
__global__ void __launch_bounds__(kThreads, 1) kv8_chunk_kernel(const __grid_constant__ Kv8ChunkParams p) {
  using C = ChunkCfg<D>;
  // what needs no memory of other kernels comes before the wait for them
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sP = smem + C::OFF_P;
  uint8_t* sKV = smem + C::OFF_KV;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* kv_full = q_full + 2;
  uint64_t* kv_empty = kv_full + C::NST;
  uint64_t* s_full = kv_empty + C::NST;
  uint64_t* s_free = s_full + 2;
  uint64_t* p_full = s_full + 4;
  uint64_t* o_done = s_full + 6;
  uint64_t* fin = s_full + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + C::N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(kv_full + s, kProducers);
      mbar_init(kv_empty + s, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full + t, 128);
      mbar_init(s_full + t, 1);
      mbar_init(s_free + t, 128);
      mbar_init(p_full + t, 128);
      mbar_init(o_done + t, 1);
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();
  const int piece = blockIdx.x;
  const bool whole = piece < p.n_whole;
  const int unit = whole ? piece : p.n_whole + (piece - p.n_whole) / p.splits;
  const int split = whole ? 0 : (piece - p.n_whole) % p.splits;
  const Work w = work_of(p, unit, whole ? 1 : p.splits);
  if (w.nrow == 0 || split >= w.n_split) {
    if (warp == 12) tmem_dealloc(tmem, 512);
    return;
  }
  const int kv0 = static_cast<int>(static_cast<long long>(w.n_kv) * split / w.n_split);
  const int kv1 = static_cast<int>(static_cast<long long>(w.n_kv) * (split + 1) / w.n_split);
  const int n = kv1 - kv0;
  const bool two = !ONE && w.nrow > 128;
  constexpr int LAG = ONE ? 2 : 1;
  uint32_t* err = p.err;

  // Registers: 128 a thread at launch; 176 + 176 + 80 + 80 = 4 * 128.
  if (warp >= 8) {
    regs_dec<80>();
    if (warp != 12) {
      const int tid = threadIdx.x - 256 - (warp > 12 ? 32 : 0);
      produce<D, LAG>(p, w, kv0, n, tid, smem_u32(sKV), kv_full, kv_empty, abort_flag, err);
    } else if (elect_one()) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t kIdescS = idesc_f16(128, 128, 0);
      constexpr uint32_t kIdescO = idesc_f16(128, D, 1);
      const uint32_t sQa = smem_u32(sQ), sPa = smem_u32(sP), sKVa = smem_u32(sKV);
      uint32_t n_kvc = 0, n_s[2] = {0, 0}, n_pv[2] = {0, 0};
      bool ok = true;

      auto s_mma = [&](int t, uint32_t ka) -> bool {
        if (n_s[t] > 0 && !mbar_wait(s_free + t, (n_s[t] - 1) & 1, abort_flag, err)) return false;
        if (n_s[t] == 0 && !mbar_wait(q_full + t, 0, abort_flag, err)) return false;
        tc_fence_after();
        const uint32_t qa = sQa + t * C::Q_BYTES;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::BLK + (kk & 3) * 32;
          mma_bf16_ss(tmem + C::TMEM_S + t * 128, smem_desc(qa + off, 16, 1024), smem_desc(ka + off, 16, 1024), kIdescS,
                      kk > 0 ? 1u : 0u);
        }
        mma_commit(s_full + t);
        ++n_s[t];
        return true;
      };
      auto pv_mma = [&](int t, uint32_t va, bool first) -> bool {
        if (!mbar_wait(p_full + t, n_pv[t] & 1, abort_flag, err)) return false;
        tc_fence_after();
        const uint32_t pa = sPa + t * C::P_BYTES;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t ad = smem_desc(pa + (kk >> 2) * C::BLK + (kk & 3) * 32, 16, 1024);
          const uint64_t bd = smem_desc(va + kk * 2048, C::BLK, 1024);
          mma_bf16_ss(tmem + C::TMEM_O + t * D, ad, bd, kIdescO, (!first || kk > 0) ? 1u : 0u);
        }
        mma_commit(o_done + t);
        ++n_pv[t];
        return true;
      };
      auto kv_ready = [&](uint32_t li, uint32_t& addr) -> bool {
        const int stage = static_cast<int>(li % C::NST);
        if (!mbar_wait(kv_full + stage, (li / C::NST) & 1, abort_flag, err)) return false;
        tc_fence_after();
        addr = sKVa + stage * C::KV_BYTES;
        return true;
      };
      auto kv_release = [&](uint32_t li) { mma_commit(kv_empty + static_cast<int>(li % C::NST)); };

      // Blocks are fetched into L2 ahead of their use, each by one of the CTAs that share them.
      const size_t first = kv8_tile(p.c, w.b, 0, w.h) * (kKv8Block * D);
      const size_t step = static_cast<size_t>(p.c.kv_heads) * (kKv8Block * D);
      auto prefetch = [&](int j) {
        for (int block = (kv0 + j) * 2; block < (kv0 + j) * 2 + 2 && block * kKv8Block < w.len; ++block) {
          prefetch_l2(p.c.k8 + first + block * step, kKv8Block * D);
          prefetch_l2(p.c.v8 + first + block * step, kKv8Block * D);
        }
      };
      int mine = ((w.row0 / 256 - kv0) % p.row_blocks + p.row_blocks) % p.row_blocks;  // the next tile that is this CTA's
      for (; mine < min(n, kPrefetchTiles); mine += p.row_blocks) prefetch(mine);
      uint32_t ka = 0, va = 0;
      for (int j = 0; j < n && ok; ++j) {
        if (j + kPrefetchTiles == mine) {
          if (mine < n) prefetch(mine);
          mine += p.row_blocks;
        }
        if constexpr (ONE) {
          // tile j's scores go to group j mod 2 while it still makes probabilities of tile j - 2's
          if (!(ok = kv_ready(n_kvc, ka) && s_mma(j & 1, ka))) break;
          kv_release(n_kvc++);
          if (j >= 2) {
            if (!(ok = kv_ready(n_kvc, va) && pv_mma(j & 1, va, j < 4))) break;
            kv_release(n_kvc++);
          }
        } else {
          const uint32_t ek = n_kvc;  // K_j; V_{j-1} follows it in the ring
          if (!(ok = kv_ready(ek, ka) && s_mma(0, ka))) break;
          if (j >= 1 && !(ok = kv_ready(ek + 1, va) && pv_mma(0, va, j == 1))) break;
          if (two && !(ok = s_mma(1, ka))) break;
          kv_release(ek);
          if (j >= 1) {
            if (two && !(ok = pv_mma(1, va, j == 1))) break;
            kv_release(ek + 1);
          }
          n_kvc += (j >= 1) ? 2 : 1;
        }
      }
      if constexpr (ONE) {
        for (int j = max(0, n - 2); j < n && ok; ++j, ++n_kvc) ok = kv_ready(n_kvc, va) && pv_mma(j & 1, va, j < 2);
      } else if (ok && n > 0) {
        ok = kv_ready(n_kvc, va) && pv_mma(0, va, n == 1);
        if (ok && two) ok = pv_mma(1, va, n == 1);
      }
      mma_commit(fin);
      mbar_wait(fin, 0, abort_flag, err);
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    regs_inc<176>();
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;
    // ONE: the groups have the same rows, and every other key tile each
    constexpr int STEP = ONE ? 2 : 1;
    const int tile_row = ONE ? 0 : t * 128, lrow = tile_row + r;
    const int row = w.row0 + lrow;
    const bool live = lrow < w.nrow;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::TMEM_S + t * 128;
    const uint32_t tO = tmem + lane_off + C::TMEM_O + t * D;
    const uint32_t in_tile = (r >> 3) * 1024 + (r & 7) * 128;
    const uint32_t p_row = smem_u32(sP + t * C::P_BYTES) + in_tile;
    const int seen = live ? min(w.len, seen_by(w, p.causal, p.group, row)) : 0;
    float m_run = -CUDART_INF_F, l_run = 0.f;
    float unit_e = kNoUnit;  // R
    bool ok = true;
    if (ONE || t == 0 || two) {
      // ---- the row's query, scaled into f16.  A warp brings its 32 rows into their
      // places as they are, whole rows at a time (a thread that loads its own row moves
      // half sectors: 3 us more), then each thread rewrites its row there.
      constexpr int CPR = D / 8;                       // 16-byte chunks per row
      const int lane = threadIdx.x & 31;
      const uint32_t q_tile = smem_u32(sQ + t * C::Q_BYTES), p_tile = smem_u32(sP + t * C::P_BYTES);
      auto chunk_at = [&](int i, int c) {  // chunk c of the warp's row i in a tile of column blocks
        return (c >> 3) * C::BLK + (warp & 3) * 4096 + i * 128 + (((c & 7) ^ (i & 7)) << 4);
      };
      float factor;
      {
        const int c = lane % CPR;
        RowWalk walk(p, w, w.row0 + tile_row + (warp & 3) * 32 + lane / CPR, 32 / CPR);
#pragma unroll
        for (int k = 0; k < CPR; ++k) {
          const int i = k * (32 / CPR) + lane / CPR;
          const bool in = tile_row + (warp & 3) * 32 + i < w.nrow;
          cp_async16(q_tile + chunk_at(i, c), static_cast<const uint4*>(p.q) + (in ? walk.at : 0) * CPR + c, in ? 16 : 0);
          walk.next();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        uint4 x[CPR];
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
          x[i] = ld_shared_v4(q_tile + chunk_at(lane, i));
          const uint32_t m = 0x7fff7fffu;
          amax = __vmaxu2(__vmaxu2(amax, __vmaxu2(x[i].x & m, x[i].y & m)), __vmaxu2(x[i].z & m, x[i].w & m));
        }
        amax = max(amax >> 16, amax & 0xffffu);
        if (amax >= 0x7f80u) {  // only finite values scale a row
          amax = 0;
#pragma unroll
          for (int i = 0; i < CPR; ++i)
            amax = max(amax, max(max(bf16x2_finite_max(x[i].x), bf16x2_finite_max(x[i].y)),
                                 max(bf16x2_finite_max(x[i].z), bf16x2_finite_max(x[i].w))));
        }
        const int k = clampi(static_cast<int>(amax >> 7) - 127, -100, 127);
        const float up = pow2i(14 - k);
        factor = pow2i(k - 14) * p.scale_log2;
#pragma unroll
        for (int i = 0; i < CPR; ++i)
          st_shared_v4(q_tile + chunk_at(lane, i),
                       pack_f16x2(bf16_lo(x[i].x) * up, bf16_hi(x[i].x) * up),
                       pack_f16x2(bf16_lo(x[i].y) * up, bf16_hi(x[i].y) * up),
                       pack_f16x2(bf16_lo(x[i].z) * up, bf16_hi(x[i].z) * up),
                       pack_f16x2(bf16_lo(x[i].w) * up, bf16_hi(x[i].w) * up));
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full + t);

      // Scales of 16 tiles at a time: lane l holds those of block l (blocks past the keys: any valid one does).
      float ks = 0.f, vs = 0.f;
      const int last_block = (w.n_keys - 1) / kKv8Block;
      const int j0 = ONE ? t : 0;
      for (int j = j0; j < n; j += STEP) {
        if ((j & 15) < STEP) {
          const size_t tile = kv8_tile(p.c, w.b, min(2 * (kv0 + (j & ~15)) + lane, last_block), w.h);
          ks = __ldcg(p.c.ks + tile);
          vs = __ldcg(p.c.vs + tile);
        }
        const int at = 2 * (j & 15);
        // the factor of a score must not underflow to 0: 0 * -inf has no value
        float f0 = fmaxf(factor * __shfl_sync(0xffffffffu, ks, at), 1.2e-38f);
        float f1 = fmaxf(factor * __shfl_sync(0xffffffffu, ks, at + 1), 1.2e-38f);
        const float ev0 = static_cast<float>(exponent_of(__shfl_sync(0xffffffffu, vs, at)));
        const float ev1 = static_cast<float>(exponent_of(__shfl_sync(0xffffffffu, vs, at + 1)));

        if (!(ok = mbar_wait(s_full + t, (j / STEP) & 1, abort_flag, err))) break;
        tc_fence_after();
        float s[128];
        tmem_ld32(tS + 0, s);
        tmem_ld32(tS + 32, s + 32);
        tmem_ld32(tS + 64, s + 64);
        tmem_ld32(tS + 96, s + 96);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(s_free + t);
        const int valid = seen - (kv0 + j) * 128;
        if (valid < 128) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= valid) s[c] = -CUDART_INF_F;
        }
        float mk[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mk[k] = fmaxf(s[(k >> 2) * 64 + (k & 3)], s[(k >> 2) * 64 + 4 + (k & 3)]);
#pragma unroll
        for (int c = 8; c < 64; c += 8)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mk[k] = max3f(mk[k], s[(k >> 2) * 64 + c + (k & 3)], s[(k >> 2) * 64 + c + 4 + (k & 3)]);
        const float top0 = fmaxf(max3f(mk[0], mk[1], mk[2]), mk[3]) * f0;
        const float top1 = fmaxf(max3f(mk[4], mk[5], mk[6]), mk[7]) * f1;
        const float m_new = fmaxf(top0, top1);
        float alpha = 1.0f;
        if (m_new > m_run + 4.0f) {
          alpha = ex2_approx(m_run - m_new);
          unit_e += m_run - m_new;
          m_run = m_new;
        }
        float m_at = m_run == -CUDART_INF_F ? 0.f : m_run;
        // the largest contribution of the tile: -infinity where the row sees nothing of it
        const float most = fmaxf(ev0 + fminf(top0 - m_at, 0.f), ev1 + fminf(top1 - m_at, 0.f));
        float scale_o = 1.0f;
        if (most > unit_e + kMaxDrift) {
          scale_o = ex2_approx(unit_e - most);
          unit_e = most;
        }
        // Offsets of the exponents.  Below -30 all of the half's probabilities are 0 in f16, and the sum
        // keeps its precision.
        float c0 = fmaxf(kOff + ev0 - unit_e, -30.f), c1 = fmaxf(kOff + ev1 - unit_e, -30.f);
        // The fused product of a score leaves the rounding of the maximum in the exponent, half a unit in its last
        // place, which past 2^27 would overflow f16.  From 2^24 on, where that unit is a factor of 2 and more and the
        // scores' own errors are larger still, distances count as if the maximum were below 2^24: the largest
        // scores keep all the weight, and everything stays finite.
        if (fabsf(m_at) > 16777216.f) {
          const float less = pow2i(23 - exponent_of(m_at));
          f0 = fmaxf(f0 * less, 1.2e-38f);
          f1 = fmaxf(f1 * less, 1.2e-38f);
          m_at *= less;
          c0 = fminf(c0, kOff + kMaxDrift);
          c1 = fminf(c1, kOff + kMaxDrift);
        }
        uint32_t pk[64];
        float sums[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float f = half ? f1 : f0;
          const float add = (half ? c1 : c0) - m_at;
          float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float a0, a1;
            fma2(a0, a1, s[half * 64 + c], s[half * 64 + c + 1], f, add);
            const float p0 = ex2_approx(a0);
            const float p1 = ex2_approx(a1);
            const int k = (c >> 1) & 3;
            add2(acc[2 * k], acc[2 * k + 1], p0, p1);
            pk[half * 32 + (c >> 1)] = pack_f16x2(p0, p1);
          }
          sums[half] = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
        }
        l_run = __fmaf_rn(l_run, alpha, __fmaf_rn(sums[0], ex2_approx(-c0), sums[1] * ex2_approx(-c1)));
        if (j >= STEP) {
          if (!(ok = mbar_wait(o_done + t, (j / STEP - 1) & 1, abort_flag, err))) break;
          tc_fence_after();
          if (__any_sync(0xffffffffu, scale_o != 1.0f)) {
#pragma unroll
            for (int cc = 0; cc < D; cc += 32) {
              float o[32];
              tmem_ld32(tO + cc, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= scale_o;
              tmem_st32(tO + cc, o);
            }
            tmem_wait_st();
          }
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint32_t addr = p_row + (c >> 3) * C::BLK + (((c & 7) ^ (r & 7)) << 4);
          st_shared_v4(addr, pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(p_full + t);
      }
      // ---- epilogue
      const int n_mine = ONE ? (n + 1 - t) / 2 : n;  // key tiles of this group
      if (ok && n_mine > 0) {
        ok = mbar_wait(o_done + t, (n_mine - 1) & 1, abort_flag, err);
        tc_fence_after();
      }
      float unit = ex2_approx(unit_e - kOff) * inverse_sum(l_run);  // of an output divided by its sum
      // ONE: the second group hands its maxima, sums and outputs to the first through the
      // ring, once no product reads it any more.  Both come to the barrier whatever happened.
      float other_f = 0.f;
      const uint32_t other = smem_u32(sKV) + r * 16;
      if constexpr (ONE) {
        float2* ml = reinterpret_cast<float2*>(sKV + 128 * D * 4);
        if (t == 1) {
          ok = ok && mbar_wait(fin, 0, abort_flag, err);
          if (ok) {
            ml[r] = make_float2(m_run, l_run);
            if (n_mine > 0) {
#pragma unroll
              for (int cc = 0; cc < D; cc += 32) {
                float o[32];
                tmem_ld32(tO + cc, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  st_shared_f4(other + (cc / 4 + i) * 2048, o[4 * i] * unit, o[4 * i + 1] * unit, o[4 * i + 2] * unit,
                               o[4 * i + 3] * unit);
              }
            }
          }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (t == 1) {
          ok = false;  // the first group has the rest
        } else if (n > 1) {
          const float2 x = ml[r];
          const float top = fmaxf(m_run, x.x), at_m = top == -CUDART_INF_F ? 0.f : top;
          const float mine = l_run * ex2_approx(m_run - at_m), theirs = x.y * ex2_approx(x.x - at_m);
          m_run = top;
          l_run = mine + theirs;
          unit *= mine * inverse_sum(l_run);
          other_f = theirs * inverse_sum(l_run);
        }
      }
      // 32 features of the row's output
      auto load_o = [&](int cc, float (&o)[32]) {
        tmem_ld32(tO + cc, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= unit;
        if constexpr (ONE) {
          if (n > 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 x = ld_shared_f4(other + (cc / 4 + i) * 2048);
              o[4 * i] = __fmaf_rn(x.x, other_f, o[4 * i]);
              o[4 * i + 1] = __fmaf_rn(x.y, other_f, o[4 * i + 1]);
              o[4 * i + 2] = __fmaf_rn(x.z, other_f, o[4 * i + 2]);
              o[4 * i + 3] = __fmaf_rn(x.w, other_f, o[4 * i + 3]);
            }
          }
        }
      };
      if (ok) {
        if (whole) {
          // rows as bf16 into the warp's part of P's tile, then out whole rows at a time
          const bool any = seen > 0;
#pragma unroll
          for (int cc = 0; cc < D; cc += 32) {
            float o[32];
            if (n > 0) load_o(cc, o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // a row that sees nothing gives zeros, whatever its sums are
              const uint32_t keep = any ? 0xffffffffu : 0u;
              st_shared_v4(p_tile + chunk_at(lane, cc / 8 + i), pack_bf16x2(o[8 * i], o[8 * i + 1]) & keep,
                           pack_bf16x2(o[8 * i + 2], o[8 * i + 3]) & keep,
                           pack_bf16x2(o[8 * i + 4], o[8 * i + 5]) & keep,
                           pack_bf16x2(o[8 * i + 6], o[8 * i + 7]) & keep);
            }
          }
          __syncwarp();
          const int c = lane % CPR;
          RowWalk walk(p, w, w.row0 + tile_row + (warp & 3) * 32 + lane / CPR, 32 / CPR);
#pragma unroll 4
          for (int k = 0; k < CPR; ++k) {
            const int i = k * (32 / CPR) + lane / CPR;
            if (tile_row + (warp & 3) * 32 + i < w.nrow)
              static_cast<uint4*>(p.out)[walk.at * CPR + c] = ld_shared_v4(p_tile + chunk_at(i, c));
            walk.next();
          }
          if (live) {
            const size_t at = query_at(p, w, row);
            const float lse2 = m_run + log2f(l_run);
            if (p.lse) p.lse[at] = any ? lse2 * CUDART_LN2_F : -CUDART_INF_F;
            if (p.lse2) p.lse2[at] = any ? lse2 : CUDART_INF_F;
          }
        } else {
          // partials lie [4 features][row]: a warp's rows side by side
          const size_t cut = piece - p.n_whole;
          float4* dst = reinterpret_cast<float4*>(p.part_o) + cut * (256 * D / 4) + lrow;
#pragma unroll
          for (int cc = 0; cc < D; cc += 32) {
            float o[32];
            if (n > 0) load_o(cc, o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[(cc / 4 + i) * 256] = n > 0 ? make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3])
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          reinterpret_cast<float2*>(p.part_ml)[cut * 256 + lrow] = make_float2(m_run, l_run);
        }
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

// Merge of the key ranges of the split units: a lane has G groups of 4 features of
// a row (eight lanes' rows side by side, as the partials lie), FLY ranges in
// flight.  Reads of the partials bound it: G = D / 16 with FLY = 2 where units
// are many, G = 1 with FLY = 8 where they are few.  Measured, the first form and
// the second: 84 units of 5 ranges at d 128 11.5 and 16 us, 24 of 6 ranges 8.5 and
// 7, 4 units of 36 ranges at d 64 61 and 8.
constexpr int kMergeWarps = 4;
constexpr int kMergeRows = 8 * kMergeWarps;
constexpr int kFewUnits = 48;

template <int D, int G, int FLY>
__global__ void __launch_bounds__(32 * kMergeWarps) kv8_chunk_merge_kernel(const __grid_constant__ Kv8ChunkParams p) {
  const int lane = threadIdx.x & 31;
  const int group = blockIdx.z * (4 * G) + (lane >> 3);  // of 4 features, and 4, 8, .. from it
  grid_wait();
  const int ru = blockIdx.x;
  const Work w = work_of(p, p.n_whole + ru, p.splits);
  const int lrow = blockIdx.y * kMergeRows + (threadIdx.x >> 5) * 8 + (lane & 7);
  if (lrow >= w.nrow) return;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + static_cast<size_t>(ru) * p.splits * 256 + lrow;
  const float4* part = reinterpret_cast<const float4*>(p.part_o) + static_cast<size_t>(ru) * p.splits * (256 * D / 4) +
                       group * 256 + lrow;
  float mx = -CUDART_INF_F, sum = 0.f;
  float4 acc[G];
#pragma unroll
  for (int i = 0; i < G; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < w.n_split; k0 += FLY) {
    float2 x[FLY];
    float4 o[FLY][G];
#pragma unroll
    for (int k = 0; k < FLY; ++k) {
      x[k] = make_float2(-CUDART_INF_F, 0.f);
#pragma unroll
      for (int i = 0; i < G; ++i) o[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + k < w.n_split) {
        x[k] = __ldcg(ml + (k0 + k) * 256);
#pragma unroll
        for (int i = 0; i < G; ++i) o[k][i] = __ldcg(part + static_cast<size_t>(k0 + k) * (256 * D / 4) + i * 1024);
      }
    }
    float top = mx;
#pragma unroll
    for (int k = 0; k < FLY; ++k) top = fmaxf(top, x[k].x);
    const float at_m = top == -CUDART_INF_F ? 0.f : top;
    const float before = sum * exp2f(mx - at_m);
    sum = before;
#pragma unroll
    for (int k = 0; k < FLY; ++k) {
      x[k].y *= exp2f(x[k].x - at_m);
      sum += x[k].y;
    }
    const float inv = inverse_sum(sum), f0 = before * inv;
#pragma unroll
    for (int i = 0; i < G; ++i) acc[i] = make_float4(acc[i].x * f0, acc[i].y * f0, acc[i].z * f0, acc[i].w * f0);
#pragma unroll
    for (int k = 0; k < FLY; ++k) {
      const float f = x[k].y * inv;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        acc[i].x = __fmaf_rn(o[k][i].x, f, acc[i].x);
        acc[i].y = __fmaf_rn(o[k][i].y, f, acc[i].y);
        acc[i].z = __fmaf_rn(o[k][i].z, f, acc[i].z);
        acc[i].w = __fmaf_rn(o[k][i].w, f, acc[i].w);
      }
    }
    mx = top;
  }
  const int row = w.row0 + lrow;
  const bool any = seen_by(w, p.causal, p.group, row) > 0 && w.len > 0;
  const size_t at = query_at(p, w, row);
  uint2* dst = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at * D) + group;
#pragma unroll
  for (int i = 0; i < G; ++i)
    dst[4 * i] = any ? make_uint2(pack_bf16x2(acc[i].x, acc[i].y), pack_bf16x2(acc[i].z, acc[i].w))
                     : make_uint2(0u, 0u);
  if (group == 0) {
    const float lse2 = mx + log2f(sum);
    if (p.lse) p.lse[at] = any ? lse2 * CUDART_LN2_F : -CUDART_INF_F;
    if (p.lse2) p.lse2[at] = any ? lse2 : CUDART_INF_F;
  }
}

}  // namespace

namespace {
template <int D>
cudaError_t configure_chunk() {
  const cudaError_t e =
      cudaFuncSetAttribute(kv8_chunk_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkCfg<D>::SMEM);
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(kv8_chunk_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 ChunkCfg<D>::SMEM);
}

template <int D>
cudaError_t launch_chunk(const Kv8ChunkParams& p, cudaStream_t s) {
  const int rest = p.units - p.n_whole;
  const dim3 grid(p.n_whole + rest * p.splits), mgrid(rest, 256 / kMergeRows, rest <= kFewUnits ? D / 16 : 1);
  const bool one = static_cast<long long>(p.n) * p.group <= kKv8OneTile;
  const cudaError_t e = launch_kernel(one ? kv8_chunk_kernel<D, true> : kv8_chunk_kernel<D, false>, grid, kThreads,
                                      ChunkCfg<D>::SMEM, s, 1, p);
  if (e != cudaSuccess || rest == 0) return e;
  return launch_kernel(rest <= kFewUnits ? kv8_chunk_merge_kernel<D, 1, 8> : kv8_chunk_merge_kernel<D, D / 16, 2>, mgrid,
                       32 * kMergeWarps, 0, s, 1, p);
}
}  // namespace

cudaError_t kv8_chunk_configure(int head_dim) {
  return head_dim == 128 ? configure_chunk<128>() : configure_chunk<64>();
}

cudaError_t launch_kv8_chunk_attn(int head_dim, const Kv8ChunkParams& p, cudaStream_t s) {
  return head_dim == 128 ? launch_chunk<128>(p, s) : launch_chunk<64>(p, s);
}

}  // namespace ff
