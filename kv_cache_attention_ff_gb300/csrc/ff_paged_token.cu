// Attention of few query rows (at most 8 per kv head) over pages.
//
// For one (request, kv head) the query rows are the `group` heads of each of its
// new tokens (row r = token r / group, head r mod group): they read the same keys,
// so they share every loaded tile.
//
// Scores and outputs run on the m16n8k16 bf16 matrix instruction with fp32
// accumulation and the queries as its 8 columns (S^T = K Q^T, O^T = V^T P^T), so a
// single token does not pay for 16 rows.  (More columns are bound by this
// instruction's rate.)  Probabilities enter as two bf16 pieces, p = hi + lo with 16 bits
// between them, so that the output's only rounding to fewer bits is its own; the second
// product costs nothing beside the stream of keys.
//
// A block of 4 warps has one piece, a key range of one (request, kv head); the plan
// has listed the pieces.  The warps take stages of 16 keys in turn, each with a
// ring of its own that tensor copies of 16 rows fill (a page holds one to eight
// such boxes), its own reference and its own sums: no barrier until the piece
// ends.  The reference of a row's exponents (log2) is its running maximum plus 8 as it was
// when that was last passed, so that it seldom moves and no exponent is above 0.
// The warps' results merge in shared memory, the ranges' through partial results
// that the last range to finish merges in their order.
//
// The stream of keys and values bounds it: one row of 12 heads over 31200 rows (192 MB)
// 35 us, 5.5 TB/s, of which 6 us are launch, first loads and merge; 64 requests of up to
// 8190 rows with 32/8 heads (1.1 GB) 165 us, 6.7 TB/s; 208 rows of 2 heads 4.1 us.  Two
// blocks per SM with rings of three stages; three with two measured the same, one of six
// stages 42 us in place of 35.
#include <algorithm>

#include <cuda_bf16.h>
#include <math_constants.h>

#include "ff_paged.cuh"
#include "ff_ptx.cuh"

namespace ff {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kBlocksPerSm = 2;
constexpr int kKeys = kPagedStage;
constexpr int kRows = kPagedTokenRows;
static_assert(kRows == 8, "columns of the matrix instruction");
constexpr float kRise = 8.f;  // log2

template <int D>
struct TokenCfg {
  // A tile lies as two groups of eight keys, a group's blocks of 64 features one after the other, 128-byte swizzled lines
  // (1 KB each).
  static constexpr int KB = D / 64;
  static constexpr int TILE = 2 * KB * 1024;     // K or V of a stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int NST = D == 128 ? 3 : 6;
  static constexpr int RING = kWarps * NST * STAGE;
  static constexpr int OT = D / 16;              // 16-feature tiles of the output
  static constexpr int ORow = D + 4;             // floats of a row of the warps' results (4 apart in banks)
  static constexpr int MERGE = kWarps * kRows * (ORow + 2) * 4;  // which take the ring's place
  static constexpr int SMEM = RING + kWarps * NST * 8 + 1024;
  static_assert(MERGE <= RING, "the warps' results fit the ring");
  static_assert(kBlocksPerSm * (SMEM + 2048) <= 233472, "shared memory");
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements over the warp: thread 4 g + c
// holds elements 2c, 2c + 1 of row g before and of column g after.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <int D>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    paged_token_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                       const __grid_constant__ PagedTokenParams p) {
  using C = TokenCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::RING);
  __shared__ int is_last, abort_word;
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  uint64_t* full = bars + warp * C::NST;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWarps * C::NST; ++i) mbar_init(bars + i, 1);
    abort_word = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_wait();

  const int heads = p.kv_heads * p.group;
  const PagedPiece first = p.pieces[blockIdx.x / p.kv_heads];  // there or not: one load less in the chain to the keys
  const int blocks = *p.n_pieces * p.kv_heads;
  uint8_t* ring = smem + warp * (C::NST * C::STAGE);
  uint32_t done = 0;  // stages that this warp has been through
  for (int block = blockIdx.x; block < blocks; block += gridDim.x) {
    const int h = block % p.kv_heads;
    const PagedPiece pc = block == blockIdx.x ? first : p.pieces[block / p.kv_heads];
    const int nrow = clampi(p.n - pc.first, 0, pc.count) * p.group;
    if (pc.count > p.most || nrow == 0) continue;
    const int nst = (pc.length + kKeys - 1) / kKeys;
    const int st0 = static_cast<int>(static_cast<long long>(nst) * pc.split / pc.n_split);
    const int st1 = static_cast<int>(static_cast<long long>(nst) * (pc.split + 1) / pc.n_split);
    // nothing is loaded any more once a wait has run out
    const int n_mine = st1 - st0 > warp && !*abort_flag ? (st1 - st0 - warp + kWarps - 1) / kWarps : 0;

    // ---- keys and values: lane l has the page of the warp's stage l of 32
    const int* table = p.tables + static_cast<size_t>(pc.request) * p.width;
    auto pages_from = [&](int i) {
      const int st = st0 + warp + (i + lane) * kWarps;
      return i + lane < n_mine ? clampi(__ldcg(table + ((st * kKeys) >> p.shift)), 0, p.pages - 1) : 0;
    };
    int pages = pages_from(0), pages_next = pages_from(32);
    auto issue = [&](int i) {
      if (i >= n_mine) return;
      if (i > 0 && (i & 31) == 0) {
        pages = pages_next;
        pages_next = pages_from(i + 32);
      }
      const int page = __shfl_sync(0xffffffffu, pages, i & 31);
      if (lane == 0) {
        const int key = (st0 + warp + i * kWarps) * kKeys;
        const int group = ((page * p.kv_heads + h) << (p.shift - 3)) + ((key & ((1 << p.shift) - 1)) >> 3);
        const uint32_t slot = (done + i) % C::NST;
        uint8_t* to = ring + slot * C::STAGE;
        mbar_expect_tx(full + slot, C::STAGE);
        tma_load_4d(to, &tk, group, full + slot);
        tma_load_4d(to + C::TILE, &tv, group, full + slot);
      }
    };
#pragma unroll
    for (int i = 0; i < C::NST - 1; ++i) issue(i);

    // ---- queries as a B fragment: features 16 k + 2 c, + 1 and 8 more of row g
    uint32_t qf[C::OT][2];
    {
      const uint32_t* q = static_cast<const uint32_t*>(p.q) +
                          (static_cast<size_t>(pc.first + g / p.group) * heads + h * p.group + g % p.group) * (D / 2) + c;
#pragma unroll
      for (int k = 0; k < C::OT; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) qf[k][i] = g < nrow ? __ldcg(q + k * 8 + i * 4) : 0u;
    }
    // rows 2 c and + 1 are this thread's columns; row r sees keys below seen
    float o[C::OT][4], ref[2], sum[2];
    int seen[2];
#pragma unroll
    for (int i = 0; i < C::OT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 2 * c + j;
      ref[j] = -CUDART_INF_F;
      sum[j] = 0.f;
      seen[j] = r < nrow ? pc.length - pc.count + r / p.group + 1 : 0;
    }
    const int seen_min = pc.length - pc.count + 1;  // the first row sees least

    int it = 0;
    for (; it < n_mine; ++it) {
      issue(it + C::NST - 1);  // into the slot that the warp finished with one stage ago
      const uint32_t slot = (done + it) % C::NST;
      if (!mbar_wait(full + slot, ((done + it) / C::NST) & 1, abort_flag, p.err)) break;
      const int key0 = (st0 + warp + it * kWarps) * kKeys;
      uint8_t* tile = ring + slot * C::STAGE;
      const uint32_t k_a = smem_u32(tile), v_a = k_a + C::TILE;
      if (key0 + kKeys > pc.length) {
        // rows past the last may hold NaN, which a probability of 0 would not hide
        const int held = pc.length - key0;
        for (int i = lane; i < (kKeys - held) * 8 * C::KB; i += 32) {
          const int row = held + i / (8 * C::KB), kb = i / 8 % C::KB;
          st_shared_v4(v_a + ((row >> 3) * C::KB + kb) * 1024 + (row & 7) * 128 + (i & 7) * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }

      // ---- scores: keys g and g + 8, rows 2 c and + 1
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < C::OT; ++k) {
        uint32_t a[4];
        const int r = lane & 15, ch = (k & 3) * 2 + (lane >> 4);
        ldmatrix4(a, k_a + ((r >> 3) * C::KB + (k >> 2)) * 1024 + (r & 7) * 128 + ((ch ^ (r & 7)) << 4));
        mma_bf16(s, a, qf[k][0], qf[k][1]);
      }

      // ---- softmax
      const bool all = key0 + kKeys <= seen_min;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s[k] *= p.scale_log2;
        if (!all && key0 + (k >> 1) * 8 + g >= seen[k & 1]) s[k] = -CUDART_INF_F;
      }
      if (__any_sync(0xffffffffu, fmaxf(s[0], s[2]) > ref[0] || fmaxf(s[1], s[3]) > ref[1])) {
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float top = fmaxf(s[j], s[2 + j]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          f[j] = 1.f;
          if (top > ref[j]) {
            f[j] = ex2_approx(ref[j] - (top + kRise));
            ref[j] = top + kRise;
          }
          sum[j] *= f[j];
        }
#pragma unroll
        for (int i = 0; i < C::OT; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][k] *= f[k & 1];
      }
      uint32_t hi[2], lo[2];  // P^T as B fragments: keys 2 c, + 1 (and 8 more), row g
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float at = ref[k & 1] == -CUDART_INF_F ? 0.f : ref[k & 1];
        s[k] = ex2_approx(s[k] - at);
        sum[k & 1] += s[k];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t x = pack_bf16x2(s[2 * k], s[2 * k + 1]);
        hi[k] = transpose8x8(x);
        lo[k] = transpose8x8(pack_bf16x2(s[2 * k] - bf16_lo(x), s[2 * k + 1] - bf16_hi(x)));
      }

      // ---- output: features 16 i + g and + 8, rows 2 c and + 1
#pragma unroll
      for (int i = 0; i < C::OT; ++i) {
        uint32_t a[4];
        const int r = (lane & 7) + ((lane >> 4) << 3), ch = (i & 3) * 2 + ((lane >> 3) & 1);
        ldmatrix4_trans(a, v_a + ((r >> 3) * C::KB + (i >> 2)) * 1024 + (r & 7) * 128 + ((ch ^ (r & 7)) << 4));
        mma_bf16(o[i], a, hi[0], hi[1]);
        mma_bf16(o[i], a, lo[0], lo[1]);
      }
      __syncwarp();  // the slot is free
    }
    // a wait that ran out: the copies in flight come to their end first, for at most a second
    volatile int no = 0;
    for (int i = it; i < min(n_mine, it + C::NST); ++i)
      mbar_wait(full + (done + i) % C::NST, ((done + i) / C::NST) & 1, &no, p.err, 1000000000ull);
    done += n_mine;

    // ---- merge the warps: output, reference and sum of each row
    __syncthreads();
    float* so = reinterpret_cast<float*>(smem);                           // [warps][kRows][ORow]
    float2* sml = reinterpret_cast<float2*>(so + kWarps * kRows * C::ORow);  // [warps][kRows]
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 2 * c + j;
      float x = sum[j];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      if (g == 0) sml[warp * kRows + r] = make_float2(ref[j], x);
      if (r < nrow) {
        float* to = so + (warp * kRows + r) * C::ORow + g;
#pragma unroll
        for (int i = 0; i < C::OT; ++i) {
          to[16 * i] = o[i][j];
          to[16 * i + 8] = o[i][2 + j];
        }
      }
    }
    __syncthreads();

    // From here on a warp has a row, a lane PER of its features.
    constexpr int PER = D / 32;
    struct Merged {
      float ref, sum, acc[PER];
    };
    static_assert(kWarps == 4, "the warps merge at once");
    // Row r of the first `parts` of four results in shared memory, relative to the largest reference.
    auto merged = [&](int r, int parts) {
      Merged x;
      float2 ml[4];
      x.ref = -CUDART_INF_F;
      x.sum = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        ml[w] = w < parts ? sml[w * kRows + r] : make_float2(-CUDART_INF_F, 0.f);
        x.ref = fmaxf(x.ref, ml[w].x);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) x.acc[i] = 0.f;
      const float at = x.ref == -CUDART_INF_F ? 0.f : x.ref;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = ex2_approx(ml[w].x - at);
        x.sum = __fmaf_rn(ml[w].y, f, x.sum);
        if (w < parts)
#pragma unroll
          for (int i = 0; i < PER; ++i) x.acc[i] = __fmaf_rn(so[(w * kRows + r) * C::ORow + i * 32 + lane], f, x.acc[i]);
      }
      return x;
    };
    auto finish = [&](int r, const Merged& x) {
      const size_t at = static_cast<size_t>(pc.first + r / p.group) * heads + h * p.group + r % p.group;
      const float inv = 1.f / x.sum;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        static_cast<__nv_bfloat16*>(p.out)[at * D + i * 32 + lane] = __float2bfloat16(x.acc[i] * inv);
      if (lane == 0 && p.lse) p.lse[at] = (x.ref + log2f(x.sum)) * CUDART_LN2_F;
    };
    const size_t part = static_cast<size_t>(pc.part) * p.kv_heads + h;  // the first range's; the next is kv_heads on
    for (int r = warp; r < nrow; r += kWarps) {
      const Merged x = merged(r, kWarps);
      if (pc.n_split == 1) {
        finish(r, x);
      } else {
        const size_t row = (part + static_cast<size_t>(pc.split) * p.kv_heads) * kRows + r;
#pragma unroll
        for (int i = 0; i < PER; ++i) p.part_o[row * D + i * 32 + lane] = x.acc[i];
        if (lane == 0) reinterpret_cast<float2*>(p.part_ml)[row] = make_float2(x.ref, x.sum);
      }
    }
    if (pc.n_split > 1) {
      // ---- the last range of the (request, kv head) to finish merges them all
      __syncthreads();
      if (threadIdx.x == 0) {
        unsigned* ticket = p.tickets + static_cast<size_t>(pc.request) * p.kv_heads + h;
        unsigned before;
        // releases the block's partial results (ordered before by the barrier) and acquires the others'
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(ticket) : "memory");
        is_last = before == static_cast<unsigned>(pc.n_split - 1);
        if (is_last) *ticket = 0;
      }
      __syncthreads();
      if (is_last) {
        // the warps share rows, or with fewer than four rows each row's ranges
        const int row_warps = nrow >= 4 ? 4 : nrow >= 2 ? 2 : 1, range_warps = 4 / row_warps;
        const int mine = warp / row_warps;  // of each row's ranges: mine, mine + range_warps, ..
        for (int r = warp % row_warps; r < nrow; r += row_warps) {
          Merged x;
          x.ref = -CUDART_INF_F;
          x.sum = 0.f;
#pragma unroll
          for (int i = 0; i < PER; ++i) x.acc[i] = 0.f;
          constexpr int FLY = 16;  // ranges in flight
          for (int k0 = mine; k0 < pc.n_split; k0 += FLY * range_warps) {
            float2 ml[FLY];
            float v[FLY][PER];
#pragma unroll
            for (int k = 0; k < FLY; ++k) {
              const int range = k0 + k * range_warps;
              const size_t row = (part + static_cast<size_t>(range) * p.kv_heads) * kRows + r;
              const bool in = range < pc.n_split;
              ml[k] = in ? __ldcg(reinterpret_cast<const float2*>(p.part_ml) + row) : make_float2(-CUDART_INF_F, 0.f);
#pragma unroll
              for (int i = 0; i < PER; ++i) v[k][i] = in ? __ldcg(p.part_o + row * D + i * 32 + lane) : 0.f;
            }
            float top = x.ref;
#pragma unroll
            for (int k = 0; k < FLY; ++k) top = fmaxf(top, ml[k].x);
            const float at = top == -CUDART_INF_F ? 0.f : top;
            const float before = ex2_approx(x.ref - at);
            x.sum *= before;
#pragma unroll
            for (int i = 0; i < PER; ++i) x.acc[i] *= before;
#pragma unroll
            for (int k = 0; k < FLY; ++k) {
              const float f = ex2_approx(ml[k].x - at);
              x.sum = __fmaf_rn(ml[k].y, f, x.sum);
#pragma unroll
              for (int i = 0; i < PER; ++i) x.acc[i] = __fmaf_rn(v[k][i], f, x.acc[i]);
            }
            x.ref = top;
          }
          if (lane == 0) sml[mine * kRows + r] = make_float2(x.ref, x.sum);
#pragma unroll
          for (int i = 0; i < PER; ++i) so[(mine * kRows + r) * C::ORow + i * 32 + lane] = x.acc[i];
        }
        __syncthreads();
        for (int r = warp; r < nrow; r += kWarps) finish(r, merged(r, range_warps));
      }
    }
    fence_proxy_async_smem();  // the next piece's copies come where the results are
    __syncthreads();
  }
}

}  // namespace

cudaError_t paged_token_configure(int head_dim) {
  return head_dim == 128 ? cudaFuncSetAttribute(paged_token_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                TokenCfg<128>::SMEM)
                         : cudaFuncSetAttribute(paged_token_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                TokenCfg<64>::SMEM);
}

int paged_token_blocks(int sms) { return sms * kBlocksPerSm; }

cudaError_t launch_paged_token(int head_dim, const CUtensorMap& k, const CUtensorMap& v, const PagedTokenParams& p,
                               int requests, int token_blocks, cudaStream_t s) {
  // as many blocks as there can be pieces; a block takes another piece where that is more than fill the GPU 16 times.  One
  // token of 8 kv heads over 208 keys takes 4.6 us in a handle of up to 64 requests, 5.8 in one of 300, 7.6 in one of 2000.
  const long long pieces = static_cast<long long>(paged_piece_cap(token_blocks, p.kv_heads, requests)) * p.kv_heads;
  const int grid = static_cast<int>(std::min<long long>(pieces, 16ll * token_blocks));
  return head_dim == 128 ? launch_kernel(paged_token_kernel<128>, grid, kThreads, TokenCfg<128>::SMEM, s, 1, k, v, p)
                         : launch_kernel(paged_token_kernel<64>, grid, kThreads, TokenCfg<64>::SMEM, s, 1, k, v, p);
}

}  // namespace ff
