// Attention of few query rows (at most 32 per kv head) over the 8-bit cache, and
// the weight that every key received from them.
//
// For one (sequence, kv head) the query rows are the `group` heads of each of
// its tokens (row r = token r / group, head r mod group): they read the same
// keys, so they share every loaded tile.
//
// Scores and outputs run on the m16n8k16 f16 matrix instruction with fp32
// accumulation and the queries as its 8 columns (S^T = K Q^T, O^T = V^T P^T): one
// to four column tiles, so a single token does not pay for 16 rows.  (The 8-bit
// instruction converts its operands to f16 each time it is issued: with three
// pieces for the bits of P it took twice the instructions.)
//   * a code becomes f16 exactly (one conversion for two codes), so the block
//     scales stay out of the operands: K's multiplies the scores, V's enters
//     as an exponent of the probabilities;
//   * a query row is scaled by a power of two to put its largest magnitude
//     into [2^14, 2^15): exact in f16 for every value above 2^-29 of it;
//   * probabilities go to f16 relative to the running row maximum (11 bits
//     against bf16's 8; the maximum m only rises by more than 2^4), times
//     2^(kPOff + ev - R) where 2^ev is the V block's scale and 2^(m + R) the unit
//     in which the row's output accumulates.  The unit belongs to the row and is
//     the running maximum of probability times scale over the keys that it sees:
//     a large block that it does not see, or gives no weight, costs it nothing.
//     It rises by more than 2^2 at a time, and only that rescales the
//     accumulators (where m rises R falls as much).  f16 holds 11 bits of
//     what lies down to 2^-19 below the unit; anything is rounded by at
//     most 2^-30 of the unit times its code.
// Which feature a matrix slot means is free as long as Q and K agree: a thread
// takes 16 consecutive codes of a key.  V's codes are transposed by the load
// itself (ldmatrix, 8-bit), P in registers (movmatrix): the matrix slots of the
// keys are numbered in the order in which that leaves them.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>
#include <math_constants.h>

#include "ff_kv8.cuh"
#include "ff_ptx.cuh"

namespace ff {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStageKeys = 32;  // keys of one warp's stage
constexpr float kRise = 4.f;    // the running maximum only rises by more than this (log2)
constexpr float kPOff = 5.f;
constexpr float kNoUnit = -200.f;  // of a row that has seen nothing: below every scale's exponent
constexpr float kMaxDrift = 2.f;  // a contribution above the unit before that moves: 2^(4 + 5 + 2) stays below f16's 65504

// Thread blocks per SM: three, or two where 32 query rows need the registers.
constexpr int blocks_per_sm(int rows) { return rows > 16 ? 2 : 3; }

template <int D, int NQ>
struct TokenCfg {
  static constexpr int OT = D / 16;                        // 16-feature tiles of the output
  static constexpr int RT = 8 * NQ;                        // query rows
  static constexpr int TILE = kStageKeys * D;              // bytes of K or V of a stage
  static constexpr int STAGE = 2 * TILE + 128;             // and the two scales
  static constexpr int NST = 2;
  static constexpr int RING = kWarps * NST * STAGE;
  static constexpr int Q_BYTES = RT * D * 2;
  static constexpr int ORow = D + 4;                       // floats of a row of the warps' results (4 apart in banks)
  static constexpr int MERGE = kWarps * RT * (ORow + 2) * 4;  // which take the place of ring and queries
  static constexpr int BODY = RING + Q_BYTES > MERGE ? RING + Q_BYTES : MERGE;
  static constexpr int SMEM = BODY + RT * 8 + 128;         // and each row's factor and visible keys
  static_assert(blocks_per_sm(RT) * (SMEM + 2048) <= 233472, "shared memory");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void ldmatrix_trans8(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Transpose of an 8 x 8 matrix of 16-bit elements over the warp: thread 4 g + c
// holds elements 2c, 2c + 1 of row g before and of column g after.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A stage's tiles in shared memory: 128-byte lines (one row of 128 codes, or two
// of 64) of eight 16-byte chunks.  A chunk's place is xored with a number of
// its row that keeps each access apart in banks: copies write whole lines; a K
// load takes four chunks of two adjacent rows; a V load one chunk of the rows
// 0, 1, 8, 9, 2, 3, 10, 11 (then 4, 5, 12, ..), the order of P's keys.
template <int D>
__device__ __forceinline__ int k_at(int r, int ch) {
  if (D == 128) return r * 128 + ((ch ^ ((r & 6) ^ ((r & 1) << 2))) << 4);
  const int line = r >> 1;
  return line * 128 + ((((r & 1) << 2 | ch) ^ ((line & 1) | ((line >> 1) & 2))) << 4);
}
template <int D>
__device__ __forceinline__ int v_at(int r, int ch) {
  if (D == 128) return r * 128 + ((ch ^ ((r & 3) | ((r >> 1) & 4))) << 4);
  return k_at<D>(r, ch);
}

__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}

// Query rows 0 .. rows - 1 of a (sequence, kv head) into shared memory as B
// fragments of the matrix instruction (f16, scaled per row), with each row's
// factor (score = accumulator * factor * K scale, in log2 units).  The fragment
// of column tile t and step s holds, for lane 4 g + c, features
// 16 (c + 4 (s / 4)) + 4 (s mod 4) .. + 3 of row 8 t + g.  Rows past `valid` are
// zeros.
template <int D>
__device__ __forceinline__ void pack_queries(uint8_t* sq, float* factor, const void* q, size_t q_row0, int group,
                                             size_t token_stride, int rows, int valid, float scale_log2, int warp,
                                             int warps) {
  constexpr int W = D / 64;  // words of two features per lane
  constexpr int BATCH = 4;   // rows of a warp in flight
  const int lane = threadIdx.x & 31;
  for (int r0 = warp; r0 < rows; r0 += BATCH * warps) {
    uint32_t w[BATCH][W];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int r = r0 + k * warps;
#pragma unroll
      for (int i = 0; i < W; ++i) w[k][i] = 0;
      if (r < valid) {
        const uint32_t* src = static_cast<const uint32_t*>(q) +
                              (q_row0 + static_cast<size_t>(r / group) * token_stride + r % group) * (D / 2) + lane * W;
#pragma unroll
        for (int i = 0; i < W; ++i) w[k][i] = __ldcg(src + i);
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int r = r0 + k * warps;
      if (r >= rows) break;
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) amax = max(amax, bf16x2_finite_max(w[k][i]));
      amax = __reduce_max_sync(0xffffffffu, amax);
      const int e = clampi(static_cast<int>(amax >> 7) - 127, -100, 127);  // exponent of the largest magnitude
      const float up = pow2i(14 - e);
      const int f0 = lane * 2 * W;
      const int c = (f0 % 64) / 16, s = (f0 / 64) * 4 + (f0 % 16) / 4;
      uint32_t* dst = reinterpret_cast<uint32_t*>(sq) + (((r / 8) * (D / 16) + s) * 32 + (r % 8) * 4 + c) * 2 + (f0 % 4) / 2;
#pragma unroll
      for (int i = 0; i < W; ++i) dst[i] = pack_f16x2(bf16_lo(w[k][i]) * up, bf16_hi(w[k][i]) * up);
      if (lane == 0) factor[r] = pow2i(e - 14) * scale_log2;
    }
  }
}

// Scores of 32 keys against the packed queries: keys 16 u + g and + 8, queries
// 8 t + 2 c and + 1.  kw: this thread's 16-code chunks of rows 16 u + 8 k + g,
// features 16 (c + 4 half) ...
template <int D, int NQ>
__device__ __forceinline__ void scores(float (&s)[NQ][2][4], const uint4 (&kw)[D / 64][2][2], uint32_t sq_a) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int t = 0; t < NQ; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[t][u][k] = 0.f;
#pragma unroll
  for (int half = 0; half < D / 64; ++half)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint2 q[NQ];
#pragma unroll
      for (int t = 0; t < NQ; ++t) q[t] = lds64(sq_a + ((t * (D / 16) + half * 4 + k) * 32 + lane) * 8);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint4 x = kw[half][u][0], y = kw[half][u][1];
        const uint32_t lo = k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w;
        const uint32_t hi = k == 0 ? y.x : k == 1 ? y.y : k == 2 ? y.z : y.w;
        const uint32_t a[4] = {e4m3x2_to_f16x2(lo & 0xffffu), e4m3x2_to_f16x2(hi & 0xffffu), e4m3x2_to_f16x2(lo >> 16),
                               e4m3x2_to_f16x2(hi >> 16)};
#pragma unroll
        for (int t = 0; t < NQ; ++t) mma_f16(s[t][u], a, q[t].x, q[t].y);
      }
    }
}

// Rows of K seen by query row r.
__device__ __forceinline__ int seen_by(int r, int group, int causal, int len, int count) {
  return causal ? max(0, len - count + r / group + 1) : len;
}

// ------------------------------------------------------------ token attention
//
// Thread blocks of 4 warps, two or three per SM, so that one block's start and end pass
// under the others' streams.  A block takes one piece: a key range of one
// (sequence, kv head).  How many pieces a sequence's heads are cut into goes by
// its share of all keys, worked out by each block from the lengths on the device:
// unequal sequences keep the SMs equally long.  In a piece the warps take stages
// of 32 keys in turn, each with its own ring filled by asynchronous 16-byte
// copies and its own maximum, sum and output: no barrier until the piece ends.
// The warps' results merge in shared memory, the pieces' through partials that
// the last piece to finish merges in order (more than 8 rows: a launch of their own).
// One query row: the stream of keys and values bounds it.  12 heads over 31200 rows
// (96 MB) 21.5 us, 4.5 TB/s, of which 5 us are launch, first loads and merge (208 rows
// of 2 heads take that alone); 32 sequences of 8 kv heads, 4 rows each (286 MB) 54 us, 5.3
// TB/s.  From some 16 rows on the matrix instructions do: 25 rows (96 MB) 34 us.
// Equal runs of stages cut across heads and sequences, in place of pieces, measured
// 62 us for the batch and 68 for the 25 rows with their merge and weights (52).

// A row's mean over pieces (acc), each weighted by its sum times 2^(its maximum - the
// largest so far): a lane has D / 32 features; 16 pieces are in flight.
template <int D>
struct RowMerge {
  static constexpr int PER = D / 32;
  float mx, sum, acc[PER];

  __device__ __forceinline__ RowMerge() : mx(-HUGE_VALF), sum(0.f) {
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  }
  // Pieces k0, k0 + step, .. below n; piece k's row is row `row0 + k * tile_rows`.
  __device__ __forceinline__ void pieces(const float* part_o, const float* part_ml, size_t row0, int tile_rows, int k0,
                                         int n, int step) {
    const int lane = threadIdx.x & 31;
    for (; k0 < n; k0 += 16 * step) {
      float2 ml[16];
      float v[16][PER];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int piece = k0 + k * step;
        const size_t row = row0 + static_cast<size_t>(piece) * tile_rows;
        ml[k] = make_float2(-CUDART_INF_F, 0.f);
#pragma unroll
        for (int i = 0; i < PER; ++i) v[k][i] = 0.f;
        if (piece < n) {
          ml[k] = __ldcg(reinterpret_cast<const float2*>(part_ml) + row);
          if (PER == 4) {
            const float4 t = __ldcg(reinterpret_cast<const float4*>(part_o + row * D) + lane);
            v[k][0] = t.x;
            v[k][1] = t.y;
            v[k][PER - 2] = t.z;
            v[k][PER - 1] = t.w;
          } else {
            const float2 t = __ldcg(reinterpret_cast<const float2*>(part_o + row * D) + lane);
            v[k][0] = t.x;
            v[k][1] = t.y;
          }
        }
      }
      float top = mx;
#pragma unroll
      for (int k = 0; k < 16; ++k) top = fmaxf(top, ml[k].x);
      const float at = top == -CUDART_INF_F ? 0.f : top;
      const float before = sum * ex2_approx(mx - at);
      sum = before;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        ml[k].y *= ex2_approx(ml[k].x - at);
        sum += ml[k].y;
      }
      const float inv = inverse_sum(sum);
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] *= before * inv;
#pragma unroll
      for (int k = 0; k < 16; ++k)
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = __fmaf_rn(v[k][i], ml[k].y * inv, acc[i]);
      mx = top;
    }
  }
};

struct Piece {
  int b, h, split, n_split;  // n_split 0: nothing to do
};

// Stages of 32 keys of sequence b; one for queries over no rows (somebody writes their zeros).
__device__ __forceinline__ int stages_of(const Kv8AttnParams& p, int b) {
  const int count = p.counts ? clampi(p.counts[b], 0, p.n) : p.n;
  return count ? max(1, (kv8_length(p.c, b) + kStageKeys - 1) / kStageKeys) : 0;
}
// For the weights: rows that no query asks about are copied.
__device__ __forceinline__ int stages_of(const Kv8WeighParams& p, int b) {
  return (kv8_length(p.c, b) + kStageKeys - 1) / kStageKeys;
}

// Pieces per kv head of a sequence with nst of all sequences' `sum` stages (per head).
__device__ __forceinline__ int pieces_of(int nst, long long sum, int per_head, int warps) {
  if (nst == 0) return 0;
  const int share = static_cast<int>(static_cast<float>(nst) / static_cast<float>(sum) * per_head + 0.01f);
  return clampi(share, 1, (nst + warps - 1) / warps);  // at least a stage for each warp
}

// The piece of block blockIdx.x (the same for all its threads; every warp works it out).
template <class P>
__device__ __forceinline__ Piece piece_of(const P& p, int warps) {
  const int lane = threadIdx.x & 31, kv = p.c.kv_heads, batch = p.c.batch;
  const int block = blockIdx.x;
  Piece r{0, 0, 0, 0};
  if (p.per_head == 0) {  // enough heads and sequences to fill the GPU: one piece each
    r.b = block / kv;
    r.h = block - r.b * kv;
    r.n_split = stages_of(p, r.b) ? 1 : 0;
    return r;
  }
  if (batch == 1) {
    r.n_split = pieces_of(stages_of(p, 0), stages_of(p, 0), p.per_head, warps);
    if (block >= r.n_split * kv) r.n_split = 0;
    if (r.n_split) {
      r.h = block / r.n_split;
      r.split = block - r.h * r.n_split;
    }
    return r;
  }
  long long sum = 0;
  for (int b0 = 0; b0 < batch; b0 += 32) sum += b0 + lane < batch ? stages_of(p, b0 + lane) : 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  int base = 0;
  for (int b0 = 0; b0 < batch; b0 += 32) {
    const int n = b0 + lane < batch ? pieces_of(stages_of(p, b0 + lane), sum, p.per_head, warps) : 0;
    int run = n * kv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    const unsigned here = __ballot_sync(0xffffffffu, block < base + run);
    if (here) {
      const int at = __ffs(here) - 1;
      r.b = b0 + at;
      r.n_split = __shfl_sync(0xffffffffu, n, at);
      const int local = block - (base + __shfl_sync(0xffffffffu, run, at) - r.n_split * kv);
      r.h = local / r.n_split;
      r.split = local - r.h * r.n_split;
      return r;
    }
    base += __shfl_sync(0xffffffffu, run, 31);
  }
  return r;
}

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(8 * NQ)) kv8_token_kernel(const __grid_constant__ Kv8AttnParams p) {
  using C = TokenCfg<D, NQ>;
  constexpr int RT = C::RT;
  grid_wait();
  const Piece pc = piece_of(p, kWarps);
  if (pc.n_split == 0) return;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  uint8_t* sq = smem + C::RING;
  float* sfactor = reinterpret_cast<float*>(smem + C::BODY);
  int* sseen = reinterpret_cast<int*>(sfactor + RT);
  __shared__ int is_last;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int kv_heads = p.c.kv_heads, heads = kv_heads * p.group;
  const int b = pc.b, h = pc.h;
  const int len = kv8_length(p.c, b);
  const int count = p.counts ? clampi(p.counts[b], 0, p.n) : p.n;
  const int nrow = count * p.group;
  const int nst = max(1, (len + kStageKeys - 1) / kStageKeys);
  const int st0 = static_cast<int>(static_cast<long long>(nst) * pc.split / pc.n_split);
  const int st1 = static_cast<int>(static_cast<long long>(nst) * (pc.split + 1) / pc.n_split);
  const int n_mine = st1 - st0 > warp ? (st1 - st0 - warp + kWarps - 1) / kWarps : 0;
  const uint32_t ring_a = smem_u32(smem + warp * (C::NST * C::STAGE));
  const uint32_t sq_a = smem_u32(sq);

  auto issue = [&](int i) {
    if (i < n_mine) {
      const int key0 = (st0 + warp + i * kWarps) * kStageKeys;
      const size_t tile = kv8_tile(p.c, b, key0 / kKv8Block, h);
      const size_t at = tile * (kKv8Block * D) + (key0 % kKv8Block) * D + lane * 16;
      const uint32_t dst = ring_a + (i % C::NST) * C::STAGE;
      const uint8_t* k8 = p.c.k8 + at;
      const uint8_t* v8 = p.c.v8 + at;
      constexpr int CPR = D / 16, ROWS = 32 / CPR;  // chunks per row, rows per pass
      const int held = len - key0;
      if (held >= kStageKeys) {
#pragma unroll
        for (int j = 0; j < CPR; ++j) {
          const int r = j * ROWS + lane / CPR, ch = lane % CPR;
          cp_async16(dst + k_at<D>(r, ch), k8 + j * 512, 16);
          cp_async16(dst + C::TILE + v_at<D>(r, ch), v8 + j * 512, 16);
        }
      } else {
        // rows that are not held are filled with zeros: what they hold may be NaN
#pragma unroll 1
        for (int j = 0; j < CPR; ++j) {
          const int r = j * ROWS + lane / CPR, ch = lane % CPR;
          cp_async16(dst + k_at<D>(r, ch), k8 + j * 512, r < held ? 16 : 0);
          cp_async16(dst + C::TILE + v_at<D>(r, ch), v8 + j * 512, r < held ? 16 : 0);
        }
      }
      if (lane < 2) cp_async4(dst + 2 * C::TILE + lane * 4, (lane ? p.c.vs : p.c.ks) + tile);
    }
    cp_async_commit();
  };
  issue(0);

  pack_queries<D>(sq, sfactor, p.q, (static_cast<size_t>(b) * p.n) * heads + h * p.group, p.group, heads, RT, nrow,
                  p.scale_log2, warp, kWarps);
  if (threadIdx.x < RT)
    sseen[threadIdx.x] = threadIdx.x < nrow ? min(len, seen_by(threadIdx.x, p.group, p.causal, len, count)) : 0;
  __syncthreads();

  float o[NQ][C::OT][4];
  float m[NQ][2], l[NQ][2], unit_e[NQ][2], factor[NQ][2];  // unit_e: R
  // queries 8 t + 2 c + j are this thread's columns
#pragma unroll
  for (int t = 0; t < NQ; ++t) {
#pragma unroll
    for (int i = 0; i < C::OT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[t][i][k] = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      m[t][j] = -CUDART_INF_F;
      l[t][j] = 0.f;
      unit_e[t][j] = kNoUnit;
      factor[t][j] = sfactor[t * 8 + 2 * c + j];
    }
  }
  const int seen_min = sseen[0];  // the first row sees least

  for (int it = 0; it < n_mine; ++it) {
    issue(it + 1);  // into the slot that the warp finished with one iteration ago
    cp_async_wait<1>();
    __syncwarp();
    const uint32_t st = ring_a + (it % C::NST) * C::STAGE;
    const int key0 = (st0 + warp + it * kWarps) * kStageKeys;

    float s[NQ][2][4];
    {
      uint4 kw[D / 64][2][2];
#pragma unroll
      for (int half = 0; half < D / 64; ++half)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int k = 0; k < 2; ++k) kw[half][u][k] = lds128(st + k_at<D>(u * 16 + k * 8 + g, c + 4 * half));
      scores<D, NQ>(s, kw, sq_a);
    }

    // ---- softmax
    const float2 sc = lds_f2(st + 2 * C::TILE);
    const float ev = static_cast<float>(exponent_of(sc.y));
    const bool full = key0 + kStageKeys <= seen_min;
    uint32_t pb[NQ][4];  // P^T as B fragments: keys 8 k + 2 c, + 1, query g
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      float w[2][4];
      bool may_rise = false;  // a contribution is at most the block's scale
      float mx[2], m_at[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float f = factor[t][j] * sc.x;
        mx[j] = -CUDART_INF_F;
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // key 8 k + g
          w[j][k] = s[t][k >> 1][(k & 1) * 2 + j] * f;
          if (!full && key0 + k * 8 + g >= sseen[t * 8 + 2 * c + j]) w[j][k] = -CUDART_INF_F;
          mx[j] = fmaxf(mx[j], w[j][k]);
        }
        mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 4));
        mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 8));
        mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 16));
        if (mx[j] > m[t][j] + kRise) {
          l[t][j] *= ex2_approx(m[t][j] - mx[j]);
          unit_e[t][j] += m[t][j] - mx[j];
          m[t][j] = mx[j];
        }
        m_at[j] = m[t][j] == -CUDART_INF_F ? 0.f : m[t][j];
        may_rise |= ev > unit_e[t][j] + kMaxDrift;
      }
      if (__any_sync(0xffffffffu, may_rise)) {
        float scale_o[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // the stage's largest contribution: -infinity where the row sees nothing of it
          const float most = ev + fminf(mx[j] - m_at[j], 0.f);
          scale_o[j] = 1.f;
          if (most > unit_e[t][j] + kMaxDrift) {
            scale_o[j] = ex2_approx(unit_e[t][j] - most);
            unit_e[t][j] = most;
          }
        }
#pragma unroll
        for (int i = 0; i < C::OT; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[t][i][k] *= scale_o[k & 1];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // Offset of the exponents.  Below -30 all of the stage's probabilities are 0 in f16, and the sum keeps
        // its precision.
        const float c_at = fmaxf(kPOff + ev - unit_e[t][j], -30.f);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[j][k] = ex2_approx((w[j][k] - m_at[j]) + c_at);
          sum += w[j][k];
        }
        l[t][j] = __fmaf_rn(sum, ex2_approx(-c_at), l[t][j]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) pb[t][k] = transpose8x8(pack_f16x2(w[0][k], w[1][k]));
    }

    // ---- output: rows g and g + 8 of tile i are features 16 i + g and + 8.  The load
    // leaves lane 4 g + c four keys of a feature: P's fragments hold keys 8 k + 2 c, + 1,
    // so matrix row 4 c + x of the 16 that a load transposes is key 2 c + x, or 8 + 2 c + x - 2.
#pragma unroll
    for (int i = 0; i < C::OT; ++i) {
      uint32_t v[4];
      const int x = lane & 3, r = (lane & 16) + 2 * ((lane & 15) >> 2) + (x & 1) + (x & 2) * 4;
      ldmatrix_trans8(v, st + C::TILE + v_at<D>(r, i));
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t a[4] = {e4m3x2_to_f16x2(v[2 * u] & 0xffffu), e4m3x2_to_f16x2(v[2 * u + 1] & 0xffffu),
                               e4m3x2_to_f16x2(v[2 * u] >> 16), e4m3x2_to_f16x2(v[2 * u + 1] >> 16)};
#pragma unroll
        for (int t = 0; t < NQ; ++t) mma_f16(o[t][i], a, pb[t][2 * u], pb[t][2 * u + 1]);
      }
    }
  }
  cp_async_wait<0>();

  // ---- merge the warps: output, maximum and sum of each row
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);                           // [warps][RT][D]
  float2* sml = reinterpret_cast<float2*>(so + kWarps * RT * C::ORow);  // [warps][RT]
#pragma unroll
  for (int t = 0; t < NQ; ++t)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = t * 8 + 2 * c + j;
      const float unit = ex2_approx(unit_e[t][j] - kPOff);
      float sum = l[t][j];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const float inv = inverse_sum(sum);
      if (g == 0) sml[warp * RT + r] = make_float2(m[t][j], sum);
      if (r < nrow) {
        float* dst = so + (warp * RT + r) * C::ORow + g;
#pragma unroll
        for (int i = 0; i < C::OT; ++i) {
          dst[16 * i] = o[t][i][j] * inv * unit;
          dst[16 * i + 8] = o[t][i][2 + j] * inv * unit;
        }
      }
    }
  __syncthreads();

  // From here on a warp has a row, a lane PER of its features.
  constexpr int PER = D / 32;
  // The mean of the first `parts` of four results of row r in shared memory, each weighted by its sum
  // times 2^(its maximum - the largest).
  struct Merged {
    float mx = -CUDART_INF_F, sum = 0.f, acc[PER] = {};
  };
  static_assert(kWarps == 4, "the warps merge at once");
  auto merged = [&](int r, int parts) {
    Merged x;
    float2 ml[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      ml[w] = w < parts ? sml[w * RT + r] : make_float2(-CUDART_INF_F, 0.f);
      x.mx = fmaxf(x.mx, ml[w].x);
    }
    const float at = x.mx == -CUDART_INF_F ? 0.f : x.mx;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      ml[w].y *= ex2_approx(ml[w].x - at);
      x.sum += ml[w].y;
    }
    const float inv = inverse_sum(x.sum);
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (w < parts)
#pragma unroll
        for (int i = 0; i < PER; ++i) x.acc[i] = __fmaf_rn(so[(w * RT + r) * C::ORow + i * 32 + lane], ml[w].y * inv, x.acc[i]);
    return x;
  };
  // writes row r
  auto finish = [&](int r, const Merged& x) {
    const size_t at = (static_cast<size_t>(b) * p.n + r / p.group) * heads + h * p.group + r % p.group;
    const bool any = sseen[r] > 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      static_cast<__nv_bfloat16*>(p.out)[at * D + i * 32 + lane] = __float2bfloat16(any ? x.acc[i] : 0.f);
    if (lane == 0) {
      const float lse2 = x.mx + log2f(x.sum);
      if (p.lse) p.lse[at] = any ? lse2 * CUDART_LN2_F : -CUDART_INF_F;
      if (p.lse2) p.lse2[at] = any ? lse2 : CUDART_INF_F;  // 2^(s - inf) = 0: a row that sees nothing weighs nothing
    }
  };
  for (int r = warp; r < nrow; r += kWarps) {
    const Merged x = merged(r, kWarps);
    if (pc.n_split == 1) {
      finish(r, x);
    } else {
      const size_t row = static_cast<size_t>(blockIdx.x) * RT + r;
#pragma unroll
      for (int i = 0; i < PER; ++i) p.part_o[row * D + i * 32 + lane] = x.acc[i];
      if (lane == 0) reinterpret_cast<float2*>(p.part_ml)[row] = make_float2(x.mx, x.sum);
    }
  }
  if (RT > 8) {
    // the rows of many queries are merged by a launch of their own
    if (threadIdx.x == 0 && pc.split == 0)
      p.pieces[static_cast<size_t>(b) * kv_heads + h] = make_int2(blockIdx.x, pc.n_split);
    return;
  }
  if (pc.n_split == 1) return;

  // ---- the last piece of the (sequence, kv head) to finish merges them all
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned* ticket = p.tickets + static_cast<size_t>(b) * kv_heads + h;
    unsigned before;
    // releases the block's partials (ordered before by the barrier) and acquires the others'
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(ticket) : "memory");
    is_last = before == static_cast<unsigned>(pc.n_split - 1);
    if (is_last) *ticket = 0;
  }
  __syncthreads();
  if (!is_last) return;
  // the warps share rows, or with fewer than four rows each row's pieces
  const size_t first = static_cast<size_t>(blockIdx.x - pc.split) * RT;
  const int row_warps = nrow >= 4 ? 4 : nrow >= 2 ? 2 : 1, piece_warps = 4 / row_warps;
  const int mine = warp / row_warps;  // of each row's pieces: mine, mine + piece_warps, ..
  for (int r = warp % row_warps; r < nrow; r += row_warps) {
    RowMerge<D> x;
    x.pieces(p.part_o, p.part_ml, first + r, RT, mine, pc.n_split, piece_warps);
    if (lane == 0) sml[mine * RT + r] = make_float2(x.mx, x.sum);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) so[(mine * RT + r) * C::ORow + lane * (D / 32) + i] = x.acc[i];
  }
  __syncthreads();
  for (int r = warp; r < nrow; r += kWarps) finish(r, merged(r, piece_warps));
}

// The rows of tiles of more than 8 queries: a warp each.
template <int D>
__global__ void __launch_bounds__(128) kv8_token_merge_kernel(const __grid_constant__ Kv8AttnParams p, int tile_rows) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.z, h = blockIdx.y, r = blockIdx.x * 4 + (threadIdx.x >> 5);
  grid_wait();
  const int count = p.counts ? clampi(p.counts[b], 0, p.n) : p.n;
  if (r >= count * p.group) return;
  const int2 by = p.pieces[static_cast<size_t>(b) * p.c.kv_heads + h];  // the first block and the number of pieces
  if (by.y <= 1) return;
  RowMerge<D> x;
  x.pieces(p.part_o, p.part_ml, static_cast<size_t>(by.x) * tile_rows + r, tile_rows, 0, by.y, 1);
  const int len = kv8_length(p.c, b);
  const bool any = min(len, seen_by(r, p.group, p.causal, len, count)) > 0;
  const size_t at = (static_cast<size_t>(b) * p.n + r / p.group) * (p.c.kv_heads * p.group) + h * p.group + r % p.group;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + at * D) + lane * (D / 64);
#pragma unroll
  for (int i = 0; i < D / 64; ++i) dst[i] = any ? pack_bf16x2(x.acc[2 * i], x.acc[2 * i + 1]) : 0u;
  if (lane == 0) {
    const float lse2 = x.mx + log2f(x.sum);
    if (p.lse) p.lse[at] = any ? lse2 * CUDART_LN2_F : -CUDART_INF_F;
    if (p.lse2) p.lse2[at] = any ? lse2 : CUDART_INF_F;
  }
}

// ------------------------------------------------------------------ weights
//
// weights[j] = weights_in[j] + sum over query rows of 2^(score - lse2): the
// second look at the scores, with their final sums.  A warp takes 32 keys at a
// time straight from global memory (L2, where the attention has just read them)
// and all query rows over them; a key's sum stays within four threads, so its
// order is fixed and nothing is added through memory.  25 rows over 48 MB of keys: 16
// to 19 us, of which the matrix instructions need 10.
constexpr int kWeighWarps = 8;
constexpr int kWeighThreads = kWeighWarps * 32;

template <int D, int NQ>
__global__ void __launch_bounds__(kWeighThreads, 2) kv8_weigh_kernel(const __grid_constant__ Kv8WeighParams p) {
  constexpr int RT = 8 * NQ;
  __shared__ __align__(16) uint8_t sq[RT * D * 2];
  __shared__ float sfactor[RT], slse[RT];
  __shared__ int sseen[RT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  grid_wait();
  const Piece pc = piece_of(p, kWeighWarps);
  const int b = pc.b, h = pc.h;
  const int len = kv8_length(p.c, b);
  if (pc.n_split == 0 || len == 0) return;
  const int heads = p.c.kv_heads * p.group;
  const int count = p.counts ? clampi(p.counts[b], 0, p.n) : p.n;
  const int nrow = count * p.group;
  const int nst = (len + kStageKeys - 1) / kStageKeys;
  const int end = min(len, static_cast<int>(static_cast<long long>(nst) * (pc.split + 1) / pc.n_split) * kStageKeys);
  constexpr int step = kWeighWarps * kStageKeys;

  uint4 kw[D / 64][2][2];
  float ks = 0.f;
  auto load = [&](int key0) {
    const size_t tile = kv8_tile(p.c, b, min(key0, len - 1) / kKv8Block, h);
    ks = __ldcg(p.c.ks + tile);
    const uint4* src = reinterpret_cast<const uint4*>(p.c.k8 + tile * (kKv8Block * D));
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          const int key = key0 + u * 16 + k * 8 + g;
          kw[half][u][k] = make_uint4(0, 0, 0, 0);
          if (key < len) kw[half][u][k] = __ldcg(src + (key % kKv8Block) * (D / 16) + c + 4 * half);
        }
  };
  int key0 = (static_cast<int>(static_cast<long long>(nst) * pc.split / pc.n_split) + warp) * kStageKeys;
  if (key0 < end) load(key0);
  pack_queries<D>(sq, sfactor, p.q, (static_cast<size_t>(b) * p.n) * heads + h * p.group, p.group, heads, RT, nrow,
                  p.scale_log2, warp, kWeighWarps);
  if (threadIdx.x < RT) {
    const int r = threadIdx.x;
    slse[r] = r < nrow ? p.lse2[(static_cast<size_t>(b) * p.n + r / p.group) * heads + h * p.group + r % p.group]
                       : CUDART_INF_F;
    sseen[r] = r < nrow ? seen_by(r, p.group, p.causal, len, count) : 0;
  }
  __syncthreads();
  const uint32_t sq_a = smem_u32(sq);
  const size_t row = (static_cast<size_t>(b) * p.c.kv_heads + h) * p.c.capacity;

  for (; key0 < end; key0 += step) {
    const int key = key0 + c * 8 + g;  // whose sum this thread writes
    const float before = key < len ? p.weights_in[row + key] : 0.f;
    float s[NQ][2][4];
    scores<D, NQ>(s, kw, sq_a);
    const float scale = ks;
    const int at = key0;
    if (key0 + step < end) load(key0 + step);
    const bool full = at + kStageKeys <= sseen[0];
    float sum[4] = {0.f, 0.f, 0.f, 0.f};  // keys 8 k + g
#pragma unroll
    for (int t = 0; t < NQ; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = t * 8 + 2 * c + j;
        const float f = sfactor[r] * scale, lse = slse[r];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float w = ex2_approx(s[t][k >> 1][(k & 1) * 2 + j] * f - lse);
          sum[k] += full || at + k * 8 + g < sseen[r] ? w : 0.f;
        }
      }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
      sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
    }
    const float mine = c == 0 ? sum[0] : c == 1 ? sum[1] : c == 2 ? sum[2] : sum[3];
    if (key < len) p.weights[row + key] = before + mine;
  }
}

template <int D, int NQ>
cudaError_t configure() {
  return cudaFuncSetAttribute(kv8_token_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              TokenCfg<D, NQ>::SMEM);
}
template <int D>
cudaError_t configure_all() {
  cudaError_t e = configure<D, 1>();
  if (e == cudaSuccess) e = configure<D, 2>();
  if (e == cudaSuccess) e = configure<D, 4>();
  return e;
}

template <int D>
cudaError_t launch_token(const Kv8AttnParams& p, int grid, cudaStream_t s) {
  const int rows = p.n * p.group;
  const cudaError_t e =
      rows <= 8 ? launch_kernel(kv8_token_kernel<D, 1>, grid, kThreads, TokenCfg<D, 1>::SMEM, s, 1, p)
      : rows <= 16 ? launch_kernel(kv8_token_kernel<D, 2>, grid, kThreads, TokenCfg<D, 2>::SMEM, s, 1, p)
                   : launch_kernel(kv8_token_kernel<D, 4>, grid, kThreads, TokenCfg<D, 4>::SMEM, s, 1, p);
  if (e != cudaSuccess || rows <= 8 || p.per_head <= 1) return e;
  return launch_kernel(kv8_token_merge_kernel<D>, dim3((rows + 3) / 4, p.c.kv_heads, p.c.batch), 128, 0, s, 1, p,
                       rows <= 16 ? 16 : 32);
}

template <int D>
cudaError_t launch_weigh(const Kv8WeighParams& p, int grid, cudaStream_t s) {
  const int rows = p.n * p.group;
  return launch_kernel(rows <= 8 ? kv8_weigh_kernel<D, 1> : rows <= 16 ? kv8_weigh_kernel<D, 2> : kv8_weigh_kernel<D, 4>,
                       grid, kWeighThreads, 0, s, 1, p);
}

}  // namespace

cudaError_t kv8_configure(int head_dim) { return head_dim == 128 ? configure_all<128>() : configure_all<64>(); }

namespace {
// Pieces: as many as run at once, shared by the heads.  A sequence has at least
// one piece per head, so a batch may have up to one more for each; with twice as
// many heads as run at once nothing is cut.
Kv8TokenPlan kv8_pieces_plan(int batch, int kv_heads, long long slots) {
  Kv8TokenPlan pl;
  const long long items = static_cast<long long>(batch) * kv_heads;
  if (items >= 2 * slots) {
    pl.per_head = 0;
    pl.grid = static_cast<int>(items);
    pl.part_blocks = 0;
  } else {
    // With more than half as many items as run at once, whole numbers of pieces leave the longest
    // up to twice the others: pieces of half the length, two rounds of them (a batch of 32 over 8
    // kv heads 61 -> 57 us; of 8, where it only adds merges, 23 -> 29).
    const long long rounds = items * 2 > slots ? 2 : 1;
    pl.per_head = static_cast<int>(std::max(1ll, rounds * slots / kv_heads));
    pl.grid = static_cast<int>(batch == 1 ? static_cast<long long>(pl.per_head) * kv_heads
                                          : static_cast<long long>(pl.per_head) * kv_heads + items);
    pl.part_blocks = pl.grid;
  }
  return pl;
}
}  // namespace

Kv8TokenPlan kv8_token_plan(int batch, int kv_heads, int rows, int sms) {
  return kv8_pieces_plan(batch, kv_heads, sms * blocks_per_sm(rows));
}
Kv8TokenPlan kv8_weigh_plan(int batch, int kv_heads, int sms) { return kv8_pieces_plan(batch, kv_heads, sms * 2); }

cudaError_t launch_kv8_token_attn(int head_dim, const Kv8AttnParams& p, int grid, cudaStream_t s) {
  return head_dim == 128 ? launch_token<128>(p, grid, s) : launch_token<64>(p, grid, s);
}

cudaError_t launch_kv8_weigh(int head_dim, const Kv8WeighParams& p, int grid, cudaStream_t s) {
  return head_dim == 128 ? launch_weigh<128>(p, grid, s) : launch_weigh<64>(p, grid, s);
}

}  // namespace ff
