// Attention of few query rows over the 8-bit cache, and the weight that every
// key received.
//
// For one (sequence, kv head) the query rows are the `group` heads of each of
// its tokens (row r = token r / group, head r mod group): they read the same
// keys, so they share every loaded tile.  Scores and outputs run on the
// m16n8k16 f16 matrix instruction with fp32 accumulation:
//   * a code becomes f16 exactly (one conversion for two codes), so the block
//     scales stay out of the operands: K's multiplies the scores, V's enters
//     as an exponent of the probabilities;
//   * a query row is scaled by a power of two to put its largest magnitude
//     into [2^14, 2^15): exact in f16 for every value above 2^-29 of it;
//   * probabilities go to f16 relative to the running row maximum (11 bits
//     against bf16's 8), times 2^(kPOff + ev - U) where 2^ev is the V block's
//     scale and 2^U the unit in which the output accumulates; U follows ev
//     only when they are more than 2^6 apart, so a block costs no rescale of
//     the accumulators and the f16 range holds whatever the scales are.
// Which feature a matrix slot means is free as long as Q and K agree, and the
// same holds for the columns of V: each thread takes 16 consecutive codes, so
// all shared loads are 16 bytes wide and nothing is transposed.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "ff_kv8.cuh"
#include "ff_ptx.cuh"

namespace ff {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStageKeys = 32;  // keys of one warp's stage
constexpr int kPOff = 8;
constexpr int kMaxDrift = 6;    // ev - U before the output's unit moves: p * 2^(8 + 6) stays below f16's 65504
constexpr int kMaxFall = 80;    // U - ev beyond which the block is nothing beside what a unit that large has summed

template <int D>
struct TokenCfg {
  static constexpr int CPR = D / 16;                       // 16-byte chunks per row
  static constexpr int KS = D / 16;                        // matrix steps over the features
  static constexpr int NT = D / 8;                         // output column tiles
  static constexpr int TILE = kStageKeys * D;              // bytes of K or V of a stage
  static constexpr int STAGE = 2 * TILE + 16;              // and the two scales
  static constexpr int NST = 3;
  static constexpr int RING = kWarps * NST * STAGE;
  static constexpr int Q_BYTES = kKv8TokenRows * D * 2;
  static constexpr int ROW_BYTES = kKv8TokenRows * 8;      // row factor and visible keys
  static constexpr int MERGE = kWarps * kKv8TokenRows * (D + 2) * 4;
  static constexpr int BODY = RING > MERGE ? RING : MERGE;
  static constexpr int SMEM = Q_BYTES + ROW_BYTES + BODY + 16;
  static_assert(SMEM <= 232448, "shared memory");
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
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk `ch` of row `r` in a stage's K or V tile.  The
// xor spreads both access patterns over all banks: a K load takes four chunks
// of two adjacent rows, a V load two chunks of four rows of equal parity.
template <int D>
__device__ __forceinline__ int chunk_at(int r, int ch) {
  if (D == 128) return r * 128 + ((ch ^ ((r & 6) ^ ((r & 1) << 2))) << 4);
  const int line = r >> 1;  // two 64-byte rows per 128-byte line
  return line * 128 + (((((r & 1) << 2) | ch) ^ (line & 7)) << 4);
}

// Query rows row0 .. row0 + rows - 1 of a (sequence, kv head) into shared memory
// as A fragments of the matrix instruction (f16, scaled per row), with each
// row's factor (score = accumulator * factor * K scale, in log2 units).  A
// fragment of step s holds, for lane 4 g + c, features 16 (c + 4 (s / 4)) +
// 4 (s mod 4) .. + 3 of rows g and g + 8.  Rows past `valid` are zeros.
template <int D>
__device__ __forceinline__ void pack_queries(uint8_t* sq, float* factor, const void* q, size_t q_row0, int group,
                                             size_t token_stride, int row0, int rows, int valid, float scale_log2,
                                             int warp, int warps) {
  constexpr int PER = D / 32;  // features per lane
  const int lane = threadIdx.x & 31;
  for (int r = warp; r < rows; r += warps) {
    float x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = 0.f;
    uint32_t amax = 0;
    if (row0 + r < valid) {
      const int row = row0 + r;
      const uint32_t* src = static_cast<const uint32_t*>(q) +
                            (q_row0 + static_cast<size_t>(row / group) * token_stride + row % group) * (D / 2) +
                            lane * (PER / 2);
#pragma unroll
      for (int i = 0; i < PER / 2; ++i) {
        const uint32_t w = __ldg(src + i);
        amax = max(amax, bf16x2_finite_max(w));
        x[2 * i] = bf16_lo(w);
        x[2 * i + 1] = bf16_hi(w);
      }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    const int k = clampi(static_cast<int>(amax >> 7) - 127, -100, 127);  // exponent of the largest magnitude
    const float up = pow2i(14 - k);
    const int f0 = lane * PER;
    const int half = f0 / 64, c = (f0 % 64) / 16, s = half * 4 + (f0 % 16) / 4;
    uint32_t* dst = reinterpret_cast<uint32_t*>(sq) + (((r / 16) * (D / 16) + s) * 32 + (r % 8) * 4 + c) * 4 +
                    ((r % 16) / 8) + ((f0 % 4) / 2) * 2;
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) dst[2 * i] = pack_f16x2(x[2 * i] * up, x[2 * i + 1] * up);
    if (lane == 0) factor[r] = pow2i(k - 14) * scale_log2;
  }
}

// Rows of K seen by query row r.
__device__ __forceinline__ int seen_by(int r, int group, int causal, int len, int count) {
  return causal ? max(0, len - count + r / group + 1) : len;
}

// ------------------------------------------------------------ token attention
//
// Grid (kv heads * row tiles, key ranges, sequences); 8 warps, each with its own
// ring of 32-key stages filled by asynchronous 16-byte copies (no barrier
// between warps until the end) and its own running maximum, sum and output.
// The warps' results merge in shared memory, the key ranges' through partials:
// the last range of a tile to finish merges them in a fixed order.
template <int D, int MT>
__global__ void __launch_bounds__(kThreads, 1) kv8_token_kernel(const __grid_constant__ Kv8AttnParams p) {
  using C = TokenCfg<D>;
  constexpr int RT = 16 * MT;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* sq = smem;
  float* sfactor = reinterpret_cast<float*>(smem + C::Q_BYTES);
  int* sseen = reinterpret_cast<int*>(sfactor + kKv8TokenRows);
  uint8_t* body = smem + C::Q_BYTES + C::ROW_BYTES;
  volatile int* flag = reinterpret_cast<int*>(body + C::BODY);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int b = blockIdx.z, h = blockIdx.x / p.row_tiles, rt = blockIdx.x - h * p.row_tiles;
  const int heads = p.c.kv_heads * p.group;
  const int len = kv8_length(p.c, b);
  const int count = p.counts ? clampi(p.counts[b], 0, p.n) : p.n;
  const int rows = count * p.group;
  const int row0 = rt * RT;
  if (row0 >= rows) return;
  const int nrow = min(RT, rows - row0);
  // keys that some row of the tile sees; the last row sees most
  const int n_keys = min(len, seen_by(row0 + nrow - 1, p.group, p.causal, len, count));
  const int n_stage = (n_keys + kStageKeys - 1) / kStageKeys;
  const int n_split = max(1, min(p.splits, (n_stage + kWarps - 1) / kWarps));
  const int split = blockIdx.y;
  if (split >= n_split) return;
  const int st0 = static_cast<int>(static_cast<long long>(n_stage) * split / n_split);
  const int st1 = static_cast<int>(static_cast<long long>(n_stage) * (split + 1) / n_split);

  uint8_t* ring = body + warp * (C::NST * C::STAGE);
  const uint32_t ring_a = smem_u32(ring);
  const int n_mine = st1 - st0 > warp ? (st1 - st0 - warp + kWarps - 1) / kWarps : 0;

  auto issue = [&](int i) {
    if (i < n_mine) {
      const int key0 = (st0 + warp + i * kWarps) * kStageKeys;
      const size_t tile = kv8_tile(p.c, b, key0 / kKv8Block, h);
      const size_t at = tile * (kKv8Block * D) + (key0 % kKv8Block) * D;
      const uint32_t dst = ring_a + (i % C::NST) * C::STAGE;
#pragma unroll
      for (int j = 0; j < C::CPR; ++j) {
        const int unit = j * 32 + lane;
        const int r = unit / C::CPR, ch = unit % C::CPR;
        // rows that are not held are filled with zeros: what they hold may be NaN
        const int bytes = key0 + r < len ? 16 : 0;
        const int to = chunk_at<D>(r, ch);
        cp_async16(dst + to, p.c.k8 + at + unit * 16, bytes);
        cp_async16(dst + C::TILE + to, p.c.v8 + at + unit * 16, bytes);
      }
      if (lane < 2) cp_async4(dst + 2 * C::TILE + lane * 4, (lane ? p.c.vs : p.c.ks) + tile);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::NST - 1; ++i) issue(i);

  pack_queries<D>(sq, sfactor, p.q, (static_cast<size_t>(b) * p.n) * heads + h * p.group, p.group, heads, row0, RT,
                  rows, p.scale_log2, warp, kWarps);
  if (threadIdx.x < RT)
    sseen[threadIdx.x] =
        threadIdx.x < nrow ? min(len, seen_by(row0 + threadIdx.x, p.group, p.causal, len, count)) : 0;
  __syncthreads();

  float o[MT][C::NT][4];
  float m[MT][2], l[MT][2], factor[MT][2];
  int seen[MT][2];
  int seen_min = 0x7fffffff;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int i = 0; i < C::NT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[mt][i][k] = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m[mt][k] = -CUDART_INF_F;
      l[mt][k] = 0.f;
      factor[mt][k] = sfactor[mt * 16 + k * 8 + g];
      seen[mt][k] = sseen[mt * 16 + k * 8 + g];
      if (mt * 16 + k * 8 + g < nrow) seen_min = min(seen_min, seen[mt][k]);
    }
  }
  seen_min = __reduce_min_sync(0xffffffffu, seen_min);
  int unit_e = 0;
  const uint32_t sq_a = smem_u32(sq);

  for (int it = 0; it < n_mine; ++it) {
    cp_async_wait<C::NST - 2>();
    __syncwarp();
    issue(it + C::NST - 1);  // into the slot that the warp finished with one iteration ago
    const uint32_t st = ring_a + (it % C::NST) * C::STAGE;
    const int key0 = (st0 + warp + it * kWarps) * kStageKeys;

    // ---- scores
    float s[MT][4][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[mt][nt][k] = 0.f;
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {
      uint32_t kw[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const uint4 w = lds128(st + chunk_at<D>(nt * 8 + g, c + 4 * half));
        kw[nt][0] = w.x;
        kw[nt][1] = w.y;
        kw[nt][2] = w.z;
        kw[nt][3] = w.w;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint4 w = lds128(sq_a + ((mt * C::KS + half * 4 + k) * 32 + lane) * 16);
          a[mt][0] = w.x;
          a[mt][1] = w.y;
          a[mt][2] = w.z;
          a[mt][3] = w.w;
        }
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const uint32_t b0 = e4m3x2_to_f16x2(kw[nt][k] & 0xffffu), b1 = e4m3x2_to_f16x2(kw[nt][k] >> 16);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) mma_f16(s[mt][nt], a[mt], b0, b1);
        }
      }
    }

    // ---- softmax
    const float* sc = reinterpret_cast<const float*>(ring + (it % C::NST) * C::STAGE + 2 * C::TILE);
    const float ks = sc[0];
    const int ev = exponent_of(sc[1]);
    if (it == 0) unit_e = ev;
    if (ev - unit_e > kMaxDrift || (unit_e - ev > kMaxDrift && unit_e - ev <= kMaxFall)) {
      const float f = pow2i(max(unit_e - ev, -126));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < C::NT; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[mt][i][k] *= f;
      unit_e = ev;
    }
    const float pscale = pow2i(max(kPOff + ev - unit_e, -126));
    const bool full = key0 + kStageKeys <= seen_min;
    uint32_t pa[MT][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float f = factor[mt][k] * ks;
        float mx = -CUDART_INF_F;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float t = s[mt][nt][2 * k + j] * f;
            if (!full && key0 + nt * 8 + 2 * c + j >= seen[mt][k]) t = -CUDART_INF_F;
            s[mt][nt][2 * k + j] = t;
            mx = fmaxf(mx, t);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = fmaxf(m[mt][k], mx);
        const float m_at = m_new == -CUDART_INF_F ? 0.f : m_new;
        const float alpha = ex2_approx(m[mt][k] - m_at);
        m[mt][k] = m_new;
        float sum = 0.f;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const float p0 = ex2_approx(s[mt][nt][2 * k] - m_at);
          const float p1 = ex2_approx(s[mt][nt][2 * k + 1] - m_at);
          sum += p0 + p1;
          pa[mt][nt >> 1][(nt & 1) * 2 + k] = pack_f16x2(p0 * pscale, p1 * pscale);
        }
        l[mt][k] = l[mt][k] * alpha + sum;
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int i = 0; i < C::NT; ++i) {
            o[mt][i][2 * k] *= alpha;
            o[mt][i][2 * k + 1] *= alpha;
          }
        }
      }
    }

    // ---- output: column i of lane group g stands for feature g * NT + i
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      constexpr int W = C::NT / 4;  // 4-code words per row of a lane
      uint32_t vw[4][W];            // rows 2c, 2c + 1, 2c + 8, 2c + 9 of the 16 keys
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 16 * j + 2 * c + (k & 1) + (k >> 1) * 8;
        if (D == 128) {
          const uint4 w = lds128(st + C::TILE + chunk_at<D>(r, g));
          vw[k][0] = w.x;
          vw[k][1] = w.y;
          vw[k][W - 2] = w.z;
          vw[k][W - 1] = w.w;
        } else {
          const uint2 w = lds64(st + C::TILE + chunk_at<D>(r, g >> 1) + (g & 1) * 8);
          vw[k][0] = w.x;
          vw[k][1] = w.y;
        }
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint32_t x0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), x1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
        const uint32_t y0 = __byte_perm(vw[2][w], vw[3][w], 0x5140), y1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
        const uint32_t lo[4] = {x0 & 0xffffu, x0 >> 16, x1 & 0xffffu, x1 >> 16};
        const uint32_t hi[4] = {y0 & 0xffffu, y0 >> 16, y1 & 0xffffu, y1 >> 16};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t b0 = e4m3x2_to_f16x2(lo[k]), b1 = e4m3x2_to_f16x2(hi[k]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) mma_f16(o[mt][4 * w + k], pa[mt][j], b0, b1);
        }
      }
    }
  }
  cp_async_wait<0>();

  // ---- merge the warps: output, maximum and sum of each row
  __syncthreads();
  float* so = reinterpret_cast<float*>(body);                    // [warps][RT][D]
  float2* sml = reinterpret_cast<float2*>(so + kWarps * RT * D);  // [warps][RT]
  const float unit = pow2i(clampi(unit_e - kPOff, -126, 127));
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = mt * 16 + k * 8 + g;
      float sum = l[mt][k];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (c == 0) sml[warp * RT + r] = make_float2(m[mt][k], sum);
      if (r < nrow) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float4* dst = reinterpret_cast<float4*>(so + (warp * RT + r) * D + (2 * c + j) * C::NT);
#pragma unroll
          for (int i = 0; i < C::NT / 4; ++i)
            dst[i] = make_float4(o[mt][4 * i][2 * k + j] * unit, o[mt][4 * i + 1][2 * k + j] * unit,
                                 o[mt][4 * i + 2][2 * k + j] * unit, o[mt][4 * i + 3][2 * k + j] * unit);
        }
      }
    }
  __syncthreads();

  const size_t item = (static_cast<size_t>(b) * p.c.kv_heads + h) * p.row_tiles + rt;
  // writes row r (feature d of its output, unnormalised, with maximum and sum)
  auto finish = [&](int r, int d, float acc, float mx, float sum) {
    const int row = row0 + r;
    const size_t at = (static_cast<size_t>(b) * p.n + row / p.group) * heads + h * p.group + row % p.group;
    const bool any = sseen[r] > 0;
    static_cast<__nv_bfloat16*>(p.out)[at * D + d] = __float2bfloat16(any ? acc / sum : 0.f);
    if (d == 0) {
      const float lse2 = mx + log2f(sum);
      if (p.lse) p.lse[at] = any ? lse2 * CUDART_LN2_F : -CUDART_INF_F;
      if (p.lse2) p.lse2[at] = any ? lse2 : CUDART_INF_F;  // 2^(s - inf) = 0: a row that sees nothing weighs nothing
    }
  };
  for (int idx = threadIdx.x; idx < nrow * D; idx += kThreads) {
    const int r = idx / D, d = idx % D;
    float mx = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sml[w * RT + r].x);
    const float at = mx == -CUDART_INF_F ? 0.f : mx;
    float acc = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sml[w * RT + r];
      const float f = exp2f(ml.x - at);
      sum += ml.y * f;
      acc += so[(w * RT + r) * D + d] * f;
    }
    if (n_split == 1) {
      finish(r, d, acc, at, sum);
    } else {
      const size_t part = (item * p.splits + split) * RT + r;
      p.part_o[part * D + d] = acc;
      if (d == 0) reinterpret_cast<float2*>(p.part_ml)[part] = make_float2(mx, sum);
    }
  }
  if (n_split == 1) return;

  // ---- the last key range to arrive merges them all
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool last = atomicAdd(p.tickets + item, 1u) == static_cast<unsigned>(n_split - 1);
    if (last) p.tickets[item] = 0;
    *flag = last;
  }
  __syncthreads();
  if (!*flag) return;
  __threadfence();
  for (int idx = threadIdx.x; idx < nrow * D; idx += kThreads) {
    const int r = idx / D, d = idx % D;
    const size_t part = item * p.splits * RT + r;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    float mx = -CUDART_INF_F;
    for (int k = 0; k < n_split; ++k) mx = fmaxf(mx, __ldcg(&ml[part + static_cast<size_t>(k) * RT].x));
    const float at = mx == -CUDART_INF_F ? 0.f : mx;
    float acc = 0.f, sum = 0.f;
#pragma unroll 4
    for (int k = 0; k < n_split; ++k) {
      const size_t pk = part + static_cast<size_t>(k) * RT;
      const float2 x = __ldcg(&ml[pk]);
      const float f = exp2f(x.x - at);
      sum += x.y * f;
      acc += __ldcg(&p.part_o[pk * D + d]) * f;
    }
    finish(r, d, acc, at, sum);
  }
}

// ------------------------------------------------------------------ weights
//
// weights[j] = weights_in[j] + sum over query rows of 2^(score - lse2): the
// second look at the scores, with their final sums.  A warp keeps the converted
// keys of its 32 rows in registers and passes all query rows over them; each key's
// sum stays in one thread's registers, so its order is fixed and nothing is added
// through memory.
constexpr int kWeighWarps = 4;
constexpr int kWeighRows = 64;  // query rows in shared memory at a time

template <int D>
__global__ void __launch_bounds__(kWeighWarps * 32) kv8_weigh_kernel(const __grid_constant__ Kv8WeighParams p) {
  constexpr int KS = D / 16;
  __shared__ __align__(16) uint8_t sq[kWeighRows * D * 2];
  __shared__ float sfactor[kWeighRows], slse[kWeighRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int b = blockIdx.z, h = blockIdx.y;
  const int heads = p.c.kv_heads * p.group;
  const int len = kv8_length(p.c, b);
  const int count = p.counts ? clampi(p.counts[b], 0, p.n) : p.n;
  const int rows = count * p.group;
  const int cta_key0 = blockIdx.x * (kWeighWarps * kStageKeys);
  if (cta_key0 >= len) return;
  const int key0 = cta_key0 + warp * kStageKeys;
  // the first token that sees the block's first key
  const int tok0 = p.causal ? clampi(cta_key0 - (len - count), 0, count) : 0;

  uint32_t kb[4][KS][2];
  float ks = 0.f;
  {
    const size_t tile = kv8_tile(p.c, b, min(key0, len - 1) / kKv8Block, h);
    ks = p.c.ks[tile];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const int key = key0 + nt * 8 + g;
#pragma unroll
      for (int half = 0; half < D / 64; ++half) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (key < len)
          w = __ldg(reinterpret_cast<const uint4*>(p.c.k8 + tile * (kKv8Block * D) + (key % kKv8Block) * D) + c +
                    4 * half);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          kb[nt][half * 4 + k][0] = e4m3x2_to_f16x2(x[k] & 0xffffu);
          kb[nt][half * 4 + k][1] = e4m3x2_to_f16x2(x[k] >> 16);
        }
      }
    }
  }
  float sum[4][2];
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) sum[nt][0] = sum[nt][1] = 0.f;
  const uint32_t sq_a = smem_u32(sq);

  for (int r0 = tok0 * p.group; r0 < rows; r0 += kWeighRows) {
    __syncthreads();
    pack_queries<D>(sq, sfactor, p.q, (static_cast<size_t>(b) * p.n) * heads + h * p.group, p.group, heads, r0,
                    kWeighRows, rows, p.scale_log2, warp, kWeighWarps);
    if (threadIdx.x < kWeighRows) {
      const int row = r0 + threadIdx.x;
      slse[threadIdx.x] =
          row < rows ? p.lse2[(static_cast<size_t>(b) * p.n + row / p.group) * heads + h * p.group + row % p.group]
                     : CUDART_INF_F;
    }
    __syncthreads();
    if (key0 >= len) continue;
    const int tiles = min(kWeighRows / 16, (rows - r0 + 15) / 16);
    for (int t = 0; t < tiles; ++t) {
      float s[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[nt][k] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint4 w = lds128(sq_a + ((t * KS + k) * 32 + lane) * 16);
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mma_f16(s[nt], a, kb[nt][k][0], kb[nt][k][1]);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = t * 16 + k * 8 + g;
        const float f = sfactor[r] * ks, lse = slse[r];
        const int seen = seen_by(r0 + r, p.group, p.causal, len, count);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float w = ex2_approx(s[nt][2 * k + j] * f - lse);
            if (key0 + nt * 8 + 2 * c + j < seen) sum[nt][j] += w;
          }
      }
    }
  }
  const size_t row = (static_cast<size_t>(b) * p.c.kv_heads + h) * p.c.capacity;
#pragma unroll
  for (int nt = 0; nt < 4; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float x = sum[nt][j];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      const int key = key0 + nt * 8 + 2 * c + j;
      if (g == 0 && key < len) p.weights[row + key] = p.weights_in[row + key] + x;
    }
}

}  // namespace

cudaError_t kv8_configure(int head_dim) {
  cudaError_t e;
  if (head_dim == 128) {
    e = cudaFuncSetAttribute(kv8_token_kernel<128, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, TokenCfg<128>::SMEM);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kv8_token_kernel<128, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, TokenCfg<128>::SMEM);
  } else {
    e = cudaFuncSetAttribute(kv8_token_kernel<64, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, TokenCfg<64>::SMEM);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kv8_token_kernel<64, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, TokenCfg<64>::SMEM);
  }
  return e;
}

cudaError_t launch_kv8_token_attn(int head_dim, const Kv8AttnParams& p, cudaStream_t s) {
  const dim3 grid(p.c.kv_heads * p.row_tiles, p.splits, p.c.batch);
  const bool one = p.n * p.group <= 16;
  if (head_dim == 128) {
    if (one)
      kv8_token_kernel<128, 1><<<grid, kThreads, TokenCfg<128>::SMEM, s>>>(p);
    else
      kv8_token_kernel<128, 2><<<grid, kThreads, TokenCfg<128>::SMEM, s>>>(p);
  } else {
    if (one)
      kv8_token_kernel<64, 1><<<grid, kThreads, TokenCfg<64>::SMEM, s>>>(p);
    else
      kv8_token_kernel<64, 2><<<grid, kThreads, TokenCfg<64>::SMEM, s>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv8_weigh(int head_dim, const Kv8WeighParams& p, cudaStream_t s) {
  const int keys = kWeighWarps * kStageKeys;
  const dim3 grid((p.c.capacity + keys - 1) / keys, p.c.kv_heads, p.c.batch);
  if (head_dim == 128)
    kv8_weigh_kernel<128><<<grid, kWeighWarps * 32, 0, s>>>(p);
  else
    kv8_weigh_kernel<64><<<grid, kWeighWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ff
