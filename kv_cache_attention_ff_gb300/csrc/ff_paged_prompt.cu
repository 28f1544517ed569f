// Attention of many query rows (prompts and chunks of them) over pages on tcgen05
// tensor cores.
//
// O = softmax(Q K^T / sqrt(d)) V, causal.  The heads of a group read the same keys,
// so a query tile is `tg` heads of a group by `tt` tokens, tg * tt <= 128 rows (row =
// token of the tile * tg + head): short prompts fill tiles, and only the last key tiles of
// a block cross the diagonal.  A unit is two such tiles, one after the other in
// the request, of one (request, kv head): the plan has listed them, longest first,
// cut into key ranges where they would leave SMs idle.
//
// One CTA per SM stays and takes units from the list in rounds, forth and back
// (so that each CTA's long and short units add up alike), 12 warps:
//   warps 0-3  softmax of query tile 0: one thread per row
//   warps 4-7  softmax of query tile 1
//   warp  8    tensor copies of K and V, page by page
//   warp  9    TMEM allocator and single-thread MMA issuer
//   warp 10    tensor copies of query tiles
//   warp 11    finds the CTA's units and leaves them in shared memory
// Per key tile j of 128 keys the MMA thread issues S0 = Q0 K_j^T, O0 += P0 V_{j-1},
// S1 = Q1 K_j^T, O1 += P1 V_{j-1}: the tensor pipe works on one tile's products
// while the other's scores become probabilities.  Tile 0 needs fewer key tiles than tile
// 1 and skips the rest.
// Probabilities stay in tensor memory: P V with P in shared memory takes 107 clocks per
// 16 keys, V's transposed reads and P's sharing the bandwidth, and 74 with P in
// tensor memory (Q K^T: 64, the rate of the pipe).  For d 128 its columns are those of a second S:
// the tiles take turns with one, which its reader has emptied while the other
// tile's P V runs.  (Two S and P in shared memory: 625 us where this takes 570, 9728
// rows behind 21472 of 8 heads.)
// Probabilities are bf16, which V's type asks for; sums and outputs are fp32.  The
// reference of a row's exponents (log2) is its running maximum plus 8 as it was when that
// was last passed: no exponent is above 0, and outputs are seldom rescaled.
//
// Long units take some 2600 clocks for a pair of query tiles and a key tile, of which their
// 32 products need 2275: 1.83 PFLOP/s at full clocks (the 9728 rows above), 0.95 of a large
// product's rate; in long series the power cap holds the clock at 1700 to 1800 MHz.  15600 rows of
// 12 heads 435 us, 475 under the cap; twelve prompts of up to 4680 rows with 32/8 heads
// (units of 13 key tiles on average, each of which costs 5000 clocks more) 480 and 530.
// With d 64 a pair of query tiles and a key tile take 2400 clocks, of which their products need some 1000 and their
// exponentials 1024 (32 a clock and SM): a softmax warp's own chain bounds it.  15600 rows of 12 heads 343 us.
// Measured and dropped: two threads a row in 16 softmax warps (588 for 530 at the time), a
// stream of products across units with results read out a tile later (equal), output warps of
// their own (the registers that they take from the others cost 20 % and more), two
// tiles' loads ahead into L2 (equal), the whole warp in the issuer's loop (711 for 632).
#include <algorithm>

#include <cuda_bf16.h>
#include <math_constants.h>

#include "ff_paged.cuh"
#include "ff_ptx.cuh"

namespace ff {
namespace {

constexpr int kThreads = 384;
constexpr float kRise = 8.f;  // log2

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(smem_dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// D[tmem] (+)= A[tmem] * B[smem desc], bf16 in, fp32 accumulate; A's row r lies in lane r, two values a column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// What a CTA works on: two query tiles of one (request, kv head) and a range of its key tiles.
struct __align__(16) Unit {
  int request, first, count, length;
  int head, heads;  // first query head of the tiles, and how many
  int kv_head;
  int kv0;          // first key tile
  int token[2];     // first token of each query tile
  int n[2];         // key tiles of each (0 where it has no rows)
  int last[2];      // keys of the last one that a row of the tile sees, up to a multiple of 16
  int n_split;      // 0: there are no more units
  int slot;         // of its partial results, and of the first range's
  int ticket;
  int pad[3];
};
constexpr int kAhead = 4;  // units in shared memory

template <int D>
struct PromptCfg {
  static constexpr int KB = D / 64;              // 128-byte column blocks per row
  static constexpr int BLK = 128 * 128;          // bytes of one [128 rows x 64 bf16] swizzled block
  static constexpr int Q_BYTES = 128 * D * 2;
  static constexpr int KV_BYTES = 128 * D * 2;
  static constexpr int NST = (D == 128) ? 4 : 8;
  static constexpr int OFF_KV = 2 * Q_BYTES;
  static constexpr int OFF_OUT = OFF_KV + NST * KV_BYTES;  // 32 rows x 64 features of each softmax warp, on their way out
  static constexpr int OFF_UNIT = OFF_OUT + 8 * 32 * 128;
  static constexpr int OFF_BAR = OFF_UNIT + kAhead * static_cast<int>(sizeof(Unit));
  static constexpr int N_BARS = 3 + 2 * NST + 10 + 2 + 2 * kAhead;
  static constexpr int SMEM = OFF_BAR + N_BARS * 8 + 16 + 1024;  // barriers, TMEM slot, abort and last flags; 1024 B alignment slack
  static_assert(SMEM <= 232448, "shared memory");
  // Tensor memory, 512 columns: O0 and O1 (D each), P0 and P1 (64 each: two probabilities a column), S (128), and with
  // D 64 a second S.
  static constexpr bool kTwoS = D == 64;
  static constexpr int TMEM_O = 0;
  static constexpr int TMEM_P = 2 * D;
  static constexpr int TMEM_S = TMEM_P + 128;
  static_assert(TMEM_S + (kTwoS ? 256 : 128) <= 512, "tensor memory");
};

// Entry `at` of the list as a unit.
__device__ __forceinline__ Unit unit_of(const PagedPromptParams& p, int at) {
  const int item = at / p.unit_heads, hh = at - item * p.unit_heads;
  const PagedPiece pc = p.units[item];
  Unit u;
  u.request = pc.request;
  u.first = pc.first;
  u.count = pc.count;
  u.length = pc.length;
  u.kv_head = hh / p.head_tiles;
  const int first = (hh - u.kv_head * p.head_tiles) * p.tg;  // of the group
  u.head = u.kv_head * p.group + first;
  u.heads = min(p.tg, p.group - first);
  int keys[2], tiles[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    u.token[t] = (2 * pc.block + t) * p.tt;
    const int tokens = clampi(pc.count - u.token[t], 0, p.tt);
    keys[t] = tokens ? pc.length - pc.count + u.token[t] + tokens : 0;
    tiles[t] = (keys[t] + 127) / 128;
  }
  const int all = max(tiles[0], tiles[1]);
  u.kv0 = static_cast<int>(static_cast<long long>(all) * pc.split / pc.n_split);
  const int kv1 = static_cast<int>(static_cast<long long>(all) * (pc.split + 1) / pc.n_split);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    u.n[t] = clampi(tiles[t] - u.kv0, 0, kv1 - u.kv0);
    u.last[t] = min(128, (keys[t] - (u.kv0 + u.n[t] - 1) * 128 + 15) / 16 * 16);
  }
  u.n_split = pc.n_split;
  u.ticket = pc.part * p.unit_heads + hh;
  u.slot = u.ticket + pc.split * p.unit_heads;
  u.pad[0] = u.pad[1] = u.pad[2] = 0;
  return u;
}

// Row of `out` of row r of query tile t, -1 where there is none.
__device__ __forceinline__ int row_of(const PagedPromptParams& p, const Unit& u, int t, int r) {
  const int i = r / p.tg, head = r - i * p.tg, token = (t ? u.token[1] : u.token[0]) + i;
  return i < p.tt && head < u.heads && token < u.count && u.first + token < p.n
             ? (u.first + token) * (p.kv_heads * p.group) + u.head + head
             : -1;
}

// The last range of a unit to finish merges them all, in their order.  A lane has a row; a warp has 32 rows and every
// 8 / `groups`-th chunk of 4 W features of them, with FLY ranges in flight: few rows in many ranges keep all
// eight softmax warps busy.
template <int D, int W, int FLY>
__device__ __noinline__ void merge(const PagedPromptParams& p, const Unit& u, int groups) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = u.n_split, group = warp & (groups - 1);
  const int row = row_of(p, u, group >> 2, (group & 3) * 32 + lane);
  if (row < 0) return;
  const size_t step = p.unit_heads;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + static_cast<size_t>(u.ticket) * 256 + group * 32 + lane;
  const float4* part = reinterpret_cast<const float4*>(p.part_o) + static_cast<size_t>(u.ticket) * (D / 4) * 256 + group * 32 + lane;
  float most = -CUDART_INF_F;
  for (int k0 = 0; k0 < n; k0 += 8) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k0 + k < n ? __ldcg(ml + (k0 + k) * step * 256).x : -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < 8; ++k) most = fmaxf(most, x[k]);
  }
  const float base = most == -CUDART_INF_F ? 0.f : most;
  for (int chunk = warp / groups; chunk < D / (4 * W); chunk += 8 / groups) {
    float sum = 0.f;
    float4 o[W];
#pragma unroll
    for (int j = 0; j < W; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < n; k0 += FLY) {
      float2 x[FLY];
      float4 v[FLY][W];
#pragma unroll
      for (int k = 0; k < FLY; ++k) {
        const bool in = k0 + k < n;
        x[k] = in ? __ldcg(ml + (k0 + k) * step * 256) : make_float2(-CUDART_INF_F, 0.f);
#pragma unroll
        for (int j = 0; j < W; ++j)
          v[k][j] = in ? __ldcg(part + ((k0 + k) * step * (D / 4) + chunk * W + j) * 256) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < FLY; ++k) {
        const float f = ex2_approx(x[k].x - base);
        sum = __fmaf_rn(x[k].y, f, sum);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          o[j].x = __fmaf_rn(v[k][j].x, f, o[j].x);
          o[j].y = __fmaf_rn(v[k][j].y, f, o[j].y);
          o[j].z = __fmaf_rn(v[k][j].z, f, o[j].z);
          o[j].w = __fmaf_rn(v[k][j].w, f, o[j].w);
        }
      }
    }
    const float inv = 1.0f / sum;
    uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + static_cast<size_t>(row) * D + chunk * 4 * W);
#pragma unroll
    for (int j = 0; j < W; j += 2)
      to[j / 2] = make_uint4(pack_bf16x2(o[j].x * inv, o[j].y * inv), pack_bf16x2(o[j].z * inv, o[j].w * inv),
                             pack_bf16x2(o[j + 1].x * inv, o[j + 1].y * inv), pack_bf16x2(o[j + 1].z * inv, o[j + 1].w * inv));
    if (chunk == 0 && p.lse) p.lse[row] = (most + log2f(sum)) * CUDART_LN2_F;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_prompt_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const __grid_constant__ PagedPromptParams p) {
  using C = PromptCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + C::OFF_KV;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_empty = q_full + 1;
  uint64_t* tail = q_full + 2;
  uint64_t* kv_full = q_full + 3;
  uint64_t* kv_empty = kv_full + C::NST;
  uint64_t* s_full = kv_empty + C::NST;
  uint64_t* s_free = s_full + 2;
  uint64_t* p_full = s_full + 4;
  uint64_t* o_done = s_full + 6;
  uint64_t* o_free = s_full + 8;
  uint64_t* fin = s_full + 10;
  uint64_t* join = s_full + 11;
  uint64_t* unit_full = s_full + 12;
  uint64_t* unit_empty = unit_full + kAhead;
  const Unit* units = reinterpret_cast<const Unit*>(smem + C::OFF_UNIT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + C::N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* is_last = abort_flag + 1;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(tail, 1);
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(kv_full + s, 1);
      mbar_init(kv_empty + s, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full + t, 1);
      mbar_init(s_free + t, 128);
      mbar_init(p_full + t, 128);
      mbar_init(o_done + t, 1);
      mbar_init(o_free + t, 128);
    }
    mbar_init(fin, 1);
    mbar_init(join, 8);
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(unit_full + i, 1);
      mbar_init(unit_empty + i, 11);  // the softmax warps, both producers and the MMA thread
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  uint32_t* err = p.err;
  grid_wait();
  // The units of this CTA, one after the other: a warp of its own finds them and leaves them in shared memory, ahead of
  // their use.  Whoever has taken what it needs of one says so (released).
  uint32_t n_unit = 0;
  auto next_unit = [&](const Unit** u) -> bool {
    if (!mbar_wait(unit_full + n_unit % kAhead, n_unit / kAhead & 1, abort_flag, err)) return false;
    *u = units + n_unit % kAhead;
    return (*u)->n_split > 0;
  };
  auto released = [&]() { mbar_arrive(unit_empty + n_unit++ % kAhead); };

  // Registers: 168 a thread at launch; 192 + 192 + 120 = 3 * 168.
  if (warp >= 8) {
    regs_dec<120>();
    if (warp == 8) {
      // ------------------------------------------------------------ K and V
      const int boxes = 128 >> p.shift;  // pages per key tile: lane l copies page l of it
      const int my_page = lane & (boxes - 1);
      const uint32_t in_tile = (my_page << p.shift) * (D * 2);
      uint32_t n_load = 0, n_tail = 0;
      bool ok = true;
      const Unit* next_one = nullptr;
      while (ok && next_unit(&next_one)) {
        const Unit u = *next_one;
        __syncwarp();
        if (lane == 0)
          released();
        else
          ++n_unit;
        const int n = max(u.n[0], u.n[1]);
        const int* table = p.tables + static_cast<size_t>(u.request) * p.width;
        // Page of this lane's box of key tile j of the unit.  It is asked for three tiles ahead and not looked at before
        // its use: a producer that waits for a table's entry leaves the ring empty.
        auto page_of = [&](int j) {
          const int i = (u.kv0 + j) * boxes + my_page;
          return j < n && i <= (u.length - 1) >> p.shift ? __ldcg(table + i) : 0;
        };
        auto load = [&](const CUtensorMap* map, int j, int page, bool is_v) -> bool {
          const int stage = static_cast<int>(n_load % C::NST);
          const uint32_t use = n_load / C::NST;
          ++n_load;
          if (use > 0 && !mbar_wait(kv_empty + stage, (use - 1) & 1, abort_flag, err)) return false;
          const int held = min(128, u.length - (u.kv0 + j) * 128);
          const int pages = (held + (1 << p.shift) - 1) >> p.shift;
          uint8_t* to = sKV + stage * C::KV_BYTES;
          uint64_t* bar = is_v && held < 128 ? tail : kv_full + stage;
          if (lane == 0) mbar_expect_tx(bar, (pages << p.shift) * 128 * C::KB);
          __syncwarp();
          if (lane < pages)
            tma_load_4d(to + in_tile, map, (clampi(page, 0, p.pages - 1) * p.kv_heads + u.kv_head) << (p.shift - 3), bar);
          if (bar == tail) {
            // values past the last row may be NaN, which a probability of 0 would not hide
            if (!mbar_wait(tail, n_tail++ & 1, abort_flag, err)) return false;
            for (int i = lane; i < (128 - held) * 8 * C::KB; i += 32) {
              const int row = held + i / (8 * C::KB), kb = i / 8 % C::KB;
              st_shared_v4(smem_u32(to) + ((row >> 3) * C::KB + kb) * 1024 + (row & 7) * 128 + (i & 7) * 16, 0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(kv_full + stage);
          }
          return true;
        };
        // consumption order: K_0, then (K_j, V_{j-1}) for j >= 1, then V_{n-1}
        int page = page_of(0), next = page_of(1), after = page_of(2), before = 0;
        for (int j = 0; j <= n && ok; ++j) {
          if (j < n) ok = load(&tk, j, page, false);
          if (ok && j >= 1) ok = load(&tv, j - 1, before, true);
          before = page;
          page = next;
          next = after;
          after = page_of(j + 3);
        }
      }
      // a wait that ran out: the copies in flight come to their end first, for a quarter of a second each at most
      volatile int no = 0;
      for (uint32_t li = ok || n_load < C::NST ? n_load : n_load - C::NST; li < n_load; ++li)
        mbar_wait(kv_full + li % C::NST, (li / C::NST) & 1, &no, err, 250000000ull);
    } else if (warp == 10 && elect_one()) {
      // ------------------------------------------------------------ queries
      uint32_t n_q = 0;
      bool ok = true;
      const Unit* ahead = nullptr;
      while (ok && next_unit(&ahead)) {
        const Unit u = *ahead;
        released();
        if (n_q > 0 && !(ok = mbar_wait(q_empty, (n_q - 1) & 1, abort_flag, err))) break;
        ++n_q;
        mbar_expect_tx(q_full, ((u.n[0] > 0) + (u.n[1] > 0)) * C::KB * 128 * p.tg * p.tt);
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (u.n[t] > 0)
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
              tma_load_3d(sQ + t * C::Q_BYTES + kb * C::BLK, &tq, kb * 64, u.head, u.first + u.token[t], q_full);
      }
      volatile int no = 0;  // a wait that ran out: the copies in flight come to their end first, for a quarter of a second at most
      if (!ok && n_q > 0) mbar_wait(q_full, (n_q - 1) & 1, &no, err, 250000000ull);
    } else if (warp == 9 && elect_one()) {
      // ------------------------------------------------------------ MMA issuer
      // The tensor pipe takes a product every 64 clocks and queues few: descriptors are sums of constants and a ring
      // index (built anew for each product they cost 10 %).
      constexpr uint32_t kIdescS = idesc_bf16(128, 0, 0);  // and the number of keys
      constexpr uint32_t kIdescO = idesc_bf16(128, D, 1);
      const uint64_t q_desc = smem_desc(smem_u32(sQ), 16, 1024);
      const uint64_t k_desc = smem_desc(smem_u32(sKV), 16, C::KB * 1024), v_desc = smem_desc(smem_u32(sKV), 1024, C::KB * 1024);
      uint32_t stage = 0, phase = 0, n_q = 0;  // of the ring's next entry; query tiles
      uint32_t n_s[2] = {0, 0}, n_pv[2] = {0, 0}, n_o[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag, err); };

      // S = Q_t K^T for the K tile of ring entry `at`, once the scores before it have been read
      int last = -1;  // query tile of the latest S
      auto s_mma = [&](int t, uint32_t at, int keys) -> bool {
        const int of = C::kTwoS ? t : last;
        if (of == 0 && n_s[0] > 0 && !wait(s_free, (n_s[0] - 1) & 1)) return false;
        if (of == 1 && n_s[1] > 0 && !wait(s_free + 1, (n_s[1] - 1) & 1)) return false;
        last = t;
        tc_fence_after();
        const uint32_t idesc = kIdescS + (static_cast<uint32_t>(keys >> 3) << 17);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          mma_bf16_ss(tmem + C::TMEM_S + (C::kTwoS ? t * 128 : 0), q_desc + ((t * C::Q_BYTES + (kk >> 2) * C::BLK + (kk & 3) * 32) >> 4),
                      k_desc + at * (C::KV_BYTES >> 4) + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), idesc, kk > 0);
        }
        mma_commit(s_full + t);
        ++n_s[t];
        return true;
      };
      // O_t (+)= P_t V for the V tile of ring entry `at`, once P_t is stored (and, for the
      // first tile of a unit, once the previous unit's O_t has been read out)
      auto pv_mma = [&](int t, uint32_t at, bool first, int keys) -> bool {
        if (first) {
          if (n_o[t] > 0 && !wait(o_free + t, (n_o[t] - 1) & 1)) return false;
          ++n_o[t];
        }
        if (!wait(p_full + t, n_pv[t] & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          if (kk * 16 >= keys) break;
          mma_bf16_ts(tmem + C::TMEM_O + t * D, tmem + C::TMEM_P + t * 64 + kk * 8,
                      v_desc + at * (C::KV_BYTES >> 4) + (kk * 2 * C::KB * 1024 >> 4), kIdescO, !first || kk > 0);
        }
        mma_commit(o_done + t);
        ++n_pv[t];
        return true;
      };
      // the ring's next entry (in load order), once its data is there
      auto kv_next = [&](uint32_t& at) -> bool {
        at = stage;
        if (!wait(kv_full + stage, phase)) return false;
        if (++stage == C::NST) {
          stage = 0;
          phase ^= 1;
        }
        return true;
      };

      const Unit* u = nullptr;
      while (ok && next_unit(&u)) {
        const int n0 = u->n[0], n1 = u->n[1], n = max(n0, n1), last0 = u->last[0], last1 = u->last[1];
        released();
        if (!(ok = wait(q_full, n_q++ & 1))) break;
        uint32_t ka = 0, va = 0;
        for (int j = 0; j <= n && ok; ++j) {
          // K_j; V_{j-1} follows it in the ring
          if (j < n && !(ok = kv_next(ka))) break;
          if (j < n0 && !(ok = s_mma(0, ka, j == n0 - 1 ? last0 : 128))) break;
          if (j >= 1 && !(ok = kv_next(va))) break;
          if (j >= 1 && j <= n0 && !(ok = pv_mma(0, va, j == 1, j == n0 ? last0 : 128))) break;
          if (j < n1 && !(ok = s_mma(1, ka, j == n1 - 1 ? last1 : 128))) break;
          if (j < n) mma_commit(kv_empty + ka);
          if (j == n - 1) mma_commit(q_empty);
          if (j >= 1) {
            if (j <= n1 && !(ok = pv_mma(1, va, j == 1, j == n1 ? last1 : 128))) break;
            mma_commit(kv_empty + va);
          }
        }
      }
      volatile int no = 0;  // the products in flight end before the tensor memory is freed, whatever happened
      mma_commit(fin);
      mbar_wait(fin, 0, &no, err);
    } else if (warp == 11 && elect_one()) {
      // ------------------------------------------------------------ units: in rounds over the list, forth and back
      const int total = *p.n_units * p.unit_heads;
      bool more = true;
      for (int round = 0; more; ++round) {
        const int at = round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        // the last round is not full: where it runs backwards, it is the first CTAs that have none
        Unit u{};
        more = at < total;
        if (more) u = unit_of(p, at);
        if (more && u.count > p.most) continue;
        if (n_unit >= kAhead && !mbar_wait(unit_empty + n_unit % kAhead, (n_unit / kAhead - 1) & 1, abort_flag, err)) break;
        reinterpret_cast<Unit*>(smem + C::OFF_UNIT)[n_unit % kAhead] = u;
        mbar_arrive(unit_full + n_unit++ % kAhead);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    regs_inc<192>();
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::TMEM_S + (C::kTwoS ? t * 128 : 0);
    const uint32_t tP = tmem + lane_off + C::TMEM_P + t * 64;
    const uint32_t tO = tmem + lane_off + C::TMEM_O + t * D;
    const int my_token = r / p.tg;
    uint32_t n_tiles = 0;  // of this query tile, over all units
    bool ok = true;
    uint32_t n_join = 0;
    // All eight warps come here; false if one of them does not.
    auto joined = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(join);
      return mbar_wait(join, n_join++ & 1, abort_flag, err);
    };
    const uint32_t out_tile = smem_u32(smem + C::OFF_OUT) + warp * 4096;
    auto out_at = [&](int row, int chunk) { return out_tile + row * 128 + ((chunk ^ (row & 7)) << 4); };
    const Unit* u = nullptr;
    while (ok && next_unit(&u)) {
      const int token = (t ? u->token[1] : u->token[0]) + my_token;
      const int n = t ? u->n[1] : u->n[0];
      const int row = row_of(p, *u, t, r);
      const int seen = u->length - u->count + min(token, u->count - 1) + 1 - u->kv0 * 128;  // keys of the range
      float ref = -CUDART_INF_F, sum = 0.f;
      for (int j = 0; j < n && ok; ++j) {
        if (!(ok = mbar_wait(s_full + t, (n_tiles + j) & 1, abort_flag, err))) break;
        tc_fence_after();
        float s[128];
        tmem_ld32(tS + 0, s);
        tmem_ld32(tS + 32, s + 32);
        tmem_ld32(tS + 64, s + 64);
        tmem_ld32(tS + 96, s + 96);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(s_free + t);
        const int valid = seen - j * 128;
        if (valid < 128) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= valid) s[c] = -CUDART_INF_F;
        }
        // row max as a tree of 3-input maxima (8 independent chains)
        float mk[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mk[k] = max3f(s[k], s[8 + k], s[16 + k]);
#pragma unroll
        for (int c = 24; c < 120; c += 16)
#pragma unroll
          for (int k = 0; k < 8; ++k) mk[k] = max3f(mk[k], s[c + k], s[c + 8 + k]);
#pragma unroll
        for (int k = 0; k < 8; ++k) mk[k] = fmaxf(mk[k], s[120 + k]);
        const float top = max3f(max3f(mk[0], mk[1], mk[2]), max3f(mk[3], mk[4], mk[5]), fmaxf(mk[6], mk[7])) * p.scale_log2;
        const bool rises = top > ref;
        float alpha = 1.0f;
        if (rises) {
          alpha = ex2_approx(ref - (top + kRise));
          ref = top + kRise;
        }
        float at = ref == -CUDART_INF_F ? 0.f : ref, factor = p.scale_log2;
        // The fused product of a score keeps the rounding of the reference in the exponent, half a unit in its last
        // place.  From 2^24 on, where that unit is a factor of 2 and more and the scores' own errors are larger still,
        // distances count as if the reference were below 2^24: the largest scores keep all the weight, and
        // everything stays finite.
        if (fabsf(at) > 16777216.f && fabsf(at) < CUDART_INF_F) {
          const float less = __int_as_float((127 + 23 + 127 - static_cast<int>((__float_as_uint(at) >> 23) & 0xffu)) << 23);
          at *= less;
          factor *= less;
        }
        uint32_t pk[64];
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // 8 independent partial sums
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          float a0, a1;
          fma2(a0, a1, s[c], s[c + 1], factor, -at);
          const float p0 = ex2_approx(a0);
          const float p1 = ex2_approx(a1);
          const int k = (c >> 1) & 3;
          add2(acc[2 * k], acc[2 * k + 1], p0, p1);
          pk[c >> 1] = pack_bf16x2(p0, p1);
        }
        sum = __fmaf_rn(sum, alpha, ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7])));
        if (j > 0) {
          if (!(ok = mbar_wait(o_done + t, (n_tiles + j - 1) & 1, abort_flag, err))) break;
          tc_fence_after();
          if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
            for (int cc = 0; cc < D; cc += 32) {
              float o[32];
              tmem_ld32(tO + cc, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= alpha;
              tmem_st32(tO + cc, o);
            }
          }
        }
        tmem_st32(tP, reinterpret_cast<const float*>(pk));
        tmem_st32(tP + 32, reinterpret_cast<const float*>(pk + 32));
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full + t);
      }
      // ---- the unit's last product
      if (ok && n > 0) {
        ok = mbar_wait(o_done + t, (n_tiles + n - 1) & 1, abort_flag, err);
        tc_fence_after();
      }
      n_tiles += n;
      if (u->n_split == 1) {
        // 64 features at a time go through shared memory and out in whole rows (a thread that stores its own row moves a
        // sector at a time, and all of them together take 4000 clocks)
        if (ok && n > 0) {
          const float inv = 1.0f / sum;
#pragma unroll
          for (int block = 0; block < C::KB; ++block) {
            float o[64];
            tmem_ld32(tO + block * 64, o);
            tmem_ld32(tO + block * 64 + 32, o + 32);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              st_shared_v4(out_at(lane, i), pack_bf16x2(o[8 * i] * inv, o[8 * i + 1] * inv),
                           pack_bf16x2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                           pack_bf16x2(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                           pack_bf16x2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r4 = i * 4 + (lane >> 3), to = __shfl_sync(0xffffffffu, row, r4);
              const uint4 x = ld_shared_v4(out_at(r4, lane & 7));
              if (to >= 0) static_cast<uint4*>(p.out)[static_cast<size_t>(to) * (D / 8) + block * 8 + (lane & 7)] = x;
            }
            __syncwarp();
          }
          if (row >= 0 && p.lse) p.lse[row] = (ref + log2f(sum)) * CUDART_LN2_F;
        }
      } else if (ok) {
        // partial results lie [4 features][row]: a warp's rows side by side
        float4* part = reinterpret_cast<float4*>(p.part_o) + static_cast<size_t>(u->slot) * (256 * D / 4) + threadIdx.x;
#pragma unroll
        for (int cc = 0; cc < D; cc += 32) {
          float o[32];
          if (n > 0) {
            tmem_ld32(tO + cc, o);
            tmem_wait_ld();
          }
          if (row >= 0)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              part[(cc / 4 + i) * 256] = n > 0 ? make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3])
                                               : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (row >= 0)
          reinterpret_cast<float2*>(p.part_ml)[static_cast<size_t>(u->slot) * 256 + threadIdx.x] = make_float2(ref, sum);
      }
      if (n > 0) {
        tc_fence_before();
        mbar_arrive(o_free + t);
      }
      if (u->n_split > 1) {
        if (!(ok = ok && joined())) break;
        if (threadIdx.x == 0) {
          unsigned* ticket = p.tickets + u->ticket;
          unsigned before;
          // releases the CTA's partial results (ordered before by the barrier) and acquires the others'
          asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(ticket) : "memory");
          *is_last = before == static_cast<unsigned>(u->n_split - 1);
          if (*is_last) *ticket = 0;
        }
        if (!(ok = joined())) break;
        if (*is_last) {
          const int rows = u->token[1] < u->count ? 256 : (u->count - u->token[0]) * p.tg;  // at most
          if (rows > 64)
            merge<D, 8, 2>(p, *u, rows > 128 ? 8 : 4);
          else
            merge<D, 4, 4>(p, *u, rows > 32 ? 2 : 1);
        }
      }
      __syncwarp();
      if (lane == 0)
        released();
      else
        ++n_unit;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t paged_prompt_configure(int head_dim) {
  return head_dim == 128 ? cudaFuncSetAttribute(paged_prompt_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                PromptCfg<128>::SMEM)
                         : cudaFuncSetAttribute(paged_prompt_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                PromptCfg<64>::SMEM);
}

cudaError_t launch_paged_prompt(int head_dim, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                const PagedPromptParams& p, int sms, cudaStream_t s) {
  return head_dim == 128
             ? launch_kernel(paged_prompt_kernel<128>, sms, kThreads, PromptCfg<128>::SMEM, s, 1, q, k, v, p)
             : launch_kernel(paged_prompt_kernel<64>, sms, kThreads, PromptCfg<64>::SMEM, s, 1, q, k, v, p);
}

}  // namespace ff
