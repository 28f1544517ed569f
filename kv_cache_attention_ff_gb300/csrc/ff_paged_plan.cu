// A step's plan on the GPU (pages of every request, places of the new rows) and
// the rows' way into their places.
#include <algorithm>
#include <climits>

#include <cooperative_groups.h>
#include <math_constants.h>

#include "ff_kv8.h"
#include "ff_launch.cuh"
#include "ff_paged.h"
#include "ff_paged.cuh"

namespace ff {
namespace {

// --------------------------------------------------------------------- plan
//
// A cluster of blocks.  Every block works out all requests' prefix sums (rows,
// pages given back, pages taken) in its own shared memory: they are few, and it
// saves handing them round.  The pages that move and the new rows are then
// spread over all threads, which find their request by binary search.  The k-th
// page taken is the k-th given back, as long as there are some, so that no block waits for
// another but at the end, before lengths change; two of them list the attention's work
// meanwhile.  A chain of scans and dependent loads bounds it: 7 us for 128 decoding
// requests of 8 kv heads (10 of one, whose key ranges' length is sought), 10 for 300 of which a
// fifth are prompts of up to 1111 rows.
constexpr int kPlanThreads = 1024;
constexpr int kPlanBlocks = 8;
constexpr unsigned kTop = 1u << 30;  // prefix sums saturate here

size_t plan_smem(int requests) { return (static_cast<size_t>(requests) * 6 + 4) * sizeof(int); }

// Exclusive prefix sums of N values of each of the block's threads, each sum at most `top` (2^30 or less), and their totals.
// sh: 32 N words.
template <int N>
__device__ __forceinline__ void block_scan(unsigned (&x)[N], unsigned top, unsigned* sh, unsigned (&total)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned run[N], w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) run[i] = min(x[i], top);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned y = __shfl_up_sync(0xffffffffu, run[i], o);
      if (lane >= o) run[i] = min(run[i] + y, top);
    }
  __syncthreads();  // the sums of the scan before this one have been read
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < N; ++i) sh[i * 32 + warp] = run[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = sh[i * 32 + lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned y = __shfl_up_sync(0xffffffffu, w[i], o);
      if (lane >= o) w[i] = min(w[i] + y, top);
    }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    total[i] = __shfl_sync(0xffffffffu, w[i], 31);
    const unsigned before = __shfl_sync(0xffffffffu, w[i], max(warp - 1, 0));
    const unsigned mine = __shfl_up_sync(0xffffffffu, run[i], 1);
    x[i] = min((warp ? before : 0u) + (lane ? mine : 0u), top);
  }
}
__device__ __forceinline__ unsigned block_scan(unsigned x, unsigned top, unsigned* sh, unsigned* total) {
  unsigned v[1] = {x}, all[1];
  block_scan(v, top, sh, all);
  *total = all[0];
  return v[0];
}

// The token form's pieces.  All key ranges are of about equal length, X stages: the
// least with which they all run at once, or with more work some waves of them, which
// the GPU hands out as thread blocks end.  Then not less than
//  - what the merge costs: a range of X stages and L / X ranges to merge, each as much as
//    0.06 stages and 0.13 for every row, cost least together at the root of their product;
//  - the time in which the memory delivers everything, in stages of one block: 115 blocks draw as
//    much as there is (152 SMs have two each), so ranges of that length cost nothing, but that long ones end apart, by a
//    tenth of their time: 3.2 times the root at most.  A merge costs 20 stages and one for every row besides; a request
//    that is not longer than both is one piece, in steps that are not long themselves.
// Ranges of cut requests come first: a long one that begins late ends late.
// Of 280 steps (one to 512 requests, 100 to 60000 keys), with the time of 24 lengths each, this takes on average 1.1 %
// more than the least; 10000 keys of one kv head and eight query heads 12.5 us (157 ranges 24 to 30).
constexpr float kStageRate = 115.f;  // of head_dim 128
constexpr float kShortStep = 300.f;  // stages
template <class Holds>
__device__ void list_tokens(const PagedPlanParams& p, const int* first, const int* kept, int* list, unsigned* scan,
                            const Holds& holds) {
  const PagedState& s = p.s;
  const int R = s.requests, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int best;
  // list[r]: stages of request r if it takes the token form
  unsigned requests = 0;
  unsigned long long stages = 0;
  int most = 0, rows = 0;
  for (int r0 = 0; r0 < R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    int n = 0;
    if (r < R) {
      const int length = holds(r), news = length - kept[r];
      if (news > 0 && news <= kPagedTokenRows / p.group) {
        n = (length + kPagedStage - 1) / kPagedStage;
        rows = max(rows, news * p.group);
      }
      list[r] = n;
    }
    requests += __syncthreads_count(n > 0);
    stages += n;
    most = max(most, n);
  }
  if (tid == 0) *s.n_pieces = 0;
  if (requests == 0) return;
  __shared__ unsigned long long all;  // not saturated: the number of pieces hangs on it
  __shared__ int longest, most_rows;
  if (tid == 0) all = longest = most_rows = 0;
  __syncthreads();
#pragma unroll
  for (int o = 16; o; o >>= 1) stages += __shfl_xor_sync(0xffffffffu, stages, o);
  most = __reduce_max_sync(0xffffffffu, most);
  rows = __reduce_max_sync(0xffffffffu, rows);
  if (lane == 0) {
    atomicAdd(&all, stages);
    atomicMax(&longest, most);
    atomicMax(&most_rows, rows);
  }
  __syncthreads();
  const int at_once = max(1, p.token_blocks / p.kv_heads);
  const unsigned long long waves = static_cast<unsigned long long>(kPagedWaves) * p.token_blocks;
  int x = static_cast<int>(min((all * p.kv_heads + waves - 1) / waves, 1ull << 20));  // no request has more stages than that
  x = max(x, kPagedRange);
  if (requests <= static_cast<unsigned>(at_once)) {
    // 32 candidates at a time: the least of them with which the pieces run at once
    int lo = 0, hi = kPagedRange;  // in (lo, hi], if there is one
    auto fits = [&](int candidate) {
      int n = 0;
      for (int r = lane; r < R; r += 32) n += (list[r] + candidate - 1) / candidate;
      return static_cast<int>(__reduce_add_sync(0xffffffffu, n)) <= at_once;
    };
    if (tid == 0) best = hi + 1;
    __syncthreads();
    while (lo < hi) {
      const int candidate = lo + max(1, static_cast<int>(static_cast<long long>(hi - lo) * (warp + 1) / 32));
      const bool ok = fits(candidate);
      __syncthreads();
      if (lane == 0 && ok) atomicMin(&best, candidate);
      __syncthreads();
      const int found = best;
      if (found > hi) break;
      // the candidate before the one found does not fit
      int below = lo;
      for (int w = 0; w < 32; ++w) {
        const int c = lo + max(1, static_cast<int>(static_cast<long long>(hi - lo) * (w + 1) / 32));
        if (c < found) below = c;
      }
      lo = below;
      hi = found;
      if (hi - lo <= 1) break;
    }
    if (best <= kPagedRange) x = best;
  }
  const float root = sqrtf((0.06f + 0.13f * most_rows) * longest);
  x = max(x, max(static_cast<int>(root * 0.25f + 0.5f), 1) * 4);  // the warps take four at a time
  const float time = static_cast<float>(all) * p.kv_heads * (p.head_dim / 128.f) / kStageRate;
  x = max(x, static_cast<int>(fminf(time, 3.2f * root)));
  if (time <= kShortStep && longest <= time + 20.f + most_rows) x = max(x, longest);
  unsigned parts = 0, whole = 0, cut[2];  // ranges of cut requests, and requests that are not
  for (int r0 = 0; R > kPlanThreads && r0 < R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    const int n = r < R ? (list[r] + x - 1) / x : 0;
    unsigned at[2] = {n > 1 ? static_cast<unsigned>(n) : 0u, n == 1};
    block_scan(at, kTop, scan, cut);
    whole += cut[0];
  }
  for (int r0 = 0; r0 < R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    const int n = r < R ? (list[r] + x - 1) / x : 0;
    unsigned at[2] = {n > 1 ? static_cast<unsigned>(n) : 0u, n == 1};
    block_scan(at, kTop, scan, cut);
    if (R <= kPlanThreads) whole = cut[0];
    const unsigned part = parts + at[0], item = n > 1 ? part : whole + at[1];
    parts += cut[0];
    whole += cut[1];
    if (n) {
      PagedPiece piece{r, first[r], 0, holds(r), 0, n, static_cast<int>(part), 0};
      piece.count = piece.length - kept[r];
      for (int i = 0; i < n; ++i) {
        piece.split = i;
        s.pieces[item + i] = piece;
      }
    }
  }
  if (tid == 0) *s.n_pieces = whole;
}

// The prompt form's units: blocks of two query tiles, longest first.  CTAs take them in
// rounds, forth and back, so a full round costs its mean and the last one, if it is not
// full, its longest.  Blocks of more than X tiles are cut into equal key ranges: each of 16 warps
// works out what one X would cost (none cut, or the longest in up to 90 ranges), the
// least wins.  All ranges of cut blocks together are at most kPagedRounds rounds, for which
// there is room.  With more rounds than that blocks are cut only where one is longer than a CTA's share; other 16 warps
// look at the last round, if it is not full, cut alone.  9728 rows
// behind 21472 of 8 heads are two even rounds; of 4680 behind 26520 of 12 heads (228 units of 209 to 244
// tiles) every block is cut in two: 687 us before, 520 after.  64 requests of three rows with 64/8 heads over 503 keys, but
// one over 30003: 70 us, 294 where nothing is cut; 200 tokens over 900 keys, one over 120000 and 64 new rows, 32/8 heads: 265,
// 1180 uncut.  Four chunks of 1024 behind 16000, 32/8 heads (3.4 rounds): 680 us, 734 with a whole last round; 20 requests of
// nine rows behind 30000, 64/8 heads (1.1 rounds) 363 and 460.  The search itself takes 3 us.
constexpr int kBuckets = 1024;
constexpr int kCandidates = 16;
// In key tiles, found from 110 steps (one request to 200, one new row to 16384) with each of the 16 lengths: the least cost
// is on average 0.2 % above the least time.
constexpr float kPieceCost = 3.f;   // of a piece's start and end
constexpr float kMergeCost = 4.f;   // of one more pass over partial results, and an eighth for every range,
constexpr float kRowCost = 0.13f;   // and for every range and eighth of a block's rows, of the CTA that merges most
constexpr float kPartCost = 0.4f;   // and of all CTAs
constexpr int kMostCut = 480;       // blocks of which the costs are worked out: a warp holds them
constexpr int kTailRounds = 8;      // rounds up to which the last one is worth a look,
constexpr int kTailTiles = 16;      // of longer blocks than this,
constexpr float kTailGain = 1.03f;  // and a cut for more than what the estimate is worth

// A block of rows in the lists below: its key tiles (up to 2^17), and how many eighths of two query tiles its rows are.
constexpr int kTileBits = 24;
__device__ __forceinline__ int tiles_of(int block) { return block & ((1 << kTileBits) - 1); }
__device__ __forceinline__ int eighths_of(int block) { return block >> kTileBits; }

// ceil(t / x) for 1 <= t <= 2^17: the half keeps a multiple of x on its side of the rounding.
__device__ __forceinline__ int ceil_div(int t, float inv_x) { return static_cast<int>((static_cast<float>(t) - 0.5f) * inv_x) + 1; }

// How blocks are cut: those of more than x tiles, and the last `tail` ones into `ways` ranges.
struct Cut {
  int x, tail, ways;
};

// What the pieces cost, in key tiles; a warp's lanes work together.
__device__ __forceinline__ float cost_of(const unsigned* list, int blocks, const Cut& by, int heads, int sms, int longest) {
  constexpr int N = kMostCut / 32;
  const int lane = threadIdx.x & 31;
  const float inv_x = __frcp_rn(static_cast<float>(by.x));
  int t[N], q[N], m[N], worst = 0, moved = 0;  // eighths of rows in ranges that are merged
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = q[i] = m[i] = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i * 32 >= blocks) break;
    const int e = i * 32 + lane;
    if (e < blocks) {
      const int block = list[e];
      t[i] = tiles_of(block);
      m[i] = e < blocks - by.tail ? ceil_div(t[i], inv_x) : min(by.ways, t[i]);
      q[i] = ceil_div(t[i], __frcp_rn(static_cast<float>(m[i])));
      if (m[i] > 1) {
        worst = max(worst, m[i] * eighths_of(block));
        moved += m[i] * eighths_of(block);
      }
    }
  }
  auto sums = [&](int least, float* n, float* work) {  // pieces of at least that many tiles
    int a = 0, b = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i * 32 >= blocks) break;
      a += q[i] >= least ? m[i] : 0;
      b += q[i] >= least ? t[i] : 0;
    }
    *n = static_cast<float>(__reduce_add_sync(0xffffffffu, a)) * heads;
    *work = static_cast<float>(__reduce_add_sync(0xffffffffu, b)) * heads;
  };
  float pieces, work;
  sums(0, &pieces, &work);
  const bool cut = by.x < longest || by.tail;
  const float full = floorf(pieces / sms) * sms, rounds = ceilf(pieces / sms);
  if (by.x < longest && rounds > kPagedRounds) return CUDART_INF_F;
  float cost = work / sms;
  if (full < pieces) {
    // the length of the longest piece of the last round: the largest with more than `full` pieces of at least it
    int lo = 1, hi = by.x + 1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      float n, w;
      sums(mid, &n, &w);
      if (n > full)
        lo = mid;
      else
        hi = mid;
    }
    float n, w;
    sums(hi, &n, &w);
    cost = (w + lo * (full - n)) / sms + lo;
  }
  return (cost + rounds * kPieceCost) * (by.tail ? kTailGain : 1.f) +
         (cut ? kMergeCost + 0.125f * (by.tail ? by.ways : static_cast<float>(longest) / by.x) +
                    kRowCost * __reduce_max_sync(0xffffffffu, worst) + kPartCost * __reduce_add_sync(0xffffffffu, moved) * heads / sms
              : 0.f);
}

// The same where one block is longer than a CTA's share of the work: the share or, if that is more, what the CTA with the
// longest piece has at least.
__device__ __forceinline__ float cost_of_uneven(const int* list, int blocks, int x, int heads, int sms, int longest) {
  const int lane = threadIdx.x & 31;
  const float inv_x = __frcp_rn(static_cast<float>(x));
  int n = 0, n_cut = 0, most = 0, fewest = INT_MAX, worst = 0;
  float work = 0.f, moved = 0.f;
  for (int e = lane; e < blocks; e += 32) {
    const int block = list[e], t = tiles_of(block), m = ceil_div(t, inv_x), q = ceil_div(t, __frcp_rn(static_cast<float>(m)));
    n += m;
    if (m > 1) {
      n_cut = min(n_cut + m, 1 << 24);
      moved += static_cast<float>(m * eighths_of(block));
      worst = max(worst, m * eighths_of(block));
    }
    most = max(most, q);
    fewest = min(fewest, q);
    work += static_cast<float>(t);
  }
  n_cut = __reduce_add_sync(0xffffffffu, n_cut);
  if (static_cast<long long>(n_cut) * heads > kPagedRounds * sms) return CUDART_INF_F;
  most = __reduce_max_sync(0xffffffffu, most);
  fewest = __reduce_min_sync(0xffffffffu, fewest);
  const float pieces = static_cast<float>(__reduce_add_sync(0xffffffffu, n)), rounds = ceilf(pieces * heads / sms);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    work += __shfl_xor_sync(0xffffffffu, work, o);
    moved += __shfl_xor_sync(0xffffffffu, moved, o);
  }
  return fmaxf(work * heads / sms, most + (rounds - 1.f) * fewest) + rounds * kPieceCost +
         (x < longest ? kMergeCost + 0.125f * longest / x + kRowCost * __reduce_max_sync(0xffffffffu, worst) +
                            kPartCost * moved * heads / sms
                      : 0.f);
}

template <class Holds>
__device__ void list_prompts(const PagedPlanParams& p, const int* first, const int* kept, int* list, unsigned* scan,
                             const Holds& holds) {
  const PagedState& s = p.s;
  const int R = s.requests, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ unsigned long long least, work;
  __shared__ int longest;
  __shared__ unsigned place[kBuckets];
  static_assert(kBuckets == kPlanThreads, "a thread has a bucket");
  // list[r]: blocks of the requests before r
  unsigned total, run = 0;
  for (int r0 = 0; r0 < R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    const int n = r < R ? (holds(r) - kept[r] + p.block_tokens - 1) / p.block_tokens : 0;
    const unsigned before = block_scan(n, kTop, scan, &total);
    if (r < R) list[r] = run + before;
    run += total;
  }
  if (tid == 0) {
    list[R] = run;
    *s.n_units = 0;
    least = ~0ull;
    work = longest = 0;
  }
  place[tid] = 0;
  __syncthreads();
  const int blocks = run;
  if (blocks == 0) return;
  int most = 0;
  unsigned sum = 0;
  bool many = false;  // rows of a request, more than the token form takes
  int own = 0;        // block tid
  auto block_at = [&](int e) { return e == tid ? own : s.tiles[e]; };
  for (int e = tid; e < blocks; e += kPlanThreads) {
    const int r = last_at_most(list, R, e), length = holds(r), news = length - kept[r];
    const int to = min(news, (e - list[r] + 1) * p.block_tokens);  // of its new rows
    const int n = (length - news + to + 127) / 128;
    const int block = n | ((to - (e - list[r]) * p.block_tokens) * 8 + p.block_tokens - 1) / p.block_tokens << kTileBits;
    s.tiles[e] = block;
    if (e == tid) own = block;
    most = max(most, n);
    sum = min(sum + n, 1u << 26);
    many |= news > kPagedTokenRows / p.group;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) {
    atomicMax(&longest, most);
    atomicAdd(&work, static_cast<unsigned long long>(sum));
  }
  many = __syncthreads_or(many);
  Cut by{longest, 0, 1};
  const long long units = static_cast<long long>(blocks) * p.unit_heads;
  const bool uneven = units > p.sms && static_cast<float>(longest) * p.sms > (work + kPieceCost * blocks) * p.unit_heads;
  const bool few = units <= static_cast<long long>(kPagedRounds) * p.sms;
  // The last round: how many blocks, and in how many ranges all of them still are one.
  const int tail = units > p.sms ? (static_cast<int>(units) % p.sms + p.unit_heads - 1) / p.unit_heads : 0;
  const int ways = tail ? p.sms / (tail * p.unit_heads) : 0;
  const bool last = ways > 1 && units <= static_cast<long long>(kTailRounds) * p.sms && longest > kTailTiles && many;
  if (uneven || (blocks <= kMostCut && (few || last))) {
    if (!uneven)
      if (tid < blocks) place[tid] = own;
    __syncthreads();
    auto candidate = [&](int i) {
      if (i < kCandidates) {
        // the longest in 1, 1.5, .. 3.5 ranges, then in 41 % more each
        const float ranges = i < 6 ? 1.f + 0.5f * i : exp2f(2.f + 0.5f * (i - 6));
        return Cut{clampi(static_cast<int>(ceilf(static_cast<float>(longest) / ranges)), 1, longest), 0, 1};
      }
      // the blocks of the last round in two to nine ranges, then 13, 17, ..
      i -= kCandidates;
      return Cut{longest, tail, i < 8 ? 2 + i : 4 * i - 19};
    };
    // the warps of those that cannot be taken leave the others their turns
    const Cut mine = candidate(warp);
    if (warp < kCandidates ? warp == 0 || uneven || few : !uneven && mine.ways <= ways) {
      const float cost = uneven ? cost_of_uneven(s.tiles, blocks, mine.x, p.unit_heads, p.sms, longest)
                                : cost_of(place, blocks, mine, p.unit_heads, p.sms, longest);
      // the least cost, of equal ones the first (costs are positive: their bits are in their order)
      if (lane == 0) atomicMin(&least, static_cast<unsigned long long>(__float_as_uint(cost)) << 32 | static_cast<unsigned>(warp));
    }
    __syncthreads();
    by = candidate(static_cast<int>(least & 0xffffffffu));
    place[tid] = 0;
    __syncthreads();
  }
  int shift = 0;
  while ((longest >> shift) >= kBuckets) ++shift;
  const float inv_x = __frcp_rn(static_cast<float>(by.x));
  auto pieces_of = [&](int e, int tiles) {  // one each where x is the longest
    return e >= blocks - by.tail ? min(by.ways, tiles) : tiles <= by.x ? 1 : ceil_div(tiles, inv_x);
  };
  auto bucket_of = [&](int tiles, int pieces) { return kBuckets - 1 - ((tiles + pieces - 1) / pieces >> shift); };
  for (int e = tid; e < blocks; e += kPlanThreads) {
    const int tiles = tiles_of(block_at(e)), n = pieces_of(e, tiles);
    atomicAdd(place + bucket_of(tiles, n), n);
  }
  __syncthreads();
  const unsigned mine = place[tid], before = block_scan(mine, kTop, scan, &total);
  place[tid] = before;
  if (tid == 0) *s.n_units = total;
  __syncthreads();
  unsigned parts = 0;
  for (int e0 = 0; e0 < blocks; e0 += kPlanThreads) {
    const int e = e0 + tid;
    const int tiles = e < blocks ? tiles_of(block_at(e)) : 0, n = e < blocks ? pieces_of(e, tiles) : 0;
    const unsigned part = parts + block_scan(n > 1 ? n : 0, kTop, scan, &total);
    parts += total;
    if (n) {
      const int r = last_at_most(list, R, e);
      PagedPiece piece{r, first[r], 0, holds(r), 0, n, static_cast<int>(part), e - list[r]};
      piece.count = piece.length - kept[r];
      const unsigned to = atomicAdd(place + bucket_of(tiles, n), n);
      for (int i = 0; i < n; ++i) {
        piece.split = i;
        s.units[to + i] = piece;
      }
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PagedPlanParams p) {
  extern __shared__ int sm[];
  __shared__ unsigned scan[64];
  const PagedState& s = p.s;
  const int R = s.requests;
  int* first = sm;             // [R + 1]
  int* back = first + R + 1;   // [R + 1] pages given back by the requests before
  int* take = back + R + 1;    // [R + 1] pages wanted by the requests before
  int* kept = take + R + 1;    // [R] rows that stay
  int* had = kept + R;         // [R] pages
  int* list = had + R;         // [R + 1] of the blocks that list work
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const int tid = threadIdx.x;
  const int at = cluster.block_rank() * kPlanThreads + tid;
  constexpr int step = kPlanBlocks * kPlanThreads;
  grid_wait();

  const int n_free = clampi(*s.n_free, 0, s.pages);
  bool dropped = false;
  unsigned run = 0, total;
  for (int r0 = 0; r0 < R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    unsigned c = 0;
    if (r < R) {
      const int held = clampi(s.lengths[r], 0, s.capacity);
      kept[r] = p.start ? clampi(p.start[r], 0, held) : held;
      had[r] = pages_of(s, held);
      const int asked = p.counts[r];
      c = clampi(asked, 0, p.n);
      dropped |= asked > p.n;
    }
    const unsigned before = min(run + block_scan(c, p.n, scan, &total), static_cast<unsigned>(p.n));
    if (r < R) first[r] = before;
    dropped |= before + c > static_cast<unsigned>(p.n);
    run = min(run + total, static_cast<unsigned>(p.n));
  }
  if (tid == 0) first[R] = run;
  __syncthreads();
  // rows that request r would hold
  auto wanted = [&](int r) { return min(kept[r] + (first[r + 1] - first[r]), s.capacity); };
  unsigned run_back = 0, run_take = 0;
  for (int r0 = 0; r0 < R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    int more = 0;
    if (r < R) more = pages_of(s, wanted(r)) - had[r];
    unsigned x[2] = {static_cast<unsigned>(max(-more, 0)), static_cast<unsigned>(max(more, 0))}, all[2];
    block_scan(x, kTop, scan, all);
    if (r < R) {
      back[r] = min(run_back + x[0], kTop);
      take[r] = min(run_take + x[1], kTop);
    }
    run_back = min(run_back + all[0], kTop);
    run_take = min(run_take + all[1], kTop);
  }
  if (tid == 0) {
    back[R] = run_back;
    take[R] = run_take;
  }
  __syncthreads();
  const int top = static_cast<int>(min(n_free + run_back, static_cast<unsigned>(s.pages)));  // of the stack, all pages given back
  // rows that request r holds in the end
  auto holds = [&](int r) {
    const int want = wanted(r), taken = pages_of(s, want) - had[r];
    return taken <= 0 ? want : min(want, (had[r] + clampi(top - take[r], 0, taken)) << s.shift);
  };
  const int n_back = min(top, static_cast<int>(run_back)), n_take = min(top, static_cast<int>(run_take));
  // The k-th page given back, and the k-th taken: that very page, or once those are used up one that was free before.
  auto given_back = [&](int k) {
    const int r = last_at_most(back, R, k);
    return page_at(s, r, pages_of(s, wanted(r)) + (k - back[r]));
  };
  auto taken = [&](int k) { return k < n_back ? given_back(k) : clampi(__ldcg(s.free + (top - 1 - k)), 0, s.pages - 1); };

  // Nobody reads what another block writes here: the stack above the pages that were free, tables behind the pages that a
  // request had.  Only lengths and the stack's height wait until all blocks have read them.
  const int rank = cluster.block_rank();
  if (rank == kPlanBlocks - 1) {
    list_tokens(p, first, kept, list, scan, holds);
  } else if (rank == kPlanBlocks - 2) {
    list_prompts(p, first, kept, list, scan, holds);
  } else {
    constexpr int spread = step - 2 * kPlanThreads;
    for (int i = at; i < p.n; i += spread) {
      int slot = -1, position = 0;
      if (i < first[R]) {
        const int r = last_at_most(first, R, i);
        const int x = kept[r] + (i - first[r]), page = x >> s.shift;
        if (x < holds(r)) {
          position = x;
          slot = ((page < had[r] ? page_at(s, r, page) : taken(take[r] + page - had[r])) << s.shift) + (x & ((1 << s.shift) - 1));
        }
      }
      s.slots[i] = slot;
      s.positions[i] = position;
    }
    for (int k = at; k < n_take; k += spread) {
      const int r = last_at_most(take, R, k);
      s.tables[static_cast<size_t>(r) * s.width + had[r] + (k - take[r])] = taken(k);
    }
    for (int k = at; k < n_back; k += spread) s.free[top - 1 - k] = given_back(k);
  }
  cluster.sync();
  if (rank == 0) {
    for (int r = tid; r < R; r += kPlanThreads) {
      const int length = holds(r);
      s.lengths[r] = length;
      s.first[r] = first[r];
      dropped |= length < kept[r] + (first[r + 1] - first[r]);
    }
    if (tid == 0) {
      s.first[R] = first[R];
      *s.n_free = top - n_take;
    }
    if (__syncthreads_or(dropped) && tid == 0) atomicOr(p.err, kErrCapacity);
  }
}

// -------------------------------------------------------------------- store
//
// 16-byte units of rows, K and V by the same thread.  Memory bounds it: 4682 rows of 40
// heads at d 128 (96 MB in, as much out) 30.7 us, 6.25 TB/s; 64 rows of 8 heads 1.4 us.
constexpr int kStoreThreads = 256;

__global__ void __launch_bounds__(kStoreThreads) paged_store_kernel(const __grid_constant__ PagedStoreParams p) {
  const unsigned per_head = p.head_dim / 8, per_row = p.kv_heads * per_head;
  const unsigned i = blockIdx.x * kStoreThreads + threadIdx.x;
  grid_wait();
  if (i >= p.n * per_row) return;
  const unsigned row = i / per_row, unit = i - row * per_row;
  const int slot = p.slots[row];
  if (static_cast<int>(row) >= *p.total || slot < 0 || (slot >> p.shift) >= p.pages) return;
  const uint4 k = __ldcs(static_cast<const uint4*>(p.k) + i), v = __ldcs(static_cast<const uint4*>(p.v) + i);
  const unsigned page = slot >> p.shift, h = unit / per_head;
  const size_t to = (((static_cast<size_t>(page) * p.kv_heads + h) << p.shift) + (slot & ((1 << p.shift) - 1))) * per_head +
                    (unit - h * per_head);
  static_cast<uint4*>(p.k_pool)[to] = k;
  static_cast<uint4*>(p.v_pool)[to] = v;
}

}  // namespace

cudaError_t paged_plan_configure() {
  return cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(plan_smem(kPagedRequests)));
}

cudaError_t launch_paged_plan(const PagedPlanParams& p, cudaStream_t s) {
  return launch_kernel(paged_plan_kernel, kPlanBlocks, kPlanThreads, plan_smem(p.s.requests), s, kPlanBlocks, p);
}

cudaError_t launch_paged_store(const PagedStoreParams& p, cudaStream_t s) {
  const unsigned units = static_cast<unsigned>(p.n) * p.kv_heads * (p.head_dim / 8);
  return launch_kernel(paged_store_kernel, (units + kStoreThreads - 1) / kStoreThreads, kStoreThreads, 0, s, 1, p);
}

}  // namespace ff
