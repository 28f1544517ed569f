// Structures shared by the host side of the paged cache (ff_paged.cpp) and its kernels.
//
// A layer's pool holds `pages` pages of page_rows rows: bf16
// [pages][kv_heads][page_rows][head_dim] for K and V each, so that a head's rows
// of a page are one contiguous run (4 KB at 16 rows and head_dim 128).  One set of
// tables serves all layers.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace ff {

// A piece of a step's work: a key range of one request, for the prompt form of one
// block of its new rows.  Its kv heads are units of their own.
struct __align__(16) PagedPiece {
  int request, first, count, length;  // its packed rows, the rows that it holds
  int split, n_split;                 // key range `split` of n_split
  int part;                           // n_split > 1: place of the first range among the partial results
  int block;                          // prompt form: two query tiles
};

struct PagedState {
  int* tables;     // [requests][width] pages of each request, in order
  int* lengths;    // [requests] rows held
  int* first;      // [requests + 1] where each request's rows begin in the packed buffers
  int* free;       // [pages] stack of the pages that no request has
  int* n_free;     // [1]
  int* slots;      // [max_rows] page * page_rows + row, or -1
  int* positions;  // [max_rows]
  PagedPiece* pieces;  // [piece_cap] the token form's work of the latest step
  int* n_pieces;   // [1]
  PagedPiece* units;   // [unit_cap] the prompt form's, longest first
  int* n_units;    // [1]
  int* tiles;      // [unit_cap] scratch of the plan: key tiles and rows of every block of rows
  int requests, width, pages, capacity;
  int shift;       // page_rows = 1 << shift
};

struct PagedPlanParams {
  PagedState s;
  const int* start;   // [requests] or null: the rows held
  const int* counts;  // [requests]
  int n;              // rows of the packed buffers
  int kv_heads, group, head_dim;
  int token_blocks;   // thread blocks of the token form that run at once
  int sms;
  int block_tokens;   // tokens of two query tiles of the prompt form
  int unit_heads;     // units of a block of rows: kv heads times tiles of a group's heads
  unsigned int* err;
};

struct PagedStoreParams {
  const void* k;  // bf16 [n, kv_heads, d]
  const void* v;
  void* k_pool;
  void* v_pool;
  const int* slots;
  const int* total;  // rows of the step: slots behind them are of earlier steps
  int n, kv_heads, head_dim, pages, shift;
};

struct PagedTokenParams {
  const PagedPiece* pieces;
  const int* n_pieces;
  const int* tables;
  float* part_o;          // [parts][kv_heads][8][d]
  float* part_ml;         // [parts][kv_heads][8][2] reference (log2 units) and sum
  unsigned int* tickets;  // [requests][kv_heads] finished ranges (0 between launches)
  const void* q;
  void* out;
  float* lse;
  int n, most, kv_heads, group, width, pages, shift;
  float scale_log2;
  unsigned int* err;
};

struct PagedPromptParams {
  const PagedPiece* units;
  const int* n_units;
  const int* tables;
  float* part_o;          // [parts][unit_heads][d / 4][256][4]
  float* part_ml;         // [parts][unit_heads][256][2]
  unsigned int* tickets;  // [parts][unit_heads] finished ranges (0 between launches)
  void* out;
  float* lse;
  int n, most, kv_heads, group, width, pages, shift;
  int tg, tt, head_tiles, unit_heads;  // a query tile is tg heads of a group by tt tokens
  float scale_log2;
  unsigned int* err;
};

// Most requests of a handle: the planning blocks keep 24 bytes of each in shared memory.
constexpr int kPagedRequests = 8192;

// Most rows of one request.  A block of the prompt form that is not cut passes through one CTA, some 2 us at most for a tile
// of 128 keys, and a warp that has no rows in the units listed ahead waits for all four of them: 1 s here, 4 s with four times
// as many, which is where a wait gives up.  It adds up in fp32, 16 keys at a time, so that at 2^28 rows an accumulator no
// longer takes what a key adds.  The lists of work count with it, too: stages (16 rows) of the 304 requests whose ranges may
// be sought are 2^29 at most.
constexpr int kPagedCapacity = 1 << 24;

// Query rows of a kv head (new rows times heads of the group) up to which a call takes the token form, by the most
// rows that it may meet.  Token form and prompt form: four rows of 64 requests of up to 8190 keys and 8 kv heads 165 and
// 171 us, eight rows of 1000 keys 9.1 and 10.3; 15 rows of eight requests of up to 20011 keys 80 (with another tile of
// columns) and 64.  A call that may meet more takes the prompt form for all of them: two launches, one after the other,
// would each leave the GPU idle at its end, and an empty one costs 2 us and more.  The plan lists the work of both.
constexpr int kPagedTokenRows = 8;
// Keys that a warp of the token form takes at a time.
constexpr int kPagedStage = 16;

// The token form's pieces: as many key ranges as thread blocks run at once, or
// with more work up to kPagedWaves times as many, none shorter than kPagedRange
// stages.  A request has at least one.
constexpr int kPagedWaves = 4;
constexpr int kPagedRange = 128;
inline int paged_piece_cap(int token_blocks, int kv_heads, int requests) {
  return kPagedWaves * token_blocks / kv_heads + requests + 1;
}
// Ranges of requests that are cut (each has less than twice as many as its share).
inline int paged_part_cap(int token_blocks, int kv_heads) { return 2 * kPagedWaves * token_blocks / kv_heads + 2; }

// Query tiles of the prompt form.
constexpr int kPagedTile = 128;
// Blocks are cut into key ranges that fill the GPU at most kPagedRounds times, besides those that are not cut.
constexpr int kPagedRounds = 3;
inline int paged_unit_cap(int sms, int unit_heads, int block_tokens, int requests, int max_rows) {
  return max_rows / block_tokens + requests + kPagedRounds * sms / unit_heads + 1;
}
inline int paged_unit_parts(int sms, int unit_heads) { return kPagedRounds * sms / unit_heads + 1; }

cudaError_t paged_plan_configure();
cudaError_t launch_paged_plan(const PagedPlanParams& p, cudaStream_t s);
cudaError_t launch_paged_store(const PagedStoreParams& p, cudaStream_t s);
cudaError_t paged_token_configure(int head_dim);
int paged_token_blocks(int sms);
cudaError_t launch_paged_token(int head_dim, const CUtensorMap& k, const CUtensorMap& v, const PagedTokenParams& p,
                               int requests, int token_blocks, cudaStream_t s);
cudaError_t paged_prompt_configure(int head_dim);
// q: tensor map over the queries [n][heads][d], boxes of 64 features, tg heads and tt tokens; k, v: over the pools, boxes of
// a page's rows.
cudaError_t launch_paged_prompt(int head_dim, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                const PagedPromptParams& p, int sms, cudaStream_t s);

}  // namespace ff
