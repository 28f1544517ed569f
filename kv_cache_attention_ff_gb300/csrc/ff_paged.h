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

// A piece of the token form's work: a key range of one request.  Its kv heads are blocks of their own.
struct __align__(16) PagedPiece {
  int request, first, count, length;  // its packed rows, the rows that it holds
  int split, n_split;                 // key range `split` of n_split
  int part;                           // n_split > 1: place of the request's first range among the partial results
  int pad;
};

struct PagedState {
  int* tables;     // [requests][width] pages of each request, in order
  int* lengths;    // [requests] rows held
  int* news;       // [requests] rows of the latest step that have a place
  int* first;      // [requests + 1] where each request's rows begin in the packed buffers
  int* free;       // [pages] stack of the pages that no request has
  int* n_free;     // [1]
  int* slots;      // [max_rows] page * page_rows + row, or -1
  int* positions;  // [max_rows]
  PagedPiece* pieces;  // [piece_cap] the token form's work of the latest step
  int* n_pieces;   // [1]
  int requests, width, pages, capacity;
  int shift;       // page_rows = 1 << shift
};

struct PagedPlanParams {
  PagedState s;
  const int* start;   // [requests] or null: the rows held
  const int* counts;  // [requests]
  int n;              // rows of the packed buffers
  int kv_heads, group;
  int token_blocks;   // thread blocks of the token form that run at once
  unsigned int* err;
};

struct PagedStoreParams {
  const void* k;  // bf16 [n, kv_heads, d]
  const void* v;
  void* k_pool;
  void* v_pool;
  const int* slots;
  int n, kv_heads, head_dim, pages, shift;
};

struct PagedTokenParams {
  const PagedPiece* pieces;
  const int* n_pieces;
  const int* tables;
  float* part_o;          // [parts][kv_heads][rows][d]
  float* part_ml;         // [parts][kv_heads][rows][2] reference (log2 units) and sum
  unsigned int* tickets;  // [requests][kv_heads] finished ranges (0 between launches)
  const void* q;
  void* out;
  float* lse;
  int n, most, kv_heads, group, width, pages, shift;
  float scale_log2;
  unsigned int* err;
};

struct PagedAttnParams {
  PagedState s;
  const void* k_pool;
  const void* v_pool;
  const void* q;  // bf16 [n, heads, d]
  void* out;      // bf16 [n, heads, d]
  float* lse;     // [n, heads] or null
  int n, most, kv_heads, group;
  float scale_log2;  // log2(e) / sqrt(d)
  unsigned int* err;
};

// Most requests of a handle: the planning blocks keep 20 bytes of each in shared memory.
constexpr int kPagedRequests = 8192;

// Query rows of a kv head (new rows times heads of the group) up to which a request takes the token form.
constexpr int kPagedTokenRows = 32;
// Keys that a warp of the token form takes at a time.
constexpr int kPagedStage = 16;

// The token form's pieces: as many key ranges as thread blocks run at once, or
// with more work up to kPagedWaves times as many, none shorter than kPagedRange
// stages.  A request has at least one.
constexpr int kPagedWaves = 4;
constexpr int kPagedRange = 64;
inline int paged_piece_cap(int token_blocks, int kv_heads, int requests) {
  return kPagedWaves * token_blocks / kv_heads + requests + 1;
}
// Ranges of requests that are cut (each has less than twice as many as its share).
inline int paged_part_cap(int token_blocks, int kv_heads) { return 2 * kPagedWaves * token_blocks / kv_heads + 2; }

cudaError_t paged_plan_configure();
cudaError_t launch_paged_plan(const PagedPlanParams& p, cudaStream_t s);
cudaError_t launch_paged_store(const PagedStoreParams& p, cudaStream_t s);
cudaError_t paged_token_configure(int head_dim);
int paged_token_blocks(int sms);
cudaError_t launch_paged_token(int head_dim, const CUtensorMap& k, const CUtensorMap& v, const PagedTokenParams& p,
                               int requests, int token_blocks, cudaStream_t s);
cudaError_t launch_paged_attn(int head_dim, const PagedAttnParams& p, cudaStream_t s);

}  // namespace ff
