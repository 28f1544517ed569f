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

struct PagedState {
  int* tables;     // [requests][width] pages of each request, in order
  int* lengths;    // [requests] rows held
  int* news;       // [requests] rows of the latest step that have a place
  int* first;      // [requests + 1] where each request's rows begin in the packed buffers
  int* free;       // [pages] stack of the pages that no request has
  int* n_free;     // [1]
  int* slots;      // [max_rows] page * page_rows + row, or -1
  int* positions;  // [max_rows]
  int requests, width, pages, capacity;
  int shift;       // page_rows = 1 << shift
};

struct PagedPlanParams {
  PagedState s;
  const int* start;   // [requests] or null: the rows held
  const int* counts;  // [requests]
  int n;              // rows of the packed buffers
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

cudaError_t paged_plan_configure();
cudaError_t launch_paged_plan(const PagedPlanParams& p, cudaStream_t s);
cudaError_t launch_paged_store(const PagedStoreParams& p, cudaStream_t s);
cudaError_t launch_paged_attn(int head_dim, const PagedAttnParams& p, cudaStream_t s);

}  // namespace ff
