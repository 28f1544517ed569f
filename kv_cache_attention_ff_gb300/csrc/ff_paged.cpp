// Host side of the paged key/value cache behind the ff_paged_* entry points of ff.h:
// argument checks, the handle's memory and stream ordering.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <memory>
#include <vector>

#include "ff.h"
#include "ff_handle.h"
#include "ff_kv8.h"
#include "ff_paged.h"
#include "ff_ptx.cuh"

using namespace ff;

struct ff_paged {
  ff_paged_desc d{};
  PagedState state{};
  size_t total_bytes = 0;
  size_t pool_bytes = 0;  // of K or V of one layer
  void* memory = nullptr;
  uint8_t* pools = nullptr;  // [layers][K, V]
  int sm_count = 0;
  int token_blocks = 0;      // thread blocks of the token form that run at once
  int tg = 1, tt = 128, head_tiles = 1;  // query tiles of the prompt form: tg heads of a group by tt tokens
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  float* part_o = nullptr;
  float* part_ml = nullptr;
  unsigned int* tickets = nullptr;
  size_t ticket_bytes = 0;
  unsigned int* err = nullptr;
  std::vector<CUtensorMap> maps;  // [layers][boxes of 16 rows, boxes of a page][K, V], 64 features each
  CallOrder order;
};

namespace {

int validate(const ff_paged_desc* d) {
  if (!d) return FF_ERR_ARG;
  if (d->n_layers < 1 || d->pages < 1 || (d->page_rows != 16 && d->page_rows != 32 && d->page_rows != 64 && d->page_rows != 128) ||
      d->requests < 1 || d->requests > kPagedRequests || d->capacity < 1 || d->kv_heads < 1 ||
      d->kv_heads > 32767 || d->heads < 1 || d->heads % d->kv_heads != 0 || (d->head_dim != 64 && d->head_dim != 128) || d->max_rows < 1 ||
      d->device < 0)
    return FF_ERR_ARG;
  // 16-byte units of a call's rows are counted in 32 bits
  if (static_cast<double>(d->max_rows) * d->heads * (d->head_dim / 8) > 0x1p31) return FF_ERR_ARG;
  // No device holds this much: the sums below stay within 64 bits, slots and rows of a pool (of all kv heads) within 31.
  if (static_cast<double>(d->pages) * d->page_rows * d->kv_heads >= 0x1p31 ||
      static_cast<double>(d->n_layers) * d->pages * d->page_rows * d->kv_heads * d->head_dim > 0x1p46 ||
      static_cast<double>(d->requests) * d->capacity / d->page_rows > 0x1p38)
    return FF_ERR_OOM;
  if (d->capacity > kPagedCapacity) return FF_ERR_ARG;
  return FF_OK;
}

void free_all(ff_paged* h) {
  if (h->memory) cudaFree(h->memory);
  h->memory = nullptr;
  if (h->order.ev) cudaEventDestroy(h->order.ev);
  h->order.ev = nullptr;
}

// Tensor map over a pool as groups of eight rows of all pages and kv heads, [groups][d / 64][8][64]: a copy leaves `rows`
// of them in shared memory group by group, a group's 64-feature blocks one after the other (128-byte swizzled).
bool pool_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, void* pool, const ff_paged_desc& d, int rows) {
  const cuuint64_t row = static_cast<cuuint64_t>(d.head_dim) * 2;
  const cuuint64_t dims[4] = {64, 8, static_cast<cuuint64_t>(d.head_dim) / 64,
                              static_cast<cuuint64_t>(d.pages) * d.kv_heads * d.page_rows / 8};
  const cuuint64_t strides[3] = {row, 128, 8 * row};
  const cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(d.head_dim) / 64, static_cast<cuuint32_t>(rows) / 8};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pool, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over queries [n][heads][d]: boxes of tt tokens and tg heads.
bool query_map(const ff_paged* h, CUtensorMap* map, const void* q, int n) {
  const ff_paged_desc& d = h->d;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d.head_dim), static_cast<cuuint64_t>(d.heads), static_cast<cuuint64_t>(n)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d.head_dim) * 2, static_cast<cuuint64_t>(d.heads) * d.head_dim * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(h->tg), static_cast<cuuint32_t>(h->tt)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return h->encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int create(const ff_paged_desc& d, ff_paged_t** out) {
  int dev_count = 0;
  if (cudaGetDeviceCount(&dev_count) != cudaSuccess || d.device >= dev_count) {
    cudaGetLastError();
    return FF_ERR_CUDA;
  }
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d.device) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, d.device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d.device) != cudaSuccess)
    return FF_ERR_CUDA;
  if (major != 10 || minor != 3) return FF_ERR_UNSUPPORTED;
  DeviceScope scope(d.device);
  if (!scope.ok()) return FF_ERR_CUDA;

  std::unique_ptr<ff_paged, void (*)(ff_paged*)> owner(new ff_paged(), [](ff_paged* x) {
    free_all(x);
    delete x;
  });
  ff_paged* h = owner.get();
  h->d = d;
  h->pool_bytes = static_cast<size_t>(d.pages) * d.kv_heads * d.page_rows * d.head_dim * 2;
  PagedState& s = h->state;
  s.requests = d.requests;
  s.width = (d.capacity + d.page_rows - 1) / d.page_rows;
  s.pages = d.pages;
  s.capacity = d.capacity;
  s.shift = d.page_rows == 16 ? 4 : d.page_rows == 32 ? 5 : d.page_rows == 64 ? 6 : 7;
  h->sm_count = sms;
  h->token_blocks = paged_token_blocks(sms);
  const int group = d.heads / d.kv_heads;
  h->tg = std::min(group, kPagedTile);
  h->tt = kPagedTile / h->tg;
  h->head_tiles = (group + h->tg - 1) / h->tg;
  const int unit_heads = d.kv_heads * h->head_tiles;
  const size_t unit_cap = paged_unit_cap(sms, unit_heads, 2 * h->tt, d.requests, d.max_rows);
  // steps of so few rows never take the prompt form
  const bool tokens_only = static_cast<long long>(d.max_rows) * group <= kPagedTokenRows;
  const size_t unit_parts = tokens_only ? 0 : static_cast<size_t>(paged_unit_parts(sms, unit_heads)) * unit_heads;
  // one allocation: a part starts where the one before it ends, on the next 256 bytes
  size_t bytes = 0;
  auto part = [&](size_t n) {
    const size_t at = bytes;
    bytes += (n + 255) / 256 * 256;
    return at;
  };
  const size_t pools_at = part(2 * h->pool_bytes * d.n_layers);  // a pool is a multiple of 2048 bytes
  const size_t tables_at = part(static_cast<size_t>(d.requests) * s.width * sizeof(int));
  const size_t lengths_at = part(d.requests * sizeof(int));
  const size_t first_at = part((d.requests + 1) * sizeof(int));
  const size_t free_at = part(d.pages * sizeof(int)), n_free_at = part(sizeof(int));
  const size_t slots_at = part(d.max_rows * sizeof(int)), positions_at = part(d.max_rows * sizeof(int));
  const size_t pieces_at = part(paged_piece_cap(h->token_blocks, d.kv_heads, d.requests) * sizeof(PagedPiece));
  const size_t n_pieces_at = part(sizeof(int));
  const size_t units_at = part(unit_cap * sizeof(PagedPiece)), n_units_at = part(sizeof(int));
  const size_t tiles_at = part(unit_cap * sizeof(int));
  // the forms' launches follow each other: they share the room for partial results
  const size_t part_rows = std::max(static_cast<size_t>(paged_part_cap(h->token_blocks, d.kv_heads)) * d.kv_heads * kPagedTokenRows,
                                    unit_parts * 2 * kPagedTile);
  const size_t part_o_at = part(part_rows * d.head_dim * sizeof(float)), part_ml_at = part(part_rows * 2 * sizeof(float));
  h->ticket_bytes = std::max(static_cast<size_t>(d.requests) * d.kv_heads, unit_parts) * sizeof(unsigned);
  const size_t tickets_at = part(h->ticket_bytes);
  const size_t err_at = part(sizeof(unsigned));
  h->total_bytes = bytes;
  if (d.max_bytes && bytes > d.max_bytes) return FF_ERR_OOM;
  if (cudaMalloc(&h->memory, bytes) != cudaSuccess) {
    cudaGetLastError();
    h->memory = nullptr;
    return FF_ERR_OOM;
  }
  uint8_t* base = static_cast<uint8_t*>(h->memory);
  h->pools = base + pools_at;
  s.tables = reinterpret_cast<int*>(base + tables_at);
  s.lengths = reinterpret_cast<int*>(base + lengths_at);
  s.first = reinterpret_cast<int*>(base + first_at);
  s.free = reinterpret_cast<int*>(base + free_at);
  s.n_free = reinterpret_cast<int*>(base + n_free_at);
  s.slots = reinterpret_cast<int*>(base + slots_at);
  s.positions = reinterpret_cast<int*>(base + positions_at);
  s.pieces = reinterpret_cast<PagedPiece*>(base + pieces_at);
  s.n_pieces = reinterpret_cast<int*>(base + n_pieces_at);
  s.units = reinterpret_cast<PagedPiece*>(base + units_at);
  s.n_units = reinterpret_cast<int*>(base + n_units_at);
  s.tiles = reinterpret_cast<int*>(base + tiles_at);
  h->part_o = reinterpret_cast<float*>(base + part_o_at);
  h->part_ml = reinterpret_cast<float*>(base + part_ml_at);
  h->tickets = reinterpret_cast<unsigned*>(base + tickets_at);
  h->err = reinterpret_cast<unsigned*>(base + err_at);
  cudaDriverEntryPointQueryResult found{};
  void* fn = nullptr;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess || !fn)
    return FF_ERR_CUDA;
  h->encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  h->maps.resize(4 * static_cast<size_t>(d.n_layers));
  for (size_t i = 0; i < h->maps.size(); ++i)
    if (!pool_map(h->encode, &h->maps[i], h->pools + (i / 4 * 2 + i % 2) * h->pool_bytes, d, i % 4 < 2 ? kPagedStage : d.page_rows))
      return FF_ERR_CUDA;
  // all pages are free, the lowest on top; no row has a place
  std::vector<int> pages(d.pages);
  for (int i = 0; i < d.pages; ++i) pages[i] = d.pages - 1 - i;
  if (cudaMemset(h->memory, 0, bytes) != cudaSuccess ||
      cudaMemset(s.slots, 0xff, d.max_rows * sizeof(int)) != cudaSuccess ||
      cudaMemcpy(s.free, pages.data(), pages.size() * sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess ||
      cudaMemcpy(s.n_free, &d.pages, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess ||
      paged_plan_configure() != cudaSuccess || paged_token_configure(d.head_dim) != cudaSuccess ||
      paged_prompt_configure(d.head_dim) != cudaSuccess ||
      cudaEventCreateWithFlags(&h->order.ev, cudaEventDisableTiming) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)
    return FF_ERR_CUDA;
  *out = owner.release();
  return FF_OK;
}

bool layer_ok(const ff_paged* h, int layer) { return h && layer >= 0 && layer < h->d.n_layers; }

void* k_pool(const ff_paged* h, int layer) { return h->pools + 2 * h->pool_bytes * layer; }
void* v_pool(const ff_paged* h, int layer) { return h->pools + 2 * h->pool_bytes * layer + h->pool_bytes; }

}  // namespace

extern "C" {

int ff_paged_desc_default(ff_paged_desc* d) {
  if (!d) return FF_ERR_ARG;
  std::memset(d, 0, sizeof(*d));
  d->n_layers = 1;
  d->pages = 1950;
  d->page_rows = 16;
  d->requests = 1;
  d->capacity = 31200;
  d->heads = 12;
  d->kv_heads = 12;
  d->head_dim = 128;
  d->max_rows = 4680;
  return FF_OK;
}

int ff_paged_create(const ff_paged_desc* desc, ff_paged_t** out) {
  if (!out) return FF_ERR_ARG;
  const int v = validate(desc);
  if (v != FF_OK) return v;
  try {
    return create(*desc, out);
  } catch (...) {  // nothing but memory can fail there
    return FF_ERR_OOM;
  }
}

int ff_paged_destroy(ff_paged_t* h) {
  if (!h) return FF_OK;
  DeviceScope scope(h->d.device);
  cudaDeviceSynchronize();
  free_all(h);
  delete h;
  return FF_OK;
}

int ff_paged_bytes(const ff_paged_t* h, size_t* bytes) {
  if (!h || !bytes) return FF_ERR_ARG;
  *bytes = h->total_bytes;
  return FF_OK;
}

int ff_paged_info(const ff_paged_t* h, int** tables, int** lengths, int** first, int** slots, int** positions, int** free,
                  int** n_free) {
  if (!h) return FF_ERR_ARG;
  const PagedState& s = h->state;
  if (tables) *tables = s.tables;
  if (lengths) *lengths = s.lengths;
  if (first) *first = s.first;
  if (slots) *slots = s.slots;
  if (positions) *positions = s.positions;
  if (free) *free = s.free;
  if (n_free) *n_free = s.n_free;
  return FF_OK;
}

int ff_paged_layer_info(const ff_paged_t* h, int layer, void** k, void** v) {
  if (!layer_ok(h, layer)) return FF_ERR_ARG;
  if (k) *k = k_pool(h, layer);
  if (v) *v = v_pool(h, layer);
  return FF_OK;
}

int ff_paged_plan(ff_paged_t* h, int n, const int* start, const int* counts, void* stream) {
  if (!h || n < 1 || n > h->d.max_rows || !counts || !aligned(counts, 4) || !aligned(start, 4)) return FF_ERR_ARG;
  DeviceScope scope(h->d.device);
  if (!scope.ok()) return FF_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CallEntry at;
  const int rc = h->order.enter(h->d.device, s, &at);
  if (rc != FF_OK) return rc;
  PagedPlanParams p{};
  p.s = h->state;
  p.start = start;
  p.counts = counts;
  p.n = n;
  p.kv_heads = h->d.kv_heads;
  p.group = h->d.heads / h->d.kv_heads;
  p.head_dim = h->d.head_dim;
  p.token_blocks = h->token_blocks;
  p.sms = h->sm_count;
  p.block_tokens = 2 * h->tt;
  p.unit_heads = h->d.kv_heads * h->head_tiles;
  p.err = h->err;
  return h->order.leave(s, at, launch_paged_plan(p, s));
}

int ff_paged_store(ff_paged_t* h, int layer, int n, const void* k, const void* v, void* stream) {
  if (!layer_ok(h, layer) || n < 1 || n > h->d.max_rows || !k || !v || !aligned(k, 16) || !aligned(v, 16)) return FF_ERR_ARG;
  DeviceScope scope(h->d.device);
  if (!scope.ok()) return FF_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CallEntry at;
  const int rc = h->order.enter(h->d.device, s, &at);
  if (rc != FF_OK) return rc;
  PagedStoreParams p{};
  p.k = k;
  p.v = v;
  p.k_pool = k_pool(h, layer);
  p.v_pool = v_pool(h, layer);
  p.slots = h->state.slots;
  p.total = h->state.first + h->d.requests;
  p.n = n;
  p.kv_heads = h->d.kv_heads;
  p.head_dim = h->d.head_dim;
  p.pages = h->d.pages;
  p.shift = h->state.shift;
  return h->order.leave(s, at, launch_paged_store(p, s));
}

int ff_paged_attn(ff_paged_t* h, int layer, int n, int most, const void* q, void* out, float* lse, void* stream) {
  if (!layer_ok(h, layer) || n < 1 || n > h->d.max_rows || most < 1 || !q || !out || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(lse, 4))
    return FF_ERR_ARG;
  const ff_paged_desc& d = h->d;
  const size_t q_bytes = static_cast<size_t>(n) * d.heads * d.head_dim * 2, lse_bytes = static_cast<size_t>(n) * d.heads * 4;
  if (overlap(q, q_bytes, out, q_bytes) ||
      (lse && (overlap(lse, lse_bytes, q, q_bytes) || overlap(lse, lse_bytes, out, q_bytes))))
    return FF_ERR_ARG;
  DeviceScope scope(d.device);
  if (!scope.ok()) return FF_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CallEntry at;
  const int rc = h->order.enter(d.device, s, &at);
  if (rc != FF_OK) return rc;
  const int group = d.heads / d.kv_heads;
  const float scale_log2 = static_cast<float>(1.4426950408889634 / __builtin_sqrt(static_cast<double>(d.head_dim)));
  most = std::min(most, d.max_rows);  // no request has more
  cudaError_t e;
  if (most <= kPagedTokenRows / group) {
    PagedTokenParams p{};
    p.pieces = h->state.pieces;
    p.n_pieces = h->state.n_pieces;
    p.tables = h->state.tables;
    p.part_o = h->part_o;
    p.part_ml = h->part_ml;
    p.tickets = h->tickets;
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.n = n;
    p.most = most;
    p.kv_heads = d.kv_heads;
    p.group = group;
    p.width = h->state.width;
    p.pages = d.pages;
    p.shift = h->state.shift;
    p.scale_log2 = scale_log2;
    p.err = h->err;
    e = launch_paged_token(d.head_dim, h->maps[4 * layer], h->maps[4 * layer + 1], p, d.requests, h->token_blocks, s);
  } else {
    CUtensorMap tq;
    if (!query_map(h, &tq, q, n)) return FF_ERR_CUDA;
    PagedPromptParams p{};
    p.units = h->state.units;
    p.n_units = h->state.n_units;
    p.tables = h->state.tables;
    p.part_o = h->part_o;
    p.part_ml = h->part_ml;
    p.tickets = h->tickets;
    p.out = out;
    p.lse = lse;
    p.n = n;
    p.most = most;
    p.kv_heads = d.kv_heads;
    p.group = group;
    p.width = h->state.width;
    p.pages = d.pages;
    p.shift = h->state.shift;
    p.tg = h->tg;
    p.tt = h->tt;
    p.head_tiles = h->head_tiles;
    p.unit_heads = d.kv_heads * h->head_tiles;
    p.scale_log2 = scale_log2;
    p.err = h->err;
    e = launch_paged_prompt(d.head_dim, tq, h->maps[4 * layer + 2], h->maps[4 * layer + 3], p, h->sm_count, s);
  }
  return h->order.leave(s, at, e);
}

int ff_paged_error_poll(ff_paged_t* h) {
  if (!h) return FF_ERR_ARG;
  DeviceScope scope(h->d.device);
  if (!scope.ok()) return FF_ERR_CUDA;
  unsigned int word = 0;
  // a kernel that gave up may have left ranges of a piece unfinished
  const int rc = take_error(h->err, &word, kErrTimeout, h->tickets, h->ticket_bytes);
  if (rc != FF_OK || !word) return rc;
  return (word & kErrTimeout) ? FF_ERR_DEVICE_TIMEOUT : FF_ERR_CAPACITY;
}

}  // extern "C"
