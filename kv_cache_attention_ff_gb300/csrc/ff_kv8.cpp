// Host side of the 8-bit key/value cache behind the ff_kv8_* entry points of ff.h:
// argument checks, the handle's memory, work plans and stream ordering.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <memory>
#include <vector>

#include "ff.h"
#include "ff_handle.h"
#include "ff_internal.h"
#include "ff_kv8.h"
#include "ff_ptx.cuh"

using namespace ff;

// Work plan of an attention call.
struct Kv8Plan {
  bool chunk = false;   // the tensor-core form (many query rows) or the token form
  int row_tiles = 0;    // query tiles per (sequence, kv head)
  int splits = 1;       // key ranges of a split tile, at most
  int n_whole = 0;      // chunk form: units that are not split
  long long items = 0;  // query tiles in all
  size_t part_rows = 0;
  int weigh_splits = 1; // chunk form, weights: ranges of query rows per 256 keys, at most
  size_t weigh_floats = 0;
};

struct ff_kv8 {
  ff_kv8_desc d{};
  int sm_count = 0;
  int blocks = 0;
  size_t total_bytes = 0;
  void* memory = nullptr;
  std::vector<Kv8Layer> layers;
  float* part_o = nullptr;
  float* part_ml = nullptr;
  unsigned int* tickets = nullptr;
  float* lse2 = nullptr;
  int2* pieces = nullptr;
  unsigned int* err = nullptr;
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  CallOrder order;
};

namespace {

constexpr int kMaxSplits = 64;

int validate(const ff_kv8_desc* d) {
  if (!d) return FF_ERR_ARG;
  if (d->n_layers < 1 || d->batch < 1 || d->batch > 65535 || d->capacity < 1 || d->capacity > (1 << 30) ||
      d->kv_heads < 1 || d->kv_heads > 32767 || d->heads < 1 || d->heads % d->kv_heads != 0 ||
      (d->head_dim != 64 && d->head_dim != 128) || d->max_tokens < 1 || d->device < 0)
    return FF_ERR_ARG;
  // query rows of a kv head, and pieces of a launch, are ints
  if (static_cast<long long>(d->max_tokens) * d->heads * d->batch > (1ll << 30)) return FF_ERR_ARG;
  // no device holds this much, and the sums below stay within 64 bits
  if (static_cast<double>(d->n_layers) * d->batch * d->capacity * d->kv_heads * d->head_dim > 0x1p46) return FF_ERR_OOM;
  return FF_OK;
}

// Chunk form: whole waves of unsplit units, then the rest in key ranges, by the
// time in key tiles (a piece costs 3 more for its prologue and epilogue, the
// merge 2 and its traffic).  Up to 128 rows go through two tiles at a time.
void plan_chunk_rows(const ff_kv8_desc& d, int sms, int n, Kv8Plan* pl) {
  const long long rows = static_cast<long long>(n) * (d.heads / d.kv_heads);
  pl->chunk = true;
  pl->row_tiles = static_cast<int>((rows + 255) / 256);
  pl->items = static_cast<long long>(d.batch) * d.kv_heads * pl->row_tiles;
  const double tiles = (d.capacity + 127) / 128 * (rows <= kKv8OneTile ? 0.5 : 1.0);
  const long long waves = (pl->items + sms - 1) / sms;
  double best = static_cast<double>(waves) * (tiles + 3.0);
  pl->n_whole = static_cast<int>(pl->items);
  for (long long m = std::max<long long>(0, waves - 2); m < waves; ++m) {
    const long long rest = pl->items - m * sms;
    if (rest <= 0) continue;
    for (int s = 2; s <= kMaxSplits && rest * s <= 4ll * sms; ++s) {
      const double cost = static_cast<double>(m) * (tiles + 3.0) +
                          static_cast<double>((rest * s + sms - 1) / sms) * (tiles / s + 3.0) + 2.0 + 0.02 * rest * s;
      if (cost < best * 0.999) {
        best = cost;
        pl->n_whole = static_cast<int>(m * sms);
        pl->splits = s;
        pl->part_rows = static_cast<size_t>(rest) * s * 256;
      }
    }
  }
}

// Weights of the chunk form: items of 256 keys, shared by one CTA per SM; few items
// are cut into ranges of query tiles where that evens them out.  An item costs
// about 2 tiles more for its start.
void plan_chunk_weigh(const ff_kv8_desc& d, int sms, int n, Kv8Plan* pl) {
  const long long items = static_cast<long long>(d.batch) * d.kv_heads * ((d.capacity + 255) / 256);
  const int group = d.heads / d.kv_heads, tg = std::min(group, 128), tt = 128 / tg;
  const long long tiles = (n + tt - 1ll) / tt * ((group + tg - 1) / tg);
  const long long most = std::max(1ll, std::min<long long>({tiles, kMaxSplits, 8ll * sms / items}));
  double best = 0.0;
  for (long long s = 1; s <= most; ++s) {
    const double cost = static_cast<double>((items * s + sms - 1) / sms) * ((tiles + s - 1) / s + 2.0);
    if (s == 1 || cost < best * 0.98) {
      best = cost;
      pl->weigh_splits = static_cast<int>(s);
    }
  }
  // room for the most ranges that any smaller n may be cut into
  pl->weigh_floats = most > 1 ? static_cast<size_t>(items) * most * 256 : 0;
}

Kv8Plan plan_attention(const ff_kv8_desc& d, int sms, int n) {
  Kv8Plan pl;
  if (static_cast<long long>(n) * (d.heads / d.kv_heads) <= kKv8TokenRows) {
    // room for whichever number of rows is planned the most thread blocks
    const int few = kv8_token_plan(d.batch, d.kv_heads, 1, sms).part_blocks;
    const int many = kv8_token_plan(d.batch, d.kv_heads, kKv8TokenRows, sms).part_blocks;
    pl.part_rows = static_cast<size_t>(std::max(few, many)) * kKv8TokenRows;
  } else {
    plan_chunk_rows(d, sms, n, &pl);
    plan_chunk_weigh(d, sms, n, &pl);
  }
  return pl;
}

void free_all(ff_kv8* h) {
  if (h->memory) cudaFree(h->memory);
  h->memory = nullptr;
  if (h->order.ev) cudaEventDestroy(h->order.ev);
  h->order.ev = nullptr;
}

int create(const ff_kv8_desc& d, ff_kv8_t** out) {
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

  std::unique_ptr<ff_kv8, void (*)(ff_kv8*)> owner(new ff_kv8(), [](ff_kv8* x) {
    free_all(x);
    delete x;
  });
  ff_kv8* h = owner.get();
  h->layers.reserve(d.n_layers);
  h->d = d;
  h->sm_count = sms;
  h->blocks = (d.capacity + kKv8Block - 1) / kKv8Block;
  const size_t tiles = static_cast<size_t>(d.batch) * h->blocks * d.kv_heads;
  const size_t code_bytes = tiles * kKv8Block * d.head_dim;
  const size_t scale_bytes = tiles * sizeof(float);
  // the most partial rows of any call; plans change only with the number of query tiles
  size_t part_rows = 0;
  const int group = d.heads / d.kv_heads;
  for (long long n = 1; n <= d.max_tokens;) {
    const Kv8Plan pl = plan_attention(d, sms, static_cast<int>(n));
    part_rows = std::max(part_rows, pl.part_rows);
    // the next n of another plan: the first of the chunk form, the first of more than 128 rows, then one
    // more tile of 256 rows at a time
    n = (!pl.chunk ? kKv8TokenRows : n * group <= kKv8OneTile ? kKv8OneTile : pl.row_tiles * 256ll) / group + 1;
  }
  // the weights pass may cut query rows into more ranges the more of them there are
  Kv8Plan most;
  plan_chunk_weigh(d, sms, d.max_tokens, &most);
  part_rows = std::max(part_rows, (most.weigh_floats + d.head_dim - 1) / d.head_dim);
  // one per item of the token form, one per 32 keys of the weights pass
  const size_t n_tickets = static_cast<size_t>(d.batch) * d.kv_heads * ((d.capacity + 255) / 256) * 8;
  // one allocation: a part starts where the one before it ends, on the next 256 bytes
  size_t bytes = 0;
  auto part = [&](size_t n) {
    const size_t at = bytes;
    bytes += (n + 255) / 256 * 256;
    return at;
  };
  const size_t layers = d.n_layers;
  const size_t k8_at = part(layers * code_bytes), v8_at = part(layers * code_bytes);
  const size_t scales_at = part(layers * scale_bytes * 2);
  const size_t seqs_at = part(layers * d.batch * 2 * sizeof(int));
  const size_t part_o_at = part(part_rows * d.head_dim * sizeof(float)), part_ml_at = part(part_rows * 2 * sizeof(float));
  const size_t tickets_at = part(n_tickets * sizeof(unsigned));
  const size_t lse_at = part(static_cast<size_t>(d.batch) * d.max_tokens * d.heads * sizeof(float));
  const size_t pieces_at = part(static_cast<size_t>(d.batch) * d.kv_heads * sizeof(int2));
  const size_t err_at = part(sizeof(unsigned));
  h->total_bytes = bytes;
  int rc = FF_OK;
  if (d.max_bytes && bytes > d.max_bytes) rc = FF_ERR_OOM;
  if (rc == FF_OK && cudaMalloc(&h->memory, bytes) != cudaSuccess) {
    cudaGetLastError();
    h->memory = nullptr;
    rc = FF_ERR_OOM;
  }
  if (rc == FF_OK && cudaMemset(h->memory, 0, bytes) != cudaSuccess) rc = FF_ERR_CUDA;
  uint8_t* base = static_cast<uint8_t*>(h->memory);
  if (rc == FF_OK && (kv8_configure(d.head_dim) != cudaSuccess || kv8_chunk_configure(d.head_dim) != cudaSuccess ||
                      kv8_chunk_weigh_configure(d.head_dim) != cudaSuccess || kv8_store_configure() != cudaSuccess))
    rc = FF_ERR_CUDA;
  if (rc == FF_OK) {
    cudaDriverEntryPointQueryResult found{};
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess || !fn)
      rc = FF_ERR_CUDA;
    h->encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  if (rc == FF_OK && cudaEventCreateWithFlags(&h->order.ev, cudaEventDisableTiming) != cudaSuccess) rc = FF_ERR_CUDA;
  if (rc == FF_OK && cudaDeviceSynchronize() != cudaSuccess) rc = FF_ERR_CUDA;
  if (rc != FF_OK) return rc;
  for (int l = 0; l < d.n_layers; ++l) {
    Kv8Layer c{};
    c.k8 = base + k8_at + l * code_bytes;
    c.v8 = base + v8_at + l * code_bytes;
    c.ks = reinterpret_cast<float*>(base + scales_at + 2 * l * scale_bytes);
    c.vs = c.ks + tiles;
    c.lengths = reinterpret_cast<int*>(base + seqs_at) + 2 * l * static_cast<size_t>(d.batch);
    c.done = reinterpret_cast<unsigned*>(c.lengths + d.batch);
    c.batch = d.batch;
    c.blocks = h->blocks;
    c.capacity = d.capacity;
    c.kv_heads = d.kv_heads;
    h->layers.push_back(c);
  }
  h->part_o = reinterpret_cast<float*>(base + part_o_at);
  h->part_ml = reinterpret_cast<float*>(base + part_ml_at);
  h->tickets = reinterpret_cast<unsigned*>(base + tickets_at);
  h->lse2 = reinterpret_cast<float*>(base + lse_at);
  h->pieces = reinterpret_cast<int2*>(base + pieces_at);
  h->err = reinterpret_cast<unsigned*>(base + err_at);
  *out = owner.release();
  return FF_OK;
}

// Tensor map over queries [batch * n][heads][d] for the weights pass: boxes of 64 features,
// up to 128 heads of a group and as many tokens as make up 128 rows.
int query_map(const ff_kv8* h, CUtensorMap* map, const void* q, int n) {
  const ff_kv8_desc& d = h->d;
  const int tg = std::min(d.heads / d.kv_heads, 128);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d.head_dim), static_cast<cuuint64_t>(d.heads),
                              static_cast<cuuint64_t>(d.batch) * n};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d.head_dim) * 2, static_cast<cuuint64_t>(d.heads) * d.head_dim * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(tg), static_cast<cuuint32_t>(128 / tg)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return h->encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? FF_OK
             : FF_ERR_CUDA;
}

bool layer_ok(const ff_kv8* h, int layer) { return h && layer >= 0 && layer < h->d.n_layers; }

// n rows of every kv head are indexed with 32-bit ints
bool rows_ok(const ff_kv8* h, int n) {
  return n >= 1 && static_cast<long long>(n) * h->d.kv_heads * (h->d.head_dim / 8) < (1ll << 30);
}

}  // namespace

extern "C" {

int ff_kv8_desc_default(ff_kv8_desc* d) {
  if (!d) return FF_ERR_ARG;
  std::memset(d, 0, sizeof(*d));
  d->n_layers = 1;
  d->batch = 1;
  d->capacity = 31200;
  d->heads = 12;
  d->kv_heads = 12;
  d->head_dim = 128;
  d->max_tokens = 4680;
  return FF_OK;
}

int ff_kv8_create(const ff_kv8_desc* desc, ff_kv8_t** out) {
  if (!out) return FF_ERR_ARG;
  const int v = validate(desc);
  if (v != FF_OK) return v;
  try {
    return create(*desc, out);
  } catch (...) {  // nothing but memory can fail there
    return FF_ERR_OOM;
  }
}

int ff_kv8_destroy(ff_kv8_t* h) {
  if (!h) return FF_OK;
  DeviceScope scope(h->d.device);
  cudaDeviceSynchronize();
  free_all(h);
  delete h;
  return FF_OK;
}

int ff_kv8_bytes(const ff_kv8_t* h, size_t* bytes) {
  if (!h || !bytes) return FF_ERR_ARG;
  *bytes = h->total_bytes;
  return FF_OK;
}

int ff_kv8_layer_info(const ff_kv8_t* h, int layer, void** k8, void** v8, float** k_scale, float** v_scale,
                      int** lengths) {
  if (!layer_ok(h, layer)) return FF_ERR_ARG;
  const Kv8Layer& c = h->layers[layer];
  if (k8) *k8 = c.k8;
  if (v8) *v8 = c.v8;
  if (k_scale) *k_scale = c.ks;
  if (v_scale) *v_scale = c.vs;
  if (lengths) *lengths = c.lengths;
  return FF_OK;
}

int ff_kv8_append(ff_kv8_t* h, int layer, int n, const void* k, const void* v, const int* start, const int* counts,
                  void* stream) {
  if (!layer_ok(h, layer) || !rows_ok(h, n) || n > h->d.capacity || !k || !v || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(start, 4) || !aligned(counts, 4))
    return FF_ERR_ARG;
  DeviceScope scope(h->d.device);
  if (!scope.ok()) return FF_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CallEntry at;
  const int rc = h->order.enter(h->d.device, s, &at);
  if (rc != FF_OK) return rc;
  Kv8AppendParams p{};
  p.c = h->layers[layer];
  p.k = k;
  p.v = v;
  p.start = start;
  p.counts = counts;
  p.n = n;
  p.err = h->err;
  return h->order.leave(s, at, launch_kv8_append(h->d.head_dim, p, s));
}

int ff_kv8_load(ff_kv8_t* h, int layer, int n, const int* start, void* k, void* v, void* stream) {
  if (!layer_ok(h, layer) || !rows_ok(h, n) || !k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4))
    return FF_ERR_ARG;
  const size_t bytes = static_cast<size_t>(h->d.batch) * n * h->d.kv_heads * h->d.head_dim * 2;
  if (overlap(k, bytes, v, bytes)) return FF_ERR_ARG;
  DeviceScope scope(h->d.device);
  if (!scope.ok()) return FF_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CallEntry at;
  const int rc = h->order.enter(h->d.device, s, &at);
  if (rc != FF_OK) return rc;
  Kv8LoadParams p{};
  p.c = h->layers[layer];
  p.k = k;
  p.v = v;
  p.start = start;
  p.n = n;
  return h->order.leave(s, at, launch_kv8_load(h->d.head_dim, p, s));
}

int ff_kv8_attn(ff_kv8_t* h, int layer, int n, const void* q, const int* counts, int causal, void* out, float* lse,
                const float* weights_in, float* weights, void* stream) {
  if (!layer_ok(h, layer) || n < 1 || n > h->d.max_tokens || !q || !out || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(counts, 4) || !aligned(lse, 4) || !aligned(weights_in, 4) || !aligned(weights, 4) ||
      (causal != 0 && causal != 1) || (weights_in && !weights))
    return FF_ERR_ARG;
  const ff_kv8_desc& d = h->d;
  const size_t q_bytes = static_cast<size_t>(d.batch) * n * d.heads * d.head_dim * 2;
  const size_t lse_bytes = static_cast<size_t>(d.batch) * n * d.heads * 4;
  const size_t w_bytes = static_cast<size_t>(d.batch) * d.kv_heads * d.capacity * 4;
  if (overlap(q, q_bytes, out, q_bytes) ||
      (lse && (overlap(lse, lse_bytes, q, q_bytes) || overlap(lse, lse_bytes, out, q_bytes))) ||
      (weights && (overlap(weights, w_bytes, q, q_bytes) || overlap(weights, w_bytes, out, q_bytes) ||
                   (lse && overlap(weights, w_bytes, lse, lse_bytes)))) ||
      (weights_in && weights_in != weights &&
       (overlap(weights_in, w_bytes, weights, w_bytes) || overlap(weights_in, w_bytes, out, q_bytes) ||
        (lse && overlap(weights_in, w_bytes, lse, lse_bytes)))))
    return FF_ERR_ARG;
  DeviceScope scope(d.device);
  if (!scope.ok()) return FF_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CallEntry at;
  const int rc = h->order.enter(h->d.device, s, &at);
  if (rc != FF_OK) return rc;
  const Kv8Plan pl = plan_attention(d, h->sm_count, n);
  const int group = d.heads / d.kv_heads;
  const float scale_log2 = static_cast<float>(1.4426950408889634 / __builtin_sqrt(static_cast<double>(d.head_dim)));
  CUtensorMap tq;
  if (pl.chunk && weights && query_map(h, &tq, q, n) != FF_OK) return FF_ERR_CUDA;
  cudaError_t e;
  if (pl.chunk) {
    Kv8ChunkParams p{};
    p.c = h->layers[layer];
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.counts = counts;
    p.n = n;
    p.group = group;
    p.causal = causal;
    p.scale_log2 = scale_log2;
    p.row_blocks = pl.row_tiles;
    p.units = static_cast<int>(pl.items);
    p.n_whole = pl.n_whole;
    p.splits = pl.splits;
    p.part_o = h->part_o;
    p.part_ml = h->part_ml;
    p.lse2 = weights ? h->lse2 : nullptr;
    p.err = h->err;
    e = launch_kv8_chunk_attn(d.head_dim, p, s);
  } else {
    Kv8AttnParams p{};
    p.c = h->layers[layer];
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.counts = counts;
    p.n = n;
    p.group = group;
    p.causal = causal;
    p.scale_log2 = scale_log2;
    const Kv8TokenPlan tp = kv8_token_plan(d.batch, d.kv_heads, n * group, h->sm_count);
    p.per_head = tp.per_head;
    p.part_o = h->part_o;
    p.part_ml = h->part_ml;
    p.tickets = h->tickets;
    p.pieces = h->pieces;
    p.lse2 = weights ? h->lse2 : nullptr;
    e = launch_kv8_token_attn(d.head_dim, p, tp.grid, s);
  }
  if (e == cudaSuccess && weights && pl.chunk) {
    Kv8ChunkWeighParams w{};
    w.c = h->layers[layer];
    w.lse2 = h->lse2;
    w.counts = counts;
    w.weights_in = weights_in ? weights_in : weights;
    w.weights = weights;
    w.n = n;
    w.group = group;
    w.causal = causal;
    w.scale_log2 = scale_log2;
    w.tg = std::min(group, 128);
    w.tt = 128 / w.tg;
    w.head_tiles = (group + w.tg - 1) / w.tg;
    w.key_tiles = (d.capacity + 255) / 256;
    w.splits = pl.weigh_splits;
    w.items = d.batch * d.kv_heads * w.key_tiles * w.splits;
    w.part = h->part_o;  // the merge of the attention's partials comes first on the stream
    w.tickets = h->tickets;
    w.err = h->err;
    e = launch_kv8_chunk_weigh(d.head_dim, tq, w, h->sm_count, s);
  } else if (e == cudaSuccess && weights) {
    Kv8WeighParams w{};
    w.c = h->layers[layer];
    w.q = q;
    w.lse2 = h->lse2;
    w.counts = counts;
    w.weights_in = weights_in ? weights_in : weights;
    w.weights = weights;
    w.n = n;
    w.group = group;
    w.causal = causal;
    w.scale_log2 = scale_log2;
    const Kv8TokenPlan wp = kv8_weigh_plan(d.batch, d.kv_heads, h->sm_count);
    w.per_head = wp.per_head;
    e = launch_kv8_weigh(d.head_dim, w, wp.grid, s);
  }
  return h->order.leave(s, at, e);
}

int ff_kv8_evict(ff_kv8_t* src, int src_layer, ff_kv8_t* dst, int dst_layer, int n_keep, int n_recent,
                 const float* weights, float* weights_out, int* kept, void* stream) {
  if (!layer_ok(src, src_layer) || !layer_ok(dst, dst_layer) || (src == dst && src_layer == dst_layer) ||
      src->d.batch != dst->d.batch || src->d.kv_heads != dst->d.kv_heads || src->d.head_dim != dst->d.head_dim ||
      src->d.device != dst->d.device || n_keep < 1 || n_keep > dst->d.capacity || n_recent < 0 || n_recent > n_keep ||
      !weights || !weights_out || !kept || !aligned(weights, 4) || !aligned(weights_out, 4) || !aligned(kept, 4))
    return FF_ERR_ARG;
  const size_t lists = static_cast<size_t>(src->d.batch) * src->d.kv_heads;
  const size_t in_bytes = lists * src->d.capacity * 4, out_bytes = lists * dst->d.capacity * 4;
  if (overlap(weights, in_bytes, weights_out, out_bytes) || overlap(weights, in_bytes, kept, lists * n_keep * 4) ||
      overlap(weights_out, out_bytes, kept, lists * n_keep * 4))
    return FF_ERR_ARG;
  DeviceScope scope(src->d.device);
  if (!scope.ok()) return FF_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CallEntry at;
  int rc = src->order.enter(src->d.device, s, &at);
  if (rc == FF_OK && dst != src) rc = dst->order.enter(dst->d.device, s, &at);
  if (rc != FF_OK) return rc;
  Kv8EvictParams p{};
  p.src = src->layers[src_layer];
  p.dst = dst->layers[dst_layer];
  p.weights = weights;
  p.weights_out = weights_out;
  p.kept = kept;
  p.n_keep = n_keep;
  p.n_recent = n_recent;
  const cudaError_t e = launch_kv8_evict(src->d.head_dim, p, src->sm_count, s);
  rc = src->order.leave(s, at, e);
  if (dst != src) {
    const int rc2 = dst->order.leave(s, at, e);
    if (rc == FF_OK) rc = rc2;
  }
  return rc;
}

int ff_kv8_error_poll(ff_kv8_t* h) {
  if (!h) return FF_ERR_ARG;
  DeviceScope scope(h->d.device);
  if (!scope.ok()) return FF_ERR_CUDA;
  unsigned int word = 0;
  const int rc = take_error(h->err, &word);
  if (rc != FF_OK || !word) return rc;
  return (word & kErrTimeout) ? FF_ERR_DEVICE_TIMEOUT : FF_ERR_CAPACITY;
}

}  // extern "C"
