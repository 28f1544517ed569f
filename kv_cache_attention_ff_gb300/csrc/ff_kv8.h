// Structures shared by the host side of the 8-bit cache (ff_kv8.cpp) and its kernels.
//
// Storage of one layer: for sequence b, token block t (kKv8Block rows) and kv
// head h one tile of K and one of V, kKv8Block x head_dim e4m3 codes each,
// tile index (b * blocks + t) * kv_heads + h, and one fp32 scale (a power of
// two) per tile.  A row stands for code * scale.  A tile is one contiguous run
// (8 KB at head_dim 128), so a head's keys are read in whole DRAM bursts
// whatever the number of heads.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace ff {

constexpr int kKv8Block = 64;
// Scale exponents are kept within these bounds: code * scale and its products
// with a query stay normal fp32 numbers, and 448 * 2^112 is finite in bf16.
constexpr int kKv8EMin = -96;
constexpr int kKv8EMax = 112;

// Bits of the handle's device error word (kErrTimeout of ff_ptx.cuh is bit 0).
enum : uint32_t { kErrCapacity = 2u };

struct Kv8Layer {
  uint8_t* k8;
  uint8_t* v8;
  float* ks;
  float* vs;
  int* lengths;          // [batch] rows held
  unsigned int* done;    // [batch] append: blocks finished in the running launch (0 between launches)
  int batch, blocks, capacity, kv_heads;
};

struct Kv8AppendParams {
  Kv8Layer c;
  const void* k;       // bf16 [batch, n, kv_heads, d]
  const void* v;
  const int* start;    // [batch] or null: the rows held
  const int* counts;   // [batch] or null: n
  int n;
  unsigned int* err;
};

struct Kv8LoadParams {
  Kv8Layer c;
  void* k;             // bf16 [batch, n, kv_heads, d]
  void* v;
  const int* start;    // [batch] or null: 0
  int n;
};

struct Kv8EvictParams {
  Kv8Layer src, dst;
  const float* weights;  // [batch, kv_heads, src capacity]
  float* weights_out;    // [batch, kv_heads, dst capacity]
  int* kept;             // [batch, kv_heads, n_keep]
  int n_keep, n_recent;
  int select_keys;       // keys that a selecting block keeps in shared memory
};

// Attention of few query rows.
struct Kv8AttnParams {
  Kv8Layer c;
  const void* q;         // bf16 [batch, n, heads, d]
  void* out;             // bf16 [batch, n, heads, d]
  float* lse;            // [batch, n, heads] or null
  const int* counts;     // [batch] or null: n
  int n, group, causal;
  float scale_log2;      // log2(e) / sqrt(d)
  int per_head;          // key ranges per kv head if all keys were one sequence's; 0: nothing is cut
  float* part_o;         // [thread blocks][rows][d], divided by the part's own sum
  float* part_ml;        // [thread blocks][rows][2]
  unsigned int* tickets; // [batch][kv_heads] finished pieces (0 between launches)
  int2* pieces;          // [batch][kv_heads] first thread block and number of pieces, for the merge of many rows
  float* lse2;           // [batch][n][heads] log2 of the softmax sum, for the weights pass (or null)
};

struct Kv8WeighParams {
  Kv8Layer c;
  const void* q;
  const float* lse2;
  const int* counts;
  const float* weights_in;  // [batch, kv_heads, capacity]
  float* weights;
  int n, group, causal;
  float scale_log2;
  int per_head;             // see Kv8AttnParams
};

// Query rows per kv head up to which the token form runs.  25 rows of four
// sequences (96 MB of keys and values): 36 us, the chunk form 64; 52 rows only fit the
// chunk form's tiles.
constexpr int kKv8TokenRows = 32;
// Up to this many, the chunk form's two groups of softmax warps share one tile of query rows
// and take every other key tile each (52 rows, 23 sequences of 13043 keys: 120 us with
// one group at work, 92 with both).
constexpr int kKv8OneTile = 128;

// Attention of many query rows.  A unit is (sequence, kv head, 256 query rows);
// units 0 .. n_whole - 1 are one piece each, the others are cut into at most
// `splits` key ranges whose partials a second launch merges.
struct Kv8ChunkParams {
  Kv8Layer c;
  const void* q;
  void* out;
  float* lse;
  const int* counts;
  int n, group, causal;
  float scale_log2;
  int row_blocks;        // 256-row blocks per (sequence, kv head)
  int units, n_whole, splits;
  float* part_o;         // [split pieces][d / 4][256][4], divided by the part's own sum
  float* part_ml;        // [split pieces][256][2]
  float* lse2;
  unsigned int* err;
};

// Weights from many query rows: an item is 256 keys and one of at most `splits` ranges of the query rows.
// A tile of query rows is tg heads of the group by tt tokens (tg * tt <= 128).
struct Kv8ChunkWeighParams {
  Kv8Layer c;
  const float* lse2;
  const int* counts;
  const float* weights_in;
  float* weights;
  int n, group, causal;
  float scale_log2;
  int tg, tt, head_tiles;
  int key_tiles, splits, items;  // items: [batch][kv_heads][key_tiles][splits]
  float* part;                   // [items][256]
  unsigned int* tickets;         // [batch][kv_heads][key_tiles][8] finished ranges of 32 keys each (0 between launches)
  unsigned int* err;
};

cudaError_t kv8_configure(int head_dim);
cudaError_t kv8_store_configure();
cudaError_t kv8_chunk_weigh_configure(int head_dim);
// tq: tensor map over q as [batch * n][heads][d], boxes of tt tokens, tg heads and 64 features.
cudaError_t launch_kv8_chunk_weigh(int head_dim, const CUtensorMap& tq, const Kv8ChunkWeighParams& p, int sms,
                                   cudaStream_t s);
cudaError_t launch_kv8_append(int head_dim, const Kv8AppendParams& p, cudaStream_t s);
cudaError_t launch_kv8_load(int head_dim, const Kv8LoadParams& p, cudaStream_t s);
cudaError_t launch_kv8_evict(int head_dim, const Kv8EvictParams& p, int sms, cudaStream_t s);
struct Kv8TokenPlan {
  int per_head, grid;
  int part_blocks;  // thread blocks that may need room for partials
};
Kv8TokenPlan kv8_token_plan(int batch, int kv_heads, int rows, int sms);
cudaError_t launch_kv8_token_attn(int head_dim, const Kv8AttnParams& p, int grid, cudaStream_t s);
cudaError_t kv8_chunk_configure(int head_dim);
cudaError_t launch_kv8_chunk_attn(int head_dim, const Kv8ChunkParams& p, cudaStream_t s);
Kv8TokenPlan kv8_weigh_plan(int batch, int kv_heads, int sms);
cudaError_t launch_kv8_weigh(int head_dim, const Kv8WeighParams& p, int grid, cudaStream_t s);

}  // namespace ff
