// gdn_cache.cuh -- what the kernels of the 8-bit paged cache share: argument blocks, the e4m3
// conversions and the launch declarations.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

// The smallest scale the cache writer stores: a block of zeros keeps a positive scale, so a
// later token of any size re-scales it and the attention never divides by zero.
constexpr float kCacheMinScale = 5.421010862427522e-20f;  // 2^-64
constexpr float kE4m3Max = 448.0f;

struct TablesArgs {
  const int32_t* lens_old;
  const int32_t* lens_new;
  int B;
  int32_t* block_table;
  int max_blocks;
  int32_t* ring;
  int num_blocks;
  const int32_t* pool;
  int32_t* pool_out;
  int block_size;
  int total_tokens;
  int32_t* cu_tokens;
  int32_t* slot_map;
  int32_t* positions;
  int32_t* lens;
  int32_t* err;
};

struct AppendArgs {
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_stride, v_stride;  // elements from one token to the next
  const int32_t* slot_map;
  int T;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scale;
  float* v_scale;
  int num_blocks, H, d, bs;
  int32_t* err;
};

// The cache and the request tables, as the attention calls read them.
struct AttnArgs {
  const uint16_t* q;
  int64_t q_stride;  // elements from one token to the next
  const int32_t* cu_tokens;  // prefill: [B + 1]; decode: null (one token per request)
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* lens;
  int B, T;
  int Hq, H, d, bs, num_blocks;
  float scale;
  uint16_t* out;
  void* workspace;
  int32_t* err;
};

cudaError_t launch_cache_tables(const TablesArgs& a, cudaStream_t s);
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s);
// The largest batch of one gdn_cache_tables call (its per-row sums stay in shared memory).
constexpr int kMaxTableBatch = 8192;

// Requests of one launch; 0 if a single one of that many blocks is too long for its heads.
int attn_decode_batch(int max_blocks, int Hq, int H, int bs);
size_t attn_decode_workspace(int B, int max_blocks, int Hq, int H, int d, int bs);
cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t s);
size_t attn_prefill_workspace(int T, int B, int max_blocks, int Hq, int H, int d, int bs);
cudaError_t launch_attn_prefill(const AttnArgs& a, cudaStream_t s);

// Tensor maps of the two pools as rows of d bytes, read in boxes of 16 rows (the smallest block) or of a
// block's rows by min(d, 128) bytes that land swizzled (128-byte pattern; 64-byte for d = 64) in
// shared memory. Encoded anew for every call; cudaErrorNotSupported if the driver lacks the entry point.
struct CacheMaps {
  CUtensorMap k_group, v_group, k_page, v_page;
};
cudaError_t encode_cache_maps(CacheMaps* maps, const AttnArgs& a);

}  // namespace gdn
