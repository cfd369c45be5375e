// gdn_cache_api.cu -- the C ABI of the paged caches and their attention (include/gdn.h): argument
// checks and error mapping. No allocation, no synchronisation.
#include "gdn_cache.cuh"
#include "gdn_cache4.cuh"

namespace {

// Tokens of a call of the tables or the writer: kernels step past the last one in 32 bits, by a grid's share at most.
constexpr int32_t kMaxTokens = 0x7fffffff - (1 << 20);

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

gdn_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// Shapes of the cache. The q heads only matter to the attention calls.
gdn_status check_cache(const gdn_cache_dims& d, int32_t num_blocks, bool attn) {
  if (d.num_kv_heads <= 0 || d.head_dim <= 0 || d.block_size <= 0 || num_blocks <= 0) return GDN_ERR_INVALID_ARG;
  if (attn && (d.num_q_heads <= 0 || d.num_q_heads % d.num_kv_heads != 0)) return GDN_ERR_INVALID_ARG;
  if (d.head_dim != 64 && d.head_dim != 128 && d.head_dim != 256) return GDN_ERR_UNSUPPORTED;
  if (d.block_size != 16 && d.block_size != 32 && d.block_size != 64 && d.block_size != 128) return GDN_ERR_UNSUPPORTED;
  if (d.num_kv_heads > 1024 || (attn && d.num_q_heads > 1024)) return GDN_ERR_UNSUPPORTED;
  // rows of the cache are addressed by 32-bit TMA coordinates (a box of up to 128 starts past the last one where there is no
  // page), tokens by 32-bit slots
  if (static_cast<int64_t>(num_blocks) * d.num_kv_heads * d.block_size > 0x7fffffffLL - 128) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// The arguments that both attention calls share.
gdn_status check_attn(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                      const float* k_scale, const float* v_scale, int32_t num_blocks,
                      const int32_t* block_table, int32_t max_blocks, const int32_t* lens, int32_t batch,
                      const gdn_cache_dims& d, float scale, void* out, void* workspace, int32_t* err,
                      gdn::AttnArgs& a) {
  const gdn_status st = check_cache(d, num_blocks, true);
  if (st != GDN_OK) return st;
  if (batch < 0 || max_blocks <= 0) return GDN_ERR_INVALID_ARG;
  if (batch > 65535) return GDN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_blocks) * d.block_size > 0x7fffffffLL - 2048) return GDN_ERR_UNSUPPORTED;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !lens || !out || !workspace)
    return GDN_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(d.num_q_heads) * d.head_dim || q_stride % 8 != 0) return GDN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(workspace, 256) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(lens, 4) ||
      !aligned(block_table, 4))
    return GDN_ERR_INVALID_ARG;
  if (!(scale == scale) || scale - scale != 0.0f) return GDN_ERR_INVALID_ARG;  // finite
  a = gdn::AttnArgs{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_table = block_table;
  a.max_blocks = max_blocks;
  a.lens = lens;
  a.B = batch;
  a.T = batch;
  a.Hq = d.num_q_heads;
  a.H = d.num_kv_heads;
  a.d = d.head_dim;
  a.bs = d.block_size;
  a.num_blocks = num_blocks;
  a.scale = scale;
  a.out = static_cast<uint16_t*>(out);
  a.workspace = workspace;
  a.err = err;
  return GDN_OK;
}

// The arrays of a 4-bit cache.
gdn_status check_cache4(const void* k_cache, const void* v_cache, const void* k_scale, const void* v_scale) {
  if (!k_cache || !v_cache || !k_scale || !v_scale) return GDN_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

// Workspace of a prompt call over the 4-bit cache: the table of its requests' pages in 8 bits, those pages, then the 8-bit
// call's own.
struct Prefill4Layout {
  size_t k, v, k_scale, v_scale, rest, total;
  int32_t held;  // pages there is room for; 0: too many for 32-bit rows
};
Prefill4Layout prefill4_layout(int32_t T, int32_t B, int32_t max_blocks, int32_t held, const gdn_cache_dims& d) {
  Prefill4Layout L = {};
  const int64_t most = static_cast<int64_t>(B) * max_blocks;
  const int64_t pages = held < most ? held : most;
  if (pages * d.num_kv_heads * d.block_size > 0x7fffffffLL - 128) return L;
  L.held = static_cast<int32_t>(pages);
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t bytes = static_cast<size_t>(pages) * d.num_kv_heads * d.block_size * d.head_dim;
  const size_t scales = static_cast<size_t>(pages) * d.num_kv_heads * sizeof(float);
  L.k = up(static_cast<size_t>(most) * sizeof(int32_t));
  L.v = up(L.k + bytes);
  L.k_scale = up(L.v + bytes);
  L.v_scale = up(L.k_scale + scales);
  L.rest = up(L.v_scale + scales);
  L.total = L.rest + gdn::attn_prefill_workspace(T, B, max_blocks, d.num_q_heads, d.num_kv_heads, d.head_dim, d.block_size);
  return L;
}

}  // namespace

extern "C" {

gdn_status gdn_cache_tables(const int32_t* lens_old, const int32_t* lens_new, int32_t batch,
                            int32_t* block_table, int32_t max_blocks, int32_t* free_ring,
                            int32_t num_blocks, const int32_t* pool, int32_t* pool_out,
                            int32_t block_size, int32_t total_tokens, int32_t* cu_tokens,
                            int32_t* slot_map, int32_t* positions, int32_t* lens, int32_t* err,
                            void* stream) {
  if (batch < 0 || max_blocks <= 0 || num_blocks <= 0 || total_tokens < 0) return GDN_ERR_INVALID_ARG;
  if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128) return GDN_ERR_UNSUPPORTED;
  if (batch > gdn::kMaxTableBatch || total_tokens > kMaxTokens) return GDN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_blocks) * block_size > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_blocks) * block_size > 0x7fffffffLL - 2048) return GDN_ERR_UNSUPPORTED;
  if (batch == 0) return GDN_OK;
  if (!lens_old || !lens_new || !block_table || !free_ring || !pool || !pool_out || !cu_tokens || !lens)
    return GDN_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!slot_map || !positions)) return GDN_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(lens_old), static_cast<const void*>(lens_new),
                        static_cast<const void*>(block_table), static_cast<const void*>(free_ring),
                        static_cast<const void*>(pool), static_cast<const void*>(pool_out),
                        static_cast<const void*>(cu_tokens), static_cast<const void*>(slot_map),
                        static_cast<const void*>(positions), static_cast<const void*>(lens)})
    if (!aligned(p, 4)) return GDN_ERR_INVALID_ARG;
  gdn::TablesArgs a{lens_old, lens_new, batch, block_table, max_blocks, free_ring, num_blocks,
                    pool, pool_out, block_size, total_tokens, cu_tokens, slot_map, positions,
                    lens, err};
  return from_cuda(gdn::launch_cache_tables(a, static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_cache_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            const int32_t* slot_map, int32_t total_tokens, void* k_cache,
                            void* v_cache, float* k_scale, float* v_scale, int32_t num_blocks,
                            gdn_cache_dims dims, int32_t* err, void* stream) {
  const gdn_status st = check_cache(dims, num_blocks, false);
  if (st != GDN_OK) return st;
  if (total_tokens < 0) return GDN_ERR_INVALID_ARG;
  if (total_tokens > kMaxTokens) return GDN_ERR_UNSUPPORTED;
  if (total_tokens == 0) return GDN_OK;
  if (!k || !v || !slot_map || !k_cache || !v_cache || !k_scale || !v_scale) return GDN_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(dims.num_kv_heads) * dims.head_dim;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0) return GDN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(slot_map, 4))
    return GDN_ERR_INVALID_ARG;
  gdn::AppendArgs a{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_stride, v_stride,
                    slot_map, total_tokens, static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache),
                    k_scale, v_scale, num_blocks, dims.num_kv_heads, dims.head_dim, dims.block_size, err};
  return from_cuda(gdn::launch_cache_append(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_attn_decode_workspace_size(int32_t batch, int32_t max_blocks, gdn_cache_dims dims) {
  if (batch <= 0 || max_blocks <= 0 || check_cache(dims, 1, true) != GDN_OK) return 0;
  if (gdn::attn_decode_batch(max_blocks, dims.num_q_heads, dims.num_kv_heads, dims.block_size) == 0) return 0;
  return gdn::attn_decode_workspace(batch, max_blocks, dims.num_q_heads, dims.num_kv_heads, dims.head_dim,
                                    dims.block_size);
}

gdn_status gdn_attn_decode(const void* q, int64_t q_stride, const void* k_cache,
                           const void* v_cache, const float* k_scale, const float* v_scale,
                           int32_t num_blocks, const int32_t* block_table, int32_t max_blocks,
                           const int32_t* lens, int32_t batch, gdn_cache_dims dims, float scale,
                           void* out, void* workspace, size_t workspace_bytes, int32_t* err,
                           void* stream) {
  if (batch == 0) return GDN_OK;
  gdn::AttnArgs a;
  const gdn_status st = check_attn(q, q_stride, k_cache, v_cache, k_scale, v_scale, num_blocks, block_table,
                                   max_blocks, lens, batch, dims, scale, out, workspace, err, a);
  if (st != GDN_OK) return st;
  if (gdn::attn_decode_batch(max_blocks, dims.num_q_heads, dims.num_kv_heads, dims.block_size) == 0) return GDN_ERR_UNSUPPORTED;
  if (workspace_bytes < gdn_attn_decode_workspace_size(batch, max_blocks, dims)) return GDN_ERR_INVALID_ARG;
  return from_cuda(gdn::launch_attn_decode(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_attn_prefill_workspace_size(int32_t total_tokens, int32_t num_seqs, int32_t max_blocks,
                                       gdn_cache_dims dims) {
  if (total_tokens < 0 || num_seqs <= 0 || max_blocks <= 0 || check_cache(dims, 1, true) != GDN_OK) return 0;
  return gdn::attn_prefill_workspace(total_tokens, num_seqs, max_blocks, dims.num_q_heads, dims.num_kv_heads,
                                     dims.head_dim, dims.block_size);
}

gdn_status gdn_attn_prefill(const void* q, int64_t q_stride, const int32_t* cu_tokens,
                            const void* k_cache, const void* v_cache, const float* k_scale,
                            const float* v_scale, int32_t num_blocks, const int32_t* block_table,
                            int32_t max_blocks, const int32_t* lens, int32_t num_seqs,
                            int32_t total_tokens, gdn_cache_dims dims, float scale, void* out,
                            void* workspace, size_t workspace_bytes, int32_t* err, void* stream) {
  if (total_tokens < 0 || num_seqs < 0) return GDN_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_tokens == 0) return GDN_OK;
  gdn::AttnArgs a;
  const gdn_status st = check_attn(q, q_stride, k_cache, v_cache, k_scale, v_scale, num_blocks, block_table,
                                   max_blocks, lens, num_seqs, dims, scale, out, workspace, err, a);
  if (st != GDN_OK) return st;
  if (!cu_tokens || !aligned(cu_tokens, 4)) return GDN_ERR_INVALID_ARG;
  // a request's (token, head) rows are counted in 32 bits
  if (static_cast<int64_t>(total_tokens) * dims.num_q_heads > 0x7fffffffLL - 65536) return GDN_ERR_UNSUPPORTED;
  if (workspace_bytes < gdn_attn_prefill_workspace_size(total_tokens, num_seqs, max_blocks, dims))
    return GDN_ERR_INVALID_ARG;
  a.cu_tokens = cu_tokens;
  a.T = total_tokens;
  return from_cuda(gdn::launch_attn_prefill(a, nullptr, static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_cache4_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const int32_t* slot_map, int32_t total_tokens, void* k_cache,
                             void* v_cache, uint8_t* k_scale, uint8_t* v_scale, int32_t num_blocks,
                             gdn_cache_dims dims, int32_t* err, void* stream) {
  gdn_status st = check_cache(dims, num_blocks, false);
  if (st != GDN_OK) return st;
  if (total_tokens < 0) return GDN_ERR_INVALID_ARG;
  if (total_tokens > kMaxTokens) return GDN_ERR_UNSUPPORTED;
  if (total_tokens == 0) return GDN_OK;
  if (!k || !v || !slot_map) return GDN_ERR_INVALID_ARG;
  st = check_cache4(k_cache, v_cache, k_scale, v_scale);
  if (st != GDN_OK) return st;
  const int64_t row = static_cast<int64_t>(dims.num_kv_heads) * dims.head_dim;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0) return GDN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4)) return GDN_ERR_INVALID_ARG;
  gdn::Append4Args a{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_stride, v_stride, slot_map, total_tokens,
                     {static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), k_scale, v_scale, num_blocks,
                      dims.num_kv_heads, dims.head_dim, dims.block_size},
                     err};
  return from_cuda(gdn::launch_cache4_append(a, static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_cache4_read(const void* k_cache, const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                           int32_t num_blocks, const int32_t* slot_map, int32_t total_tokens, gdn_cache_dims dims,
                           void* k, int64_t k_stride, void* v, int64_t v_stride, int32_t* err, void* stream) {
  gdn_status st = check_cache(dims, num_blocks, false);
  if (st != GDN_OK) return st;
  if (total_tokens < 0) return GDN_ERR_INVALID_ARG;
  if (total_tokens > kMaxTokens) return GDN_ERR_UNSUPPORTED;
  if (total_tokens == 0) return GDN_OK;
  if (!k || !v || !slot_map) return GDN_ERR_INVALID_ARG;
  st = check_cache4(k_cache, v_cache, k_scale, v_scale);
  if (st != GDN_OK) return st;
  const int64_t row = static_cast<int64_t>(dims.num_kv_heads) * dims.head_dim;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0) return GDN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4)) return GDN_ERR_INVALID_ARG;
  gdn::Read4Args a{{static_cast<uint8_t*>(const_cast<void*>(k_cache)), static_cast<uint8_t*>(const_cast<void*>(v_cache)),
                    const_cast<uint8_t*>(k_scale), const_cast<uint8_t*>(v_scale), num_blocks, dims.num_kv_heads, dims.head_dim,
                    dims.block_size},
                   slot_map, total_tokens, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), k_stride, v_stride, err};
  return from_cuda(gdn::launch_cache4_read(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_attn4_decode_workspace_size(int32_t batch, int32_t max_blocks, gdn_cache_dims dims) {
  if (batch <= 0 || max_blocks <= 0 || check_cache(dims, 1, true) != GDN_OK) return 0;
  if (gdn::attn_decode_batch(max_blocks, dims.num_q_heads, dims.num_kv_heads, dims.block_size) == 0) return 0;
  return gdn::attn4_decode_workspace(batch, max_blocks, dims.num_q_heads, dims.num_kv_heads, dims.head_dim,
                                     dims.block_size);
}

gdn_status gdn_attn4_decode(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                            const uint8_t* k_scale, const uint8_t* v_scale, int32_t num_blocks,
                            const int32_t* block_table, int32_t max_blocks, const int32_t* lens,
                            int32_t batch, gdn_cache_dims dims, float scale, void* out,
                            void* workspace, size_t workspace_bytes, int32_t* err, void* stream) {
  if (batch == 0) return GDN_OK;
  gdn::AttnArgs a;
  gdn_status st = check_attn(q, q_stride, k_cache, v_cache, reinterpret_cast<const float*>(k_scale),
                             reinterpret_cast<const float*>(v_scale), num_blocks, block_table, max_blocks, lens, batch, dims,
                             scale, out, workspace, err, a);
  if (st == GDN_OK) st = check_cache4(k_cache, v_cache, k_scale, v_scale);
  if (st != GDN_OK) return st;
  if (gdn::attn_decode_batch(max_blocks, dims.num_q_heads, dims.num_kv_heads, dims.block_size) == 0) return GDN_ERR_UNSUPPORTED;
  if (workspace_bytes < gdn_attn4_decode_workspace_size(batch, max_blocks, dims)) return GDN_ERR_INVALID_ARG;
  return from_cuda(gdn::launch_attn4_decode(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_attn4_prefill_workspace_size(int32_t total_tokens, int32_t num_seqs, int32_t max_blocks, int32_t held_blocks,
                                        gdn_cache_dims dims) {
  if (total_tokens < 0 || num_seqs <= 0 || max_blocks <= 0 || held_blocks <= 0 || check_cache(dims, 1, true) != GDN_OK) return 0;
  return prefill4_layout(total_tokens, num_seqs, max_blocks, held_blocks, dims).total;
}

gdn_status gdn_attn4_prefill(const void* q, int64_t q_stride, const int32_t* cu_tokens,
                             const void* k_cache, const void* v_cache, const uint8_t* k_scale,
                             const uint8_t* v_scale, int32_t num_blocks, const int32_t* block_table,
                             int32_t max_blocks, const int32_t* lens, int32_t num_seqs,
                             int32_t total_tokens, int32_t held_blocks, gdn_cache_dims dims, float scale, void* out,
                             void* workspace, size_t workspace_bytes, int32_t* err, void* stream) {
  if (total_tokens < 0 || num_seqs < 0 || held_blocks < 0) return GDN_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_tokens == 0) return GDN_OK;
  if (held_blocks == 0) return GDN_ERR_INVALID_ARG;
  gdn::AttnArgs a;
  gdn_status st = check_attn(q, q_stride, k_cache, v_cache, reinterpret_cast<const float*>(k_scale),
                             reinterpret_cast<const float*>(v_scale), num_blocks, block_table, max_blocks, lens, num_seqs, dims,
                             scale, out, workspace, err, a);
  if (st == GDN_OK) st = check_cache4(k_cache, v_cache, k_scale, v_scale);
  if (st != GDN_OK) return st;
  if (!cu_tokens || !aligned(cu_tokens, 4)) return GDN_ERR_INVALID_ARG;
  if (num_seqs > gdn::kExpandBatch) return GDN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(total_tokens) * dims.num_q_heads > 0x7fffffffLL - 65536) return GDN_ERR_UNSUPPORTED;
  const Prefill4Layout L = prefill4_layout(total_tokens, num_seqs, max_blocks, held_blocks, dims);
  if (L.held == 0) return GDN_ERR_UNSUPPORTED;
  if (workspace_bytes < L.total) return GDN_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  gdn::Expand4Args x{};
  x.c = {static_cast<uint8_t*>(const_cast<void*>(k_cache)), static_cast<uint8_t*>(const_cast<void*>(v_cache)),
         const_cast<uint8_t*>(k_scale), const_cast<uint8_t*>(v_scale), num_blocks, dims.num_kv_heads, dims.head_dim, dims.block_size};
  x.block_table = block_table;
  x.max_blocks = max_blocks;
  x.lens = lens;
  x.cu_tokens = cu_tokens;
  x.B = num_seqs;
  x.T = total_tokens;
  x.held = L.held;
  x.table = reinterpret_cast<int32_t*>(ws);
  x.k = ws + L.k;
  x.v = ws + L.v;
  x.k_scale = reinterpret_cast<float*>(ws + L.k_scale);
  x.v_scale = reinterpret_cast<float*>(ws + L.v_scale);
  x.err = err;
  a.cu_tokens = cu_tokens;
  a.T = total_tokens;
  a.k_cache = x.k;
  a.v_cache = x.v;
  a.k_scale = x.k_scale;
  a.v_scale = x.v_scale;
  a.block_table = x.table;
  a.num_blocks = L.held;
  a.workspace = ws + L.rest;
  return from_cuda(gdn::launch_attn_prefill(a, &x, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
