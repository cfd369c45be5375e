// gdn_attn_decode.cu -- attention of single tokens over the 8-bit paged cache, on the tcgen05 tensor
// cores.
//
// Per request b (len keys), kv head h and the G query heads that share it:
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),  k_j = ks * byte, v_j = vs * byte
// with one ks, vs per (block, kv head). Bound by memory: every cached byte is read once
// (2 d bytes per token and kv head) for 4 G operations per byte, so the kernel's job is to keep
// copies in flight and to spend few instructions on a byte. It spends none: a tile of 128 keys goes by
// TMA (page by page: pages end inside a tile) to shared memory and from
// there, as 8-bit operands, into two products,
//   S^T[key, head] = K Q^T  (M = 128 keys, N = query heads, K = d)
//   O^T[d, head]  += V^T P^T (M = 128 of d, N = query heads, K = 128 keys),
// keys and d on the 128-row side, the few query heads on the narrow one, so G <= 8 wastes nothing
// that matters. K is used K-major and V MN-major, both as they lie in the page. A first version
// that converted K and V to f16 for the warp-level instruction spent 640 instructions on 8 KB and stopped at
// 5.1 TB/s (256 requests of about 8,000 tokens); this one spends about 60.
//
// Eight-bit queries and probabilities are split into parts, side by side in N: a query into two e4m3
// values (scaled per head so that its largest element lies in [128, 256): exact down to 2^-18 of that),
// a probability into four with factors 1, 1/32, 1/32^2, 1/32^3 (16 bits, and 2^-26 of the largest).
//
// Scales of V. With x the exponent of a score and e that of vs, m is the running maximum of x + e, and p = exp2(x - m)
// goes into the sum, p vs into the product. So what a key is rounded to goes by the largest probability x scale of the row, and
// not by a scale that weighs nothing. m stands for 2^1.8 and moves when an x + e passes it by 2^5, so that almost only a
// unit's first tile stops for it. So p vs < 2^6.8 * 2 < 256, what a part leaves of it is at most 8, and 32 times that 256
// again. (With 2^8 above 2^-0.2 and factors of 1/16, at the same speed, keys below 2^-22 of the largest were lost.)
//
// Split. A (request, kv head) is cut into units of 256, 512 or 1,024 keys by its OWN length
// (unit_shift), never by the batch: a row's result depends on its own inputs alone, bit for bit, as
// for every other call of the library. A persistent grid walks the units. A request of one unit is
// finished here, a longer one leaves fp32 partial sums (with their maximum and sum) that a second,
// programmatically dependent kernel joins in unit order.
//
// Measured: 256 requests of up to 8,192 tokens (16 / 2 heads of 256) 347 us, 5.7 TB/s, where the same copies without
// the products take 297; 2 of 131,071 56 us; one of 4,097 13.1 us, a chain of set-up (2,000 cycles), two lookups (1,600), copy,
// two tiles (2,300 each), stores and the join.
//
// Roles of a CTA: four softmax warps (thread = key, then thread = d), one warp that issues MMAs, one that
// issues TMA, one that looks up pages and scales (four tiles at a time, a lane per 16 keys: a lookup is
// two dependent loads from memory), one that converts queries a unit ahead. Scores of the next tile are
// computed while this one's softmax runs; lookups and copies run ahead across units. A TMA instruction
// takes about 60 cycles to issue whatever its box, so a whole page is one box (two for d = 256) and
// only a request's last page goes in boxes of 16 keys.
#include <cudaTypedefs.h>

#include <atomic>

#include "gdn_attn.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

cudaError_t encode_cache_map(CUtensorMap* map, const uint8_t* cache, int64_t total_rows, int d, int rows) {
  static std::atomic<void*> entry{nullptr};  // the driver's function, looked up once
  void* fn = entry.load(std::memory_order_acquire);
  if (!fn) {
    cudaDriverEntryPointQueryResult found;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    entry.store(fn, std::memory_order_release);
  }
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(total_rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(d < 128 ? d : 128), static_cast<cuuint32_t>(rows)};
  const cuuint32_t step[2] = {1, 1};
  auto encode = [&] {
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
        map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(cache), dims, strides, box, step,
        CU_TENSOR_MAP_INTERLEAVE_NONE, d < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) {
    // a driver's function on a host thread that has made no call of the runtime yet, whose context is current from then on
    int device;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess) e = cudaSetDevice(device);
    if (e != cudaSuccess) return e;
    r = encode();
  }
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

std::atomic<int>& attention_test_fault() {
  static std::atomic<int> mode{0};
  return mode;
}

cudaError_t encode_cache_maps(CacheMaps* maps, const AttnArgs& a) {
  const int64_t rows = static_cast<int64_t>(a.num_blocks) * a.H * a.bs;
  cudaError_t e = encode_cache_map(&maps->k_group, a.k_cache, rows, a.d, kGroup);
  if (e == cudaSuccess) e = encode_cache_map(&maps->v_group, a.v_cache, rows, a.d, kGroup);
  if (e == cudaSuccess) e = encode_cache_map(&maps->k_page, a.k_cache, rows, a.d, a.bs);
  if (e == cudaSuccess) e = encode_cache_map(&maps->v_page, a.v_cache, rows, a.d, a.bs);
  return e;
}

namespace {

constexpr int kMaxUnitKeys = 1024;
// Requests of one launch. Their lengths stay in shared memory, next to what two CTAs an SM leave of it (static_assert
// below): with 384, batches of 330 to 384 ran one CTA an SM (384 requests of 2,000 tokens, 16 / 2 heads of 256: 205 us,
// and 167 in two launches).
constexpr int kBatchPerLaunch = 320;
constexpr int kCoarse = 16;            // requests between two kept tile sums
constexpr int kThreads = 32 * 8;
constexpr int kSmemPerSm = 228 * 1024;  // 1 KB of it taken by each resident CTA
constexpr float kRise = 5.0f;          // log2 of what a score may pass the running maximum by
constexpr float kTop = 1.8f;           // log2 of what the running maximum stands for

// log2 of the keys of one unit of a request of `len` keys, and its units. Small units shorten the chain of tiles
// that a small batch waits for, and cost a large one partial sums (d = 256, 8 query heads a kv head: 8 KB a unit next
// to 128 KB of cache for 256 keys). Units of 256 and 512 keys at length 4,097, one request: 13.5 and 17.9 us; up
// to 8,192, 256 requests: 410 and 350 us. So 256 up to 24 units, then 512 up to 24, then 1,024.
constexpr int kFewUnits = 24;
__host__ __device__ __forceinline__ int unit_shift(int len) { return len <= kFewUnits << 8 ? 8 : len <= kFewUnits << 9 ? 9 : 10; }
__host__ __device__ __forceinline__ int units_of(int len) {
  const int s = unit_shift(len);
  return (len + (1 << s) - 1) >> s;
}
// The most units that any length up to `cap` has.
int64_t most_units(int64_t cap) {
  if (cap <= kFewUnits << 8) return (cap + 255) / 256;
  return cap <= kFewUnits << 10 ? kFewUnits : (cap + kMaxUnitKeys - 1) / kMaxUnitKeys;
}

struct DecodeParams {
  AttnArgs a;
  int heads;      // query heads of one unit: min(G, 16)
  int chunks;     // units' head chunks per kv head: ceil(G / 16)
  int b0, nb;     // the launch's requests
  int fault;      // test hook: CTA 0 looks up one batch of tiles and no more
  int each;       // the most units of a request's (kv head, chunk): unit u of it has slot (b * HC + hc) * each + u
  float2* ml;     // workspace: [slots][heads] (maximum, sum) of a unit that is one of several
  float* part;    // [slots][heads][D]
};

__host__ __device__ constexpr int tmem_columns(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : n <= 256 ? 256 : 512; }

// HP: the unit's query heads, padded to 4, 8 or 16.
template <int D, int HP>
struct DecodeCfg {
  static constexpr int kNQ = HP == 16 ? 32 : 16;                 // columns of S^T: high parts, low parts
  static constexpr int kNP = 4 * HP;                             // columns of O^T: four parts
  static constexpr int kHalves = D == 256 ? 2 : 1;               // of d, 128 rows each
  // Tiles of keys or values in the ring: two CTAs an SM (their latencies overlap) with 96 KB each where they fit.
  static constexpr int kStages = D == 256 ? (HP == 16 ? 6 : 3) : HP == 16 ? 5 : 6;
  static constexpr int kStage = Tile<D>::kBytes;
  static constexpr int kQ = kNQ * D;
  static constexpr int kP = kTile * kNP;
  static constexpr int kBatch = 4;                               // tiles looked up at a time
  static constexpr int kBatches = 4;                             // batches that are kept
  static constexpr int kInfoRing = kBatch * kBatches;
  static constexpr int kFactorRing = 4;                          // units whose query factors are kept
  static constexpr int kColumns = tmem_columns(2 * kNQ + kHalves * kNP);
  static constexpr int kO = 2 * kNQ;                             // first column of O^T
  // shared memory, after alignment to 1,024 bytes (the swizzle repeats)
  static constexpr int kAtQ = kStages * kStage;
  static constexpr int kAtP = kAtQ + 2 * kQ;
  static constexpr int kAtScale = kAtP + kP;
  static constexpr int kAtRow = kAtScale + kInfoRing * kGroups * 8;
  static constexpr int kAtKeys = kAtRow + kInfoRing * kGroups * 4;
  static constexpr int kAtFactor = kAtKeys + kInfoRing * 4;
  static constexpr int kAtRed = kAtFactor + kFactorRing * 16 * 4;
  static constexpr int kBars = 2 * kStages + 2 * kBatches + kFactorRing + 11;
  static constexpr int kAtSum = kAtRed + 4 * 16 * 4;
  static constexpr int kAtBars = kAtSum + 4 * 16 * 4;
  static constexpr int kAtPre = kAtBars + kBars * 8;             // then lens[nb], tsum[nb / kCoarse + 2]
  static constexpr int kSmem = 1024 + kAtPre;
  static constexpr int smem_of(int nb) { return kSmem + 4 * (nb + nb / kCoarse + 2); }
  static_assert(kAtBars % 8 == 0 && kQ % 1024 == 0, "alignment");
  // (128: what the kernel declares itself)
  static_assert(HP == 16 || 2 * (smem_of(kBatchPerLaunch) + 128 + 1024) <= kSmemPerSm, "two CTAs an SM");
};

// The units of one CTA, in order: those whose first tile lies in its equal share of the launch's tiles (all
// requests, kv heads and head chunks end to end). A share holds whole units, so CTAs differ by a unit's
// tiles at most, and neighbours in a CTA are neighbours in memory.
struct Walk {
  const int32_t* lens;
  const int32_t* tsum;  // tiles before request kCoarse * i
  int nb, end;
  int H, chunks;
  int b, h, chunk, index;  // request, kv head, head chunk, the unit's place in its (request, head, chunk)
  int len, shift, count;   // the request's keys, log2 of the keys of a unit, units
  int pos;              // the unit's first tile

  __device__ __forceinline__ static int tiles_of(int len) { return (len + kTile - 1) / kTile; }
  __device__ __forceinline__ void request() {
    len = lens[b];
    shift = unit_shift(len);
    count = units_of(len);
  }
  __device__ __forceinline__ void next_head() {
    index = 0;
    if (++chunk == chunks) {
      chunk = 0;
      ++h;
    }
    if (h == H) {
      h = 0;
      do ++b;
      while (b < nb && lens[b] == 0);
      if (b == nb) {
        pos = end;
        return;
      }
      request();
    }
  }
  __device__ __forceinline__ void start(int share, int shares) {
    const int HC = H * chunks;
    const int all = tsum[(nb + kCoarse - 1) / kCoarse] * HC, each = all / shares, more = all - each * shares;
    const int from = each * share + min(share, more);
    end = from + each + (share < more);
    pos = from;
    if (from == end) return;
    // the last request whose tiles start at or before `from`: not an empty one
    int lo = 0;
#pragma unroll 1
    while ((lo + 1) * kCoarse < nb && tsum[lo + 1] * HC <= from) ++lo;
    int before = tsum[lo];
    b = lo * kCoarse;
#pragma unroll 1
    while ((before + tiles_of(lens[b])) * HC <= from) before += tiles_of(lens[b++]);
    request();
    const int tiles = tiles_of(len), rem = from - before * HC, ut = shift - 7;  // (a tile is 2^7 keys)
    const int hc = rem / tiles, in = rem - hc * tiles;
    h = hc / chunks;
    chunk = hc - h * chunks;
    index = (in + (1 << ut) - 1) >> ut;
    pos += min(index << ut, tiles) - in;
    if (index == count) next_head();
  }
  __device__ __forceinline__ bool more() const { return pos < end; }
  __device__ __forceinline__ void next() {
    pos += tiles();
    if (++index == count) next_head();
  }
  __device__ __forceinline__ int first() const { return index << shift; }
  __device__ __forceinline__ int keys() const { return min(1 << shift, len - first()); }
  __device__ __forceinline__ int tiles() const { return (keys() + kTile - 1) / kTile; }
};

__device__ __forceinline__ bool any_of_128(bool x) {  // over the softmax warps
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(x))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sync_128() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(x));
  return r;
}
// two values to e4m3 (RNE); the values that the bytes stand for are taken off and the rest is scaled by 32
__device__ __forceinline__ uint32_t split_off(float& a, float& b) {
  uint32_t r, w;
  asm("{.reg .b16 x; cvt.rn.satfinite.e4m3x2.f32 x, %3, %2; cvt.rn.f16x2.e4m3x2 %1, x; mov.b32 %0, {x, 0};}"
      : "=r"(r), "=r"(w) : "f"(a), "f"(b));
  float fa, fb;
  asm("{.reg .b16 x, y; mov.b32 {x, y}, %2; cvt.f32.f16 %0, x; cvt.f32.f16 %1, y;}" : "=f"(fa), "=f"(fb) : "r"(w));
  a = (a - fa) * 32.0f;
  b = (b - fb) * 32.0f;
  return r;
}
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[N]) {
  if constexpr (N % 32 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 32) tmem_ld32(taddr + i, v + i);
  } else {
    static_assert(N == 16, "16 columns, or multiples of 32");
    tc::tmem_ld16(taddr, v);
  }
  tc::tmem_wait_ld();
}

template <int D, int HP>
__global__ void __launch_bounds__(kThreads) attn_decode_kernel(const __grid_constant__ DecodeParams p,
                                                               const __grid_constant__ CacheMaps maps) {
  using C = DecodeCfg<D, HP>;
  using TL = Tile<D>;
  using TQ = Tile<D, C::kNQ>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + (-smem_addr(smem_raw) & 1023u);
  const uint32_t base = smem_addr(smem), s_q = base + C::kAtQ, s_p = base + C::kAtP;
  float2* s_scale = reinterpret_cast<float2*>(smem + C::kAtScale);  // [tile % kInfoRing][group] (ks, vs)
  int32_t* s_row = reinterpret_cast<int32_t*>(smem + C::kAtRow);    // [tile % kInfoRing][group] row of the cache
  int32_t* s_keys = reinterpret_cast<int32_t*>(smem + C::kAtKeys);  // [tile % kInfoRing] keys of the tile, 0: no more
  float* s_factor = reinterpret_cast<float*>(smem + C::kAtFactor);  // [unit % kFactorRing][16]
  // [warp][16], a tile's maxima and a unit's sums: apart, as no barrier lies between the reads of the last tile's
  // maxima and the writes of the sums
  float* s_red = reinterpret_cast<float*>(smem + C::kAtRed);
  float* s_sum = reinterpret_cast<float*>(smem + C::kAtSum);
  int32_t* lens = reinterpret_cast<int32_t*>(smem + C::kAtPre);
  int32_t* tsum = lens + p.nb;
  const uint32_t b_full = base + C::kAtBars, b_empty = b_full + 8 * C::kStages, b_info = b_empty + 8 * C::kStages,
                 b_infoe = b_info + 8 * C::kBatches, b_factor = b_infoe + 8 * C::kBatches, b_s = b_factor + 8 * C::kFactorRing, b_p = b_s + 16,
                 b_pv = b_p + 8, b_qfull = b_pv + 16, b_qempty = b_qfull + 16, b_drain = b_qempty + 16;
  __shared__ int32_t s_scan[kThreads / 32];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_fail;

  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // (known to be the same in a warp)
  const int cap = a.max_blocks * a.bs;

  int len = tid < p.nb ? a.lens[p.b0 + tid] : 0;  // (on its way under the set-up)
  if (tid < 4) prefetch_map(tid == 0 ? &maps.k_page : tid == 1 ? &maps.v_page : tid == 2 ? &maps.k_group : &maps.v_group);
  if (tid < C::kBars) {
    // who arrives: a copy, a commit or one lane, but for what warps and threads release themselves
    const uint32_t bar = b_full + 8 * tid;
    mbar_init(bar, bar >= b_infoe && bar < b_factor ? 4 : bar == b_p ? 128 : bar >= b_qfull && bar < b_qempty ? 32 : 1);
  }
  if (tid == 0) s_fail = 0;
  fence_mbar_init();
  if (warp == 4) {
    tc::tmem_alloc(&s_tmem, C::kColumns);
    tc::tmem_relinquish();
  }
  // lengths, and tiles before every kCoarse-th request
  {
    int carry = 0, flags = 0;
    for (int at = 0; at < p.nb; at += kThreads) {
      const int b = at + tid;
      if (at > 0) len = b < p.nb ? a.lens[p.b0 + b] : 0;
      if (b < p.nb) {
        if (len < 0 || len > cap) flags = GDN_DEVERR_SEQLENS;
        len = min(max(len, 0), cap);
        lens[b] = len;
      }
      int v = Walk::tiles_of(len);
      const int own = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += x;
      }
      if (lane == 31) s_scan[warp] = v;
      __syncthreads();
      int before = carry;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        carry += s_scan[w];
      }
      if (b < p.nb && b % kCoarse == 0) tsum[b / kCoarse] = before + v - own;
      __syncthreads();
    }
    if (tid == 0) tsum[(p.nb + kCoarse - 1) / kCoarse] = carry;
    if (flags && a.err && blockIdx.x == 0) atomicOr(a.err, flags);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel may take its place

  const int G = a.Hq / a.H;
  __shared__ Walk s_walk;  // where every role starts
  if (tid == 0) {
    Walk w;
    w.lens = lens;
    w.tsum = tsum;
    w.nb = p.nb;
    w.H = a.H;
    w.chunks = p.chunks;
    w.start(blockIdx.x, gridDim.x);
    s_walk = w;
  }
  __syncthreads();
  auto walk = [&]() { return s_walk; };
  // a unit's first query head, and its query heads
  auto first_head = [&](const Walk& w) { return w.h * G + w.chunk * 16; };
  auto unit_heads = [&](const Walk& w) { return min(p.heads, G - w.chunk * 16); };
  auto wait = [&](uint32_t b, int parity) { return wait_or_fail(b, parity, &s_fail); };
  // the ring's n-th use: keys of tile i are use 2 i, its values 2 i + 1
  auto full = [&](int n) { return b_full + 8 * (n % C::kStages); };
  auto empty = [&](int n) { return b_empty + 8 * (n % C::kStages); };
  auto phase = [&](int n) { return (n / C::kStages) & 1; };

  int copies = 0;  // of the copying warp
  if (warp == 7) {
    // ---- lookups: lane = (tile of the batch, 16-key group)
    const int none = a.num_blocks * a.H * a.bs;  // a row past the cache: zeros
    const int shift = 31 - __clz(a.bs);
    Walk w = walk();
    int t = 0;  // the next tile of the walk's unit
    bool ok = true;
    for (int batch = 0; ok; ++batch) {
      if (p.fault && blockIdx.x == 0 && batch == 1) break;
      int keys = 0, pos = 0, b = 0, h = 0;  // this lane's tile
#pragma unroll 1
      for (int j = 0; j < C::kBatch && w.more(); ++j) {
        if (j == lane / kGroups) {
          keys = min(kTile, w.keys() - t * kTile);
          pos = w.first() + t * kTile + (lane % kGroups) * kGroup;
          b = w.b;
          h = w.h;
        }
        if (++t == w.tiles()) {
          t = 0;
          w.next();
        }
      }
      const bool last = __shfl_sync(0xFFFFFFFFu, keys, 31) == 0;  // a batch with room left: the end is in it
      int row = none;
      float2 sc = make_float2(-1.0f, 0.0f);  // a page that is none, or no key: not seen
      if ((lane % kGroups) * kGroup < keys) {
        const int page = a.block_table[static_cast<int64_t>(p.b0 + b) * a.max_blocks + (pos >> shift)];
        if (page >= 0 && page < a.num_blocks) {
          const int64_t at = static_cast<int64_t>(page) * a.H + h;
          sc = make_float2(a.k_scale[at], a.v_scale[at]);
          row = (static_cast<int>(at) << shift) + (pos & (a.bs - 1));
        } else if (a.err) {
          atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);
        }
      }
      const int slot = batch % C::kBatches;
      ok = __all_sync(0xFFFFFFFFu, wait(b_infoe + 8 * slot, ((batch / C::kBatches) & 1) ^ 1));
      if (!ok) break;
      s_scale[slot * 32 + lane] = sc;
      s_row[slot * 32 + lane] = row;
      if (lane % kGroups == 0) s_keys[slot * C::kBatch + lane / kGroups] = keys;
      __syncwarp();
      if (lane == 0) mbar_arrive(b_info + 8 * slot);
      if (last) break;
    }
  } else if (warp == 5) {
    // ---- copies: lane g < 8 has the 16-key group g of each tile
    const int rows = a.bs;                                 // of a page
    const bool head = ((lane * kGroup) & (rows - 1)) == 0; // the group starts a page
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (i % C::kBatch == 0) ok = __all_sync(0xFFFFFFFFu, wait(b_info + 8 * ((i / C::kBatch) % C::kBatches), (i / C::kInfoRing) & 1));
      if (!ok) break;
      const int keys = s_keys[i % C::kInfoRing];
      if (keys == 0) break;
      const int row = s_row[(i % C::kInfoRing) * kGroups + lane % kGroups];
      const bool whole = ((lane * kGroup) & -rows) + rows <= keys;  // every token of the group's page is the request's
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const int n = 2 * i + which;
        ok = __all_sync(0xFFFFFFFFu, wait(empty(n), phase(n) ^ 1));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(full(n), C::kStage);
        __syncwarp();
        if (lane < kGroups && (head || !whole)) {
          const CUtensorMap* map = which ? (whole ? &maps.v_page : &maps.v_group) : (whole ? &maps.k_page : &maps.k_group);
#pragma unroll
          for (int x = 0; x < D; x += 128)
            tma_rows(base + (n % C::kStages) * C::kStage + (x / 128) * TL::kHalf + lane * kGroup * TL::kRow, map, x, row, full(n));
        }
        copies = n + 1;
      }
    }
  } else if (warp == 4) {
    // ---- MMAs
    constexpr uint32_t iqk = idesc_f8(128, C::kNQ, false, false), ipv = idesc_f8(128, C::kNP, true, true);
    bool ok = true;
    // descriptors but for their start address (bits 0 .. 13, in 16 bytes), which each MMA adds
    const uint64_t dk = TL::desc(base, 16), dq = TQ::desc(s_q, 16), dv = TL::desc(base, 512), dp = tc::smem_desc(s_p, 128, kTile * 16);
    auto k_off = [](int ks, int half) { return static_cast<uint64_t>((ks / (TL::kRow / 32)) * half + (ks % (TL::kRow / 32)) * 32) >> 4; };
    int qi = 0;             // tiles whose scores are issued
    Walk qw = walk();       // where that stands: unit,
    int qk_k = 0, qk_t = 0; // its number, tile
    auto qk = [&]() {       // scores of the next tile, if there is one
      if (!qw.more()) return true;
      if (qk_t == 0 && !wait(b_qfull + 8 * (qk_k & 1), (qk_k >> 1) & 1)) return false;
      const int n = 2 * qi;
      if (!wait(full(n), phase(n))) return false;
      tc::fence_after_sync();
      const bool last = qk_t + 1 == qw.tiles();
      if (lane == 0) {
        const uint64_t kt = dk + (n % C::kStages) * (C::kStage >> 4), qt = dq + (qk_k & 1) * (C::kQ >> 4);
        const uint32_t d = tmem + C::kNQ * (qi & 1);
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) mma_f8_ss(d, kt + k_off(ks, TL::kHalf), qt + k_off(ks, TQ::kHalf), iqk, ks > 0);
        tc::mma_commit(b_s + 8 * (qi & 1));
        tc::mma_commit(empty(n));
        if (last) tc::mma_commit(b_qempty + 8 * (qk_k & 1));
      }
      __syncwarp();
      ++qi;
      ++qk_t;
      if (last) {
        qk_t = 0;
        ++qk_k;
        qw.next();
      }
      return true;
    };
    ok = qk();
    int i = 0;
    for (Walk w = walk(); ok && w.more(); w.next()) {
      const int tiles = w.tiles(), keys = w.keys();
      for (int t = 0; t < tiles; ++t, ++i) {
        const int n = 2 * i + 1;
        const uint32_t vt = base + (n % C::kStages) * C::kStage;
        if (!(ok = qk())) break;
        if (!(ok = wait(full(n), phase(n)))) break;
        // keys past the request's length hold whatever their page holds, and 0 * NaN is not 0
        const int from = keys - t * kTile;
        if (from < kTile && (from & (kGroup - 1)) != 0) {
          const int rows = kGroup - (from & (kGroup - 1));
          for (int e = lane; e < rows * (D / 16); e += 32)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + TL::chunk_at(from + e / (D / 16), e % (D / 16))), "r"(0) : "memory");
          tc::fence_async_smem();
          __syncwarp();
        }
        if (!(ok = wait(b_p, i & 1))) break;
        tc::fence_after_sync();
        if (lane == 0) {
#pragma unroll
          for (int hf = 0; hf < C::kHalves; ++hf)
#pragma unroll
            for (int ks = 0; ks < kTile / 32; ++ks)
              // (d = 64: rows 64 .. 127 of the product are not used; the leading offset only keeps them in the ring)
              mma_f8_ss(tmem + C::kO + hf * C::kNP, dv + (n % C::kStages) * (C::kStage >> 4) + ((hf * TL::kHalf + ks * 32 * TL::kRow) >> 4),
                        dp + ks * (512 >> 4), ipv, (t > 0) | ks);
          tc::mma_commit(b_pv + 8 * (i & 1));
          tc::mma_commit(empty(n));
        }
        __syncwarp();
      }
    }
  } else if (warp == 6) {
    // ---- queries: rows of Q, high parts then low parts, one unit ahead; rows past 2 HP stay zero
    bool ok = true;
    for (int e = 2 * HP * (D / 16) + lane; e < 2 * C::kNQ * (D / 16); e += 32) {
      const int buffer = e / (C::kNQ * (D / 16)), i = e - buffer * (C::kNQ * (D / 16)), row = i / (D / 16);
      if (row >= 2 * HP)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(s_q + buffer * C::kQ + TQ::chunk_at(row, i % (D / 16))), "r"(0) : "memory");
    }
    int k = 0;
    for (Walk w = walk(); w.more() && ok; w.next(), ++k) {
      const int head0 = first_head(w), heads = unit_heads(w);
      const uint16_t* qp = a.q + static_cast<int64_t>(p.b0 + w.b) * a.q_stride + static_cast<int64_t>(head0) * D;
      ok = __all_sync(0xFFFFFFFFu, wait(b_qempty + 8 * (k & 1), ((k >> 1) & 1) ^ 1));
      if (!ok) break;
      const uint32_t qt = s_q + (k & 1) * C::kQ;
      constexpr int kPer = D / 16;          // 16-element chunks of a head, one to a lane
      constexpr int kAtOnce = 32 / kPer;    // heads at a time
      constexpr int kGroupsOf = (HP + kAtOnce - 1) / kAtOnce, kLoads = kGroupsOf < 4 ? kGroupsOf : 4;  // groups of heads; in flight
#pragma unroll 1
      for (int g0 = 0; g0 < kGroupsOf * kAtOnce; g0 += kLoads * kAtOnce) {
        uint4 all[kLoads][2];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int hd = g0 + i * kAtOnce + lane / kPer, c = lane % kPer;
          all[i][0] = all[i][1] = make_uint4(0, 0, 0, 0);
          if (hd < heads) {
            all[i][0] = *reinterpret_cast<const uint4*>(qp + hd * D + c * 16);
            all[i][1] = *reinterpret_cast<const uint4*>(qp + hd * D + c * 16 + 8);
          }
        }
#pragma unroll 1
        for (int i0 = 0; i0 < kLoads; ++i0) {
          const int hd = g0 + i0 * kAtOnce + lane / kPer, c = lane % kPer;
          const uint4 raw[2] = {all[0][0], all[0][1]};
#pragma unroll
          for (int i = 0; i + 1 < kLoads; ++i) {
            all[i][0] = all[i + 1][0];
            all[i][1] = all[i + 1][1];
          }
          const uint32_t x[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) top = max(top, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
#pragma unroll
          for (int o = 1; o < kPer; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
          const int e = min(max(static_cast<int>(top >> 7), 1), 254);  // 127 + exponent of the largest
          const int down = min(max(127 + 7 - (e - 127), 1), 254);      // * 2^(7 - exponent)
          const float sc = __int_as_float(down << 23);
          const float put = a.scale < 0.0f ? -sc : sc;                 // the factor is kept positive
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float f[4], g[4];
            f[0] = __uint_as_float(x[2 * i] << 16) * put;
            f[1] = __uint_as_float(x[2 * i] & 0xFFFF0000u) * put;
            f[2] = __uint_as_float(x[2 * i + 1] << 16) * put;
            f[3] = __uint_as_float(x[2 * i + 1] & 0xFFFF0000u) * put;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              g[z] = __uint_as_float(__float_as_uint(f[z]) & 0xFFF00000u);  // sign, exponent, 3 bits
              f[z] -= g[z];
            }
            hi[i] = e4m3x4(g[0], g[1], g[2], g[3]);
            lo[i] = e4m3x4(f[0], f[1], f[2], f[3]);
          }
          // row of the operand: high part of head hd, low part HP rows on
          if (hd < HP) {
            const uint32_t at = TQ::chunk_at(hd, c), al = TQ::chunk_at(HP + hd, c);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(qt + at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(qt + al), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
            // a query that is not finite would saturate in 8 bits: its head is NaN through its factor
            if (c == 0)
              s_factor[(k % C::kFactorRing) * 16 + hd] =
                  top < 0x7F80u ? fabsf(a.scale) * kLog2e * __int_as_float((254 - down) << 23) : __int_as_float(0x7FC00000);
          }
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_factor + 8 * (k % C::kFactorRing));
      mbar_arrive(b_qfull + 8 * (k & 1));
    }
  } else {
    // ---- softmax: thread = key of the tile; at a unit's end thread = row of O^T
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t pt = s_p + tid * 16;
    // A warp whose wait runs out (`ok` false) keeps meeting the others at the barriers until the four of them
    // leave together.
    bool ok = true, left = false;
    int i = 0, k = 0;
    for (Walk u = walk(); u.more() && !left; u.next(), ++k) {
      const int tiles = u.tiles(), keys = u.keys();
      float m[HP], l[HP], fac[HP];
      ok = __all_sync(0xFFFFFFFFu, ok && wait(b_factor + 8 * (k % C::kFactorRing), (k / C::kFactorRing) & 1));
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.0f;
        fac[h] = s_factor[(k % C::kFactorRing) * 16 + h];
      }
      for (int t = 0; t < tiles; ++t, ++i) {
        if (i % C::kBatch == 0 || t == 0) ok = ok && wait(b_info + 8 * ((i / C::kBatch) % C::kBatches), (i / C::kInfoRing) & 1);
        ok = __all_sync(0xFFFFFFFFu, ok && wait(b_s + 8 * (i & 1), (i >> 1) & 1));
        float x[HP];
        float2 own = make_float2(-1.0f, 0.0f);
        float e = 0.0f;  // of vs
        bool above = false;
        if (ok) {
          tc::fence_after_sync();
          float s[C::kNQ];
          tmem_load(tmem + C::kNQ * (i & 1) + lanes, s);
          const float2* sc = s_scale + (i % C::kInfoRing) * kGroups;
          own = sc[tid / kGroup];
          e = static_cast<float>(max(((__float_as_int(own.y) >> 23) & 255) - 127, kLeastScale));
          __syncwarp();  // the batch's last tile: its lookups have been read
          if (i % C::kBatch == C::kBatch - 1 && lane == 0) mbar_arrive(b_infoe + 8 * ((i / C::kBatch) % C::kBatches));
          const bool hidden = t * kTile + tid >= keys || own.x < 0.0f;
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            x[h] = hidden ? -INFINITY : (s[h] + s[HP + h]) * (own.x * fac[h]);
            above |= x[h] > m[h] + (kRise - e);
          }
        }
        if (any_of_128(above || !ok)) {
          if (any_of_128(!ok)) {
            left = true;
            break;
          }
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            const float w = warp_max(x[h] + e);
            if (lane == 0) s_red[warp * 16 + h] = w;
          }
          sync_128();
          float corr[HP];
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            const float top = fmaxf(fmaxf(s_red[h], s_red[16 + h]), fmaxf(s_red[32 + h], s_red[48 + h]));
            const float to = top > m[h] + kRise ? top : m[h];  // by the head alone, whatever the others do
            const float root = to == -INFINITY ? 1.0f : ex2_root(m[h] - to);
            m[h] = to;
            l[h] = l[h] * root * root;
            corr[h] = root * root;
          }
          if (t > 0) {
            ok = __all_sync(0xFFFFFFFFu, wait(b_pv + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1));
            if (ok) {
              tc::fence_after_sync();
#pragma unroll 1
              for (int c = 0; c < C::kHalves * C::kNP; c += 16) {
                float o[16];
                const uint32_t at = tmem + C::kO + c + lanes;
                tc::tmem_ld16(at, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= corr[e % HP];
                tc::tmem_st16(at, o);
              }
              tc::tmem_wait_st();
            }
          }
        }
        uint32_t part[4][HP / 2];
#pragma unroll
        for (int h = 0; h < HP; h += 2) {
          float a0 = ex2(m[h] == -INFINITY ? x[h] : x[h] - m[h] + kTop);
          float a1 = ex2(m[h + 1] == -INFINITY ? x[h + 1] : x[h + 1] - m[h + 1] + kTop);
          l[h] += a0;
          l[h + 1] += a1;
          a0 *= own.y;
          a1 *= own.y;
#pragma unroll
          for (int y = 0; y < 4; ++y) part[y][h / 2] = split_off(a0, a1);
        }
        // the tile before has to be done with P (it shares the buffer)
        ok = __all_sync(0xFFFFFFFFu, ok && (i == 0 || wait(b_pv + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1)));
        auto word = [&](int y, int w) { return part[y][2 * w] | (part[y][2 * w + 1] << 16); };
        auto put = [&](int block, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(pt + block * kTile * 16), "r"(w0), "r"(w1), "r"(w2), "r"(w3) : "memory");
        };
        if constexpr (HP == 4) {
          put(0, word(0, 0), word(1, 0), word(2, 0), word(3, 0));
        } else if constexpr (HP == 8) {
          put(0, word(0, 0), word(0, 1), word(1, 0), word(1, 1));
          put(1, word(2, 0), word(2, 1), word(3, 0), word(3, 1));
        } else {
#pragma unroll
          for (int y = 0; y < 4; ++y) put(y, word(y, 0), word(y, 1), word(y, 2), word(y, 3));
        }
        tc::fence_async_smem();
        tc::fence_before_sync();
        mbar_arrive(b_p);
      }
      if (left) break;
      // the unit's sums, then its rows of O^T
#pragma unroll
      for (int h = 0; h < HP; ++h) {
#pragma unroll
        for (int o = 16; o; o >>= 1) l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], o);
        if (lane == 0) s_sum[warp * 16 + h] = l[h];
      }
      if (any_of_128(!ok)) break;
#pragma unroll
      for (int h = 0; h < HP; ++h) l[h] = (s_sum[h] + s_sum[16 + h]) + (s_sum[32 + h] + s_sum[48 + h]);
      ok = __all_sync(0xFFFFFFFFu, wait(b_pv + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1));
      if (!ok) continue;  // to meet the others
      tc::fence_after_sync();
      const int head0 = first_head(u), heads = unit_heads(u);
      const int64_t f = ((static_cast<int64_t>(u.b) * a.H + u.h) * p.chunks + u.chunk) * p.each + u.index;
      const bool alone = u.count == 1;
      uint16_t* op = a.out + (static_cast<int64_t>(p.b0 + u.b) * a.Hq + head0) * D + tid;
      float* pp = p.part + f * p.heads * D + tid;
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        if (!alone && tid == h && h < heads) p.ml[f * p.heads + h] = make_float2(m[h], l[h]);
        // fac: what a head's sums are multiplied with
        fac[h] = !alone ? 1.0f : l[h] > 0.0f || l[h] != l[h] ? __fdividef(1.0f, l[h]) : 0.0f;
      }
#pragma unroll 1
      for (int hf = 0; hf < C::kHalves; ++hf) {
        float o[C::kNP];
        tmem_load(tmem + C::kO + hf * C::kNP + lanes, o);
        if (D >= 128 || tid < D) {
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            const float sum = (o[h] + (o[HP + h] + (o[2 * HP + h] + o[3 * HP + h] * 0.03125f) * 0.03125f) * 0.03125f) * fac[h];
            if (h < heads) {
              if (alone) {
                asm volatile("{.reg .b16 x; cvt.rn.bf16.f32 x, %1; st.global.b16 [%0], x;}" ::"l"(op + h * D + hf * 128), "f"(fac[h] == 0.0f ? 0.0f : sum) : "memory");
              } else {
                pp[h * D + hf * 128] = sum;
              }
            }
          }
        }
        __syncwarp();
      }
      tc::fence_before_sync();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (s_fail) {  // a wait ran out: leave only once what is in flight has landed
    if (tid == 0 && a.err) atomicOr(a.err, GDN_DEVERR_TIMEOUT);
    if (warp == 5)
      for (int i = max(0, copies - C::kStages); i < copies; ++i) mbar_wait_bounded(full(i), phase(i));
    if (warp == 4 && lane == 0) {
      tc::mma_commit(b_drain);
      mbar_wait_bounded(b_drain, 0);
    }
    __syncthreads();
  }
  if (warp == 4) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kColumns);
  }
}

// Joins the units of one request, kv head and head chunk; an empty request gets zeros. A thread has four d
// of one head. Up to kJoinRows units it takes in order; more are taken by kJoinRows threads, unit u by
// u mod kJoinRows, whose sums are then taken in order (for few units that is the same). Either way the order
// goes by the request's own units.
constexpr int kJoinRows = 16;

struct JoinSum {
  float m = -INFINITY, l = 0.0f;
  float4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  // the root of a unit's weight
  __device__ __forceinline__ static float weight(float m, float l, float top) {
    // a unit without keys has m = -inf, l = 0; with only NaN scores m = -inf, l = NaN
    return m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : ex2_root(m - top);
  }
  __device__ __forceinline__ void add(float2 e, const float4& v) {
    const float top = fmaxf(m, e.x), ra = weight(m, l, top), rb = weight(e.x, e.y, top), wa = ra * ra, wb = rb * rb;
    m = top;
    l = l * ra * ra + e.y * rb * rb;
    o.x = o.x * wa + v.x * wb;
    o.y = o.y * wa + v.y * wb;
    o.z = o.z * wa + v.z * wb;
    o.w = o.w * wa + v.w * wb;
  }
  // units u, u + step, ..
  __device__ __forceinline__ void add_units(const float2* ml, const float4* part, int u, int n, int step, int heads, int d4s) {
    constexpr int kAhead = 4;
#pragma unroll 1
    for (; u < n; u += kAhead * step) {
      float2 e[kAhead];
      float4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (u + i * step < n) {
          const int64_t at = static_cast<int64_t>(u + i * step) * heads;
          e[i] = ml[at];
          v[i] = part[at * d4s];
        }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (u + i * step < n) add(e[i], v[i]);
    }
  }
  __device__ __forceinline__ void store(uint16_t* out) const {
    const float inv = l > 0.0f || l != l ? __fdividef(1.0f, l) : 0.0f;
    uint2 st;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.x) : "f"(o.y * inv), "f"(o.x * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.y) : "f"(o.w * inv), "f"(o.z * inv));
    *reinterpret_cast<uint2*>(out) = st;
  }
};

template <int D>
__global__ void __launch_bounds__(256) attn_decode_join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kLanes = D / 4;
  __shared__ float4 s_o[kJoinRows][16];
  __shared__ float2 s_ml[kJoinRows];
  const AttnArgs& a = p.a;
  const int HC = a.H * p.chunks, G = a.Hq / a.H, tid = threadIdx.x;
  const int b = blockIdx.x / HC, hc = blockIdx.x - b * HC, h = hc / p.chunks, chunk = hc - h * p.chunks;
  const int heads = min(p.heads, G - chunk * 16);
  const int n = units_of(min(max(a.lens[p.b0 + b], 0), a.max_blocks * a.bs));
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (by every CTA: this kernel's end stands for the call's)
  if (n == 1 || (n <= kJoinRows && blockIdx.y > 0)) return;
  const int64_t f = static_cast<int64_t>(blockIdx.x) * p.each * p.heads;
  const float2* ml = p.ml + f;
  const float4* part = reinterpret_cast<const float4*>(p.part + f * D);
  uint16_t* out = a.out + (static_cast<int64_t>(p.b0 + b) * a.Hq + h * G + chunk * 16) * D;
  if (n <= kJoinRows) {
#pragma unroll 1
    for (int i = tid; i < heads * kLanes; i += 256) {
      JoinSum sum;
      const int head = i / kLanes;
      sum.add_units(ml + head, part + i, 0, n, 1, p.heads, kLanes);
      sum.store(out + i * 4);
    }
    return;
  }
  const int row = tid / 16, lane = tid % 16;
#pragma unroll 1
  for (int i0 = blockIdx.y * 16; i0 < heads * kLanes; i0 += gridDim.y * 16) {  // 16 lanes of one head
    JoinSum sum;
    const int head = i0 / kLanes;
    sum.add_units(ml + head, part + i0 + lane, row, n, kJoinRows, p.heads, kLanes);
    s_o[row][lane] = sum.o;
    if (lane == 0) s_ml[row] = make_float2(sum.m, sum.l);
    __syncthreads();
    if (row == 0) {
#pragma unroll 1
      for (int i = 1; i < kJoinRows; ++i) sum.add(s_ml[i], s_o[i][lane]);
      sum.store(out + (i0 + lane) * 4);
    }
    __syncthreads();
  }
}

struct DecodeLayout {
  size_t part, total;
};
DecodeLayout decode_layout(int nb, int max_blocks, int Hq, int H, int d, int bs) {
  const int G = Hq / H, heads = G < 16 ? G : 16, chunks = (G + 15) / 16;
  const size_t units = static_cast<size_t>(nb) * H * chunks * most_units(static_cast<int64_t>(max_blocks) * bs);
  DecodeLayout L;
  L.part = (units * heads * 8 + 255) & ~static_cast<size_t>(255);
  L.total = L.part + units * heads * d * 4;
  return L;
}

template <int D, int HP>
cudaError_t launch_decode_d(DecodeParams& p, const CacheMaps& maps, cudaStream_t s) {
  using C = DecodeCfg<D, HP>;
  auto kern = attn_decode_kernel<D, HP>;
  const int smem = C::smem_of(p.nb);
  // the same for every call: the limit is the kernel's, whichever thread sets it last
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem_of(kBatchPerLaunch));
  if (e != cudaSuccess) return e;
  // CTAs of an SM by its shared memory, registers and tensor memory (the occupancy query answers 1 for
  // kernels that allocate tensor memory)
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  int per_sm = kSmemPerSm / (smem + static_cast<int>(fa.sharedSizeBytes) + 1024);
  const int by_regs = 65536 / (((fa.numRegs + 7) & ~7) * kThreads), by_tmem = 512 / C::kColumns;
  if (per_sm > by_regs) per_sm = by_regs;
  if (per_sm > by_tmem) per_sm = by_tmem;
  if (per_sm < 1) per_sm = 1;
  const int64_t most = static_cast<int64_t>(p.nb) * p.a.H * p.chunks * p.each;
  const int grid = static_cast<int>(most < static_cast<int64_t>(per_sm) * sm_count() ? most : per_sm * sm_count());
  kern<<<grid, kThreads, smem, s>>>(p, maps);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // where requests may have many units, CTAs enough for all their heads and d
  cfg.gridDim = dim3(p.nb * p.a.H * p.chunks, p.each > kJoinRows ? p.heads * D / 64 : 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_join_kernel<D>, p);
}

template <int D>
cudaError_t launch_decode_h(DecodeParams& p, const CacheMaps& maps, cudaStream_t s) {
  return p.heads <= 4   ? launch_decode_d<D, 4>(p, maps, s)
         : p.heads <= 8 ? launch_decode_d<D, 8>(p, maps, s)
                        : launch_decode_d<D, 16>(p, maps, s);
}

}  // namespace

int attn_decode_batch(int max_blocks, int Hq, int H, int bs) {
  // shares of a launch are counted in 32 bits, in tiles of all its requests, kv heads and head chunks (requests may have pages
  // in common, so the cache's size is no bound)
  const int64_t each = (static_cast<int64_t>(max_blocks) * bs + kTile - 1) / kTile * H * ((Hq / H + 15) / 16);
  const int64_t most = 0x7fffffffLL / each;
  return static_cast<int>(most < kBatchPerLaunch ? most : kBatchPerLaunch);
}

size_t attn_decode_workspace(int B, int max_blocks, int Hq, int H, int d, int bs) {
  const int most = attn_decode_batch(max_blocks, Hq, H, bs);
  return decode_layout(B < most ? B : most, max_blocks, Hq, H, d, bs).total;
}

cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t s) {
  CacheMaps maps;
  cudaError_t e = encode_cache_maps(&maps, a);
  if (e != cudaSuccess) return e;
  const int G = a.Hq / a.H;
  DecodeParams p;
  p.a = a;
  p.fault = attention_test_fault().load(std::memory_order_relaxed);
  p.heads = G < 16 ? G : 16;
  p.chunks = (G + 15) / 16;
  p.each = static_cast<int>(most_units(static_cast<int64_t>(a.max_blocks) * a.bs));
  const int most = attn_decode_batch(a.max_blocks, a.Hq, a.H, a.bs);  // (not 0: the caller has checked)
  const int launches = (a.B + most - 1) / most, per = (a.B + launches - 1) / launches;
  for (int b0 = 0; b0 < a.B; b0 += per) {
    p.b0 = b0;
    p.nb = a.B - b0 < per ? a.B - b0 : per;
    const DecodeLayout L = decode_layout(p.nb, a.max_blocks, a.Hq, a.H, a.d, a.bs);
    char* ws = static_cast<char*>(a.workspace);
    p.ml = reinterpret_cast<float2*>(ws);
    p.part = reinterpret_cast<float*>(ws + L.part);
    e = a.d == 64    ? launch_decode_h<64>(p, maps, s)
        : a.d == 128 ? launch_decode_h<128>(p, maps, s)
                     : launch_decode_h<256>(p, maps, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace gdn
