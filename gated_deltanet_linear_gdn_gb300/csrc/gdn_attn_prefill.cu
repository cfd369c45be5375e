// gdn_attn_prefill.cu -- attention of prompt tokens over the 8-bit paged cache, on the
// tcgen05 tensor cores.
//
// Request b has n new tokens (rows cu[b] .. cu[b+1] of q) whose keys and values are already in
// the cache as its last n of len; token i sees keys 0 .. len - n + i. Per (request, kv head) the
// rows of the product are the pairs (token, query head of the group), token-major, so a 128-row
// tile uses each key tile for all G heads.
//
// S = Q K^T runs on 8-bit operands straight from the pages. A query is split into two e4m3 parts,
//   q = q_hi + q_lo (a row scaled by a power of two so that max |q| lies in [128, 256)),
// multiplied in two MMAs into the same fp32 accumulator: q is a bf16 value (8 significant bits), so the split is
// exact down to 2^-18 of the row's largest element. Two 8-bit MMAs cost what one 16-bit MMA costs, so the
// bound is the dense bf16 rate. P V differs by head_dim, see the two kernels below; p overwrites the scores it
// came from in tensor memory and is the A operand of the second product there.
//
// Scales. A block of keys has one ks: it enters the exponent, and its vs as a power, too: with x = s * ks * factor and
// y = x + log2(vs), p = exp2(y - m) goes into the product with V's bytes, and the row sum takes vs back by group of 16,
// l = sum p / vs. m is the running maximum of y over the keys that the row sees: what a key is rounded to goes by the
// largest probability x scale of the row itself, not by a scale that weighs nothing or that it does not see (a
// reference of its own for vs, the largest of a tile, lost rows whole next to one). m moves only when a y passes it by a power
// of two that the type of p has room for; the accumulator is rescaled only then.
//
// One CTA per unit of 128 rows: its queries stay in shared memory, its output in tensor memory. Loops over
// the columns of a tile are kept rolled: a CTA fetches every role's code, and unrolled loops waited for instructions
// (rolling the softmax's from 128 to 32 columns: 470 -> 368 us for 300 tokens at 60,000, head_dim 128).
//
// A plan kernel turns the lengths into a list of units, the longest first. A request with few
// rows over a long cache is also cut along the keys, by a rule on its own sizes alone
// (kv_splits), and a third kernel joins the fp32 partial sums in order: results do not depend on
// the rest of the batch.
#include <type_traits>

#include "gdn_attn.cuh"
#include "gdn_cache4.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBatchPerLaunch = 2048;
constexpr int kBuckets = 256;
constexpr int kManyUnits = 1 << 30;
// key splits: a request with fewer than few_units(d) row tiles x heads gets up to three times as many (head_dim 256:
// half, as its partial sums are twice as large)
constexpr int kUnitRows = 128;  // (token, head) rows of a unit
constexpr int kMaxSplits = 32, kMinSplitTiles = 8;
__host__ __device__ __forceinline__ constexpr int few_units(int d) { return d == 256 ? 76 : 152; }

struct __align__(16) PrefillUnit {
  int b, h, row0, tile0, tile1, slot;  // slot: partial sums' place, or -1: the unit is the whole
  int splits, first, n, len, pad0, pad1;  // the request's first row of q, its tokens, its cached length
};

struct PrefillParams {
  AttnArgs a;
  int b0, nb;
  int max_units, max_slots;
  int fault;                // test hook: CTA 0 looks up one batch of tiles and no more
  int beside;               // the plan's dependent may start at once
  int32_t* counts;          // [0] units, [1] split tiles, [2] units taken after the grid's first
  PrefillUnit* units;       // [max_units]
  PrefillUnit* joins;       // [max_units]: the first split of each split row tile
  float2* ml;               // [max_slots][rows] (maximum, sum)
  float* part;              // [max_slots][rows][d]
};

// How many pieces the key tiles of a request are cut into: the fewest rounds of an assumed 152
// CTAs, counted in tiles with a constant cost per piece (a prologue and an epilogue take about 8 tiles). 300 tokens at
// 60,000 (80 units of 470 tiles): 371 us in 5 pieces, 677 whole; 8 ragged prompts, none of them alone on the GPU: 322
// and 321. (152 is the SMs of the GPU that the library is built for, as a constant: results stay the same on any.)
// Pieces of unequal length that fill 152 CTAs evenly (cuts at multiples of one length over all row tiles, end to end)
// took 481: row tiles no longer read the same keys at the same time.
__host__ __device__ __forceinline__ int kv_splits(int units, int tiles, int d) {
  if (units >= few_units(d) || tiles < 2 * kMinSplitTiles) return 1;
  int best = 1, cost = 0x7fffffff;
#pragma unroll 1
  for (int s = 1; s <= kMaxSplits && s * kMinSplitTiles <= tiles && s * units <= 3 * few_units(d); ++s) {
    const int c = ((units * s + 151) / 152) * ((tiles + s - 1) / s + 8);
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

__device__ __forceinline__ void request(const PrefillParams& p, int b, int& first, int& n, int& len) {
  const int cap = p.a.max_blocks * p.a.bs;
  first = p.a.cu_tokens[p.b0 + b];
  n = p.a.cu_tokens[p.b0 + b + 1] - first;
  len = min(max(p.a.lens[p.b0 + b], 0), cap);
  if (first < 0 || n < 0 || first + static_cast<int64_t>(n) > p.a.T) n = 0;
}
// Row tiles of a request; its rows are fewer than 2^31.
__device__ __forceinline__ int row_tiles(int n, int G) { return static_cast<int>((static_cast<uint32_t>(n) * G + kUnitRows - 1) / kUnitRows); }
// Key tiles that rows row0 .. row0 + rows - 1 of a request see.
__device__ __forceinline__ int tiles_of(int row0, int rows, int n, int len, int G) {
  const int last = min((row0 + rows - 1) / G, n - 1);  // the unit's last token
  const int seen = min(len, len - n + last + 1);
  return seen > 0 ? (seen + kTile - 1) / kTile : 0;
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ PrefillParams p) {
  __shared__ int32_t s_first[kBatchPerLaunch + 1];  // units before each request
  __shared__ int32_t s_slot[kBatchPerLaunch];       // partial slots before each request
  __shared__ int32_t s_count[kBuckets], s_warp[2][32];
  __shared__ int32_t s_joins;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const AttnArgs& a = p.a;
  if (p.beside) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int G = a.Hq / a.H;
  int flags = 0, carry = 0, carry_slot = 0;
  if (tid < kBuckets) s_count[tid] = 0;
  if (tid == 0) s_joins = 0;
#pragma unroll 1
  for (int base = 0; base < p.nb; base += kPlanThreads) {
    const int b = base + tid;
    int units = 0, slots = 0;
    if (b < p.nb) {
      int first, n, len;
      request(p, b, first, n, len);
      if (n != a.cu_tokens[p.b0 + b + 1] - a.cu_tokens[p.b0 + b] || len != a.lens[p.b0 + b]) flags = GDN_DEVERR_SEQLENS;
      const int qt = row_tiles(n, G) * a.H;
      const int s = kv_splits(qt, (len + kTile - 1) / kTile, a.d);
      units = qt * s;
      slots = s > 1 ? units : 0;
    }
    int v = units, w = slots;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, v, o), y = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) {
        v += x;
        w += y;
      }
    }
    if (lane == 31) {
      s_warp[0][warp] = v;
      s_warp[1][warp] = w;
    }
    __syncthreads();
    // Ranges of cu_tokens that lie over one another may add up to more than 32 bits hold: the sum stops at kManyUnits, which no
    // list has room for (a warp's requests have at most 32 * (2^24 + 2^10) units)
    int bv = carry, bw = carry_slot;
#pragma unroll 4
    for (int i = 0; i < kPlanThreads / 32; ++i) {
      if (i < warp) {
        bv = min(bv + s_warp[0][i], kManyUnits);
        bw += s_warp[1][i];
      }
      carry = min(carry + s_warp[0][i], kManyUnits);
      carry_slot += s_warp[1][i];
    }
    if (b < p.nb) {
      s_first[b + 1] = bv + v;
      s_slot[b] = bw + w - slots;
    }
    __syncthreads();
  }
  if (tid == 0) s_first[0] = 0;
  if (carry > p.max_units || carry_slot > p.max_slots) {  // cu_tokens is not what the caller said
    flags |= GDN_DEVERR_SEQLENS;
    carry = 0;
  }
  if (flags && a.err) atomicOr(a.err, flags);
  __syncthreads();
  // unit u of the list before it is ordered
  auto describe = [&](int u) {
    int lo = 0, hi = p.nb - 1;
#pragma unroll 1
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_first[mid] <= u) lo = mid; else hi = mid - 1;
    }
    int first, n, len;
    request(p, lo, first, n, len);
    PrefillUnit d;
    d.b = lo;
    const int qt = row_tiles(n, G);
    const int s = (s_first[lo + 1] - s_first[lo]) / (qt * a.H);
    const int rem = u - s_first[lo];
    const int piece = rem % s, tile = rem / s;
    d.h = tile % a.H;
    d.row0 = (tile / a.H) * kUnitRows;
    const int tiles = tiles_of(d.row0, kUnitRows, n, len, G);
    const int each = (tiles + s - 1) / s;
    d.tile0 = min(piece * each, tiles);
    d.tile1 = min(d.tile0 + each, tiles);
    d.slot = s > 1 ? s_slot[lo] + rem : -1;
    d.splits = s;
    d.first = first;
    d.n = n;
    d.len = len;
    d.pad0 = d.pad1 = 0;
    return d;
  };
  // counts, then places (a loop, so that the code is fetched once)
#pragma unroll 1
  for (int place = 0; place < 2; ++place) {
#pragma unroll 1
    for (int u = tid; u < carry; u += kPlanThreads) {
      const PrefillUnit d = describe(u);
      // (the order within a bucket is free: it decides when a unit runs, not what it computes)
      const int at = atomicAdd(&s_count[kBuckets - 1 - min(d.tile1 - d.tile0, kBuckets - 1)], 1);
      if (place) {
        p.units[at] = d;
        if (d.splits > 1 && (d.slot - s_slot[d.b]) % d.splits == 0) p.joins[atomicAdd(&s_joins, 1)] = d;
      }
    }
    __syncthreads();
    if (warp == 0 && !place) {  // bucket counts to first places
      int before = 0;
#pragma unroll 1
      for (int i = lane; i < kBuckets; i += 32) {
        const int own = s_count[i];
        int v = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
          if (lane >= o) v += x;
        }
        s_count[i] = before + v - own;
        before += __shfl_sync(0xFFFFFFFFu, v, 31);
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    p.counts[0] = carry;
    p.counts[1] = s_joins;
    p.counts[2] = 0;
  }
}

// ---- what the two kernels share

// Looks up the pages and scales of a unit's tiles, four at a time: lane = (tile of the batch, 16-key group). Of a
// group: ks, log2 vs, 1 / vs (0 for a vs far below the usual ones), and whether its tile has one of those.
template <typename C>
__device__ __forceinline__ void look_up(const PrefillParams& p, const PrefillUnit& u, int tiles, float4* scales, int32_t* s_row,
                                        uint32_t b_info, uint32_t b_infoe, volatile int* fail) {
  const AttnArgs& a = p.a;
  const int lane = threadIdx.x & 31, shift = 31 - __clz(a.bs);
  bool ok = true;
#pragma unroll 1
  for (int j0 = 0; j0 < tiles && ok; j0 += C::kBatch) {
    if (p.fault && blockIdx.x == 0 && j0 > 0) break;
    const int j = j0 + lane / kGroups, pos = (u.tile0 + j) * kTile + (lane % kGroups) * kGroup;
    int row = a.num_blocks * a.H * a.bs;                      // past the cache: zeros
    float4 sc = make_float4(0.0f, -INFINITY, 0.0f, 0.0f);     // no key, or a page that is none: not seen
    if (j < tiles && pos < u.len) {
      const int page = a.block_table[static_cast<int64_t>(p.b0 + u.b) * a.max_blocks + (pos >> shift)];
      if (page >= 0 && page < a.num_blocks) {
        const int64_t at = static_cast<int64_t>(page) * a.H + u.h;
        sc.x = a.k_scale[at];
        sc.y = a.v_scale[at];
        row = (static_cast<int>(at) << shift) + (pos & (a.bs - 1));
        // (finite in any case: a hidden score is -infinity and has to stay that)
        asm("lg2.approx.f32 %0, %0;" : "+f"(sc.y));
        sc.y = fminf(fmaxf(sc.y, kLeastScale), 127.0f);
        sc.z = sc.y < kFarScale ? 0.0f : ex2(-sc.y);
      } else if (a.err) {
        atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);
      }
    }
    const uint32_t far = __ballot_sync(0xFFFFFFFFu, sc.z == 0.0f && sc.y != -INFINITY);
    sc.w = ((far >> (lane & -kGroups)) & ((1u << kGroups) - 1)) != 0 ? 1.0f : 0.0f;
    const int slot = (j0 / C::kBatch) % C::kBatches;
    ok = __all_sync(0xFFFFFFFFu, wait_or_fail(b_infoe + 8 * slot, ((j0 / C::kInfoRing) & 1) ^ 1, fail));
    if (!ok) break;
    s_row[slot * 32 + lane] = row;
    scales[slot * 32 + lane] = sc;
    __syncwarp();
    if (lane == 0) mbar_arrive(b_info + 8 * slot);
  }
}

// What the keys of blocks with a far vs, among 32 scores of two groups, add to a row's sum. All but never called.
__device__ __forceinline__ float far_sum(const float (&s)[32], const float4* scales, float factor, float base) {
  float sum = 0.0f;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float4 e = scales[g];
    if (e.z != 0.0f || e.y == -INFINITY) continue;
    const float ks = exponent_scale(e.x, factor);
#pragma unroll
    for (int i = 0; i < kGroup; ++i) sum += ex2(fmaf(s[g * kGroup + i], ks, base));
  }
  return sum;
}

// Copies the key or the value tiles of a unit into a ring of kStages: lane g < 8 has the 16-key group g of each
// tile. `release`: the lookup ring's barriers that this warp answers for, or 0. Returns the copies started.
template <int D, typename C, int kStages>
__device__ __forceinline__ int copy_tiles(const AttnArgs& a, const PrefillUnit& u, int tiles, const CUtensorMap* by_page,
                                          const CUtensorMap* by_group, uint32_t to, const int32_t* s_row, uint32_t b_full,
                                          uint32_t b_empty, uint32_t b_info, uint32_t release, volatile int* fail) {
  using TL = Tile<D>;
  const int lane = threadIdx.x & 31;
  const bool head = ((lane * kGroup) & (a.bs - 1)) == 0;  // the group starts a page
  bool ok = true;
  int copies = 0;
#pragma unroll 1
  for (int j = 0; j < tiles; ++j) {
    const int st = j % kStages, slot = (j / C::kBatch) % C::kBatches;
    if (j % C::kBatch == 0) ok = wait_or_fail(b_info + 8 * slot, (j / C::kInfoRing) & 1, fail);
    ok = __all_sync(0xFFFFFFFFu, ok && wait_or_fail(b_empty + 8 * st, ((j / kStages) & 1) ^ 1, fail));
    if (!ok) break;
    const int row = s_row[(j % C::kInfoRing) * kGroups + lane % kGroups];
    __syncwarp();
    if (release && j % C::kBatch == C::kBatch - 1 && lane == 0) mbar_arrive(release + 8 * slot);
    // a page of which every token is the request's goes in one box
    const bool whole = ((lane * kGroup) & -a.bs) + a.bs <= u.len - (u.tile0 + j) * kTile;
    if (lane == 0) mbar_arrive_expect_tx(b_full + 8 * st, TL::kBytes);
    __syncwarp();
    if (lane < kGroups && (head || !whole))
#pragma unroll
      for (int x = 0; x < D; x += 128)
        tma_rows(to + st * TL::kBytes + (x / 128) * TL::kHalf + lane * kGroup * TL::kRow, whole ? by_page : by_group, x, row, b_full + 8 * st);
    copies = j + 1;
  }
  return copies;
}

// 0 * NaN is not 0: a NaN in V would reach the rows of the tile that do not see its key. So in a tile that some row sees
// only in part, the keys that not every row sees (from `all_see` on) get zeros for their NaN, and s_nan[0 .. D) has the first key
// with one in each column, for the rows that do see it (s_nan[D]: whether there is any). One tile or two of a unit. Not
// inlined: in the loop of the converting warps it took 4% of the time (300 tokens at 60,000), so 1%.
template <int D, int kThreads>
__device__ __noinline__ void clear_nan(uint32_t tile, int key0, int len, int all_see, int me, int32_t* s_nan) {
  constexpr int kChunks = D / 16;  // of a key
#pragma unroll 1
  for (int i = me; i < kTile * kChunks; i += kThreads) {
    const int key = i / (8 * kChunks) * 8 + i % 8, c = i / 8 % kChunks;
    if (key0 + key < all_see || key0 + key >= len) continue;
    const uint32_t at = tile + Tile<D>::chunk_at(key, c);
    uint32_t x[4], any = 0;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
#pragma unroll
    for (int e = 0; e < 4; ++e) any |= ((x[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // (NaN: all seven bits)
    if (any == 0) continue;
#pragma unroll 1
    for (int e = 0; e < 16; ++e) {
      uint32_t byte;
      asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte) : "r"(at + e));
      if ((byte & 0x7F) != 0x7F) continue;
      asm volatile("st.shared.u8 [%0], %1;" ::"r"(at + e), "r"(0) : "memory");
      atomicMin(s_nan + c * 16 + e, key0 + key);
      s_nan[D] = 1;
    }
  }
}
// The keys that every row of a unit sees: what its first token sees.
__device__ __forceinline__ int seen_by_all(const PrefillUnit& u, int G) { return min(max(u.len - u.n + u.row0 / G + 1, 0), u.len); }
// The unit's first tile that some row sees only in part.
__device__ __forceinline__ int first_partial(const PrefillUnit& u, int G) {
  const int seen = seen_by_all(u, G);
  return seen < u.len ? seen / kTile - u.tile0 : 0x7FFFFFFF;
}

// Queries of a unit's rows: a warp takes kRows / kWarps rows, a lane 8 elements of one; each row is scaled to
// [128, 256) by a power of two and split into two e4m3 parts.
template <int D, int kRows, int kWarps>
__device__ __forceinline__ void split_queries(const AttnArgs& a, const PrefillUnit& u, int G, int rows_all, uint32_t s_q, float* s_factor) {
  using TL = Tile<D>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = u.first;
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;  // lanes of a row, rows at a time
  const float sign = a.scale < 0.0f ? -1.0f : 1.0f;     // the factor is kept positive
  constexpr int kPer = kRows / kWarps;         // rows of a warp
  constexpr int kLoads = kPer / kAtOnce < 4 ? kPer / kAtOnce : 4;  // in flight
#pragma unroll 1
  for (int i0 = 0; i0 < kPer / kAtOnce; i0 += kLoads) {
    uint4 raw[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int rr = warp * kPer + (i0 + i) * kAtOnce + lane / kLanes;  // row of the unit
      const int row = u.row0 + rr, token = row / G;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (row < rows_all)
        raw[i] = *reinterpret_cast<const uint4*>(a.q + (first + token) * a.q_stride +
                                                 (u.h * G + row - token * G) * D + (lane % kLanes) * 8);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int rr = warp * kPer + (i0 + i) * kAtOnce + lane / kLanes;
      const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t top = 0;
#pragma unroll
      for (int y = 0; y < 4; ++y) top = max(top, max(x[y] & 0x7FFFu, (x[y] >> 16) & 0x7FFFu));
      if constexpr (kLanes == 32) {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
      } else {
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      }
      const int e = min(max(static_cast<int>(top >> 7), 1), 254);       // 127 + exponent of the largest
      const int down = min(max(127 + 7 - (e - 127), 1), 253);           // * 2^(7 - exponent), whose inverse is a normal number
      const float sc = __int_as_float(down << 23), put = sc * sign;
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float f[4], g[4];
        f[0] = __uint_as_float(x[2 * y] << 16) * put;
        f[1] = __uint_as_float(x[2 * y] & 0xFFFF0000u) * put;
        f[2] = __uint_as_float(x[2 * y + 1] << 16) * put;
        f[3] = __uint_as_float(x[2 * y + 1] & 0xFFFF0000u) * put;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          g[z] = __uint_as_float(__float_as_uint(f[z]) & 0xFFF00000u);  // sign, exponent, 3 bits
          f[z] -= g[z];
        }
        hi[y] = e4m3x4(g[0], g[1], g[2], g[3]);
        lo[y] = e4m3x4(f[0], f[1], f[2], f[3]);
      }
      {
        const int c = lane % kLanes;
        const uint32_t at = s_q + TL::chunk_at(rr, c >> 1) + (c & 1) * 8;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(hi[0]), "r"(hi[1]) : "memory");
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + TL::kBytes), "r"(lo[0]), "r"(lo[1]) : "memory");
        // a query that is not finite saturates in 8 bits: its row is NaN through its sum
        if (c == 0) s_factor[rr] = top < 0x7F80u ? fabsf(a.scale) * kLog2e * __int_as_float((254 - down) << 23) : __int_as_float(0x7FC00000);
      }
    }
  }
}

// Writes kWide columns from c0 of a unit's rows, thread = row: the result, or the partial sums of a unit that is
// one of several. Through shared memory that the row tile's queries had (kBytes a warp), some columns at a
// time, so that a warp writes rows piece by piece and not 32 rows at once; 16-byte chunk c of row i at
// c ^ (i mod chunks).
template <int D, int kWide, int kBytes>
__device__ __forceinline__ void store_rows(const PrefillParams& p, const PrefillUnit& u, int rows, int r, bool live, int token, int head,
                                           int G, int tiles, float l, uint32_t taddr, int c0, uint32_t stage, const int32_t* s_nan) {
  const AttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const bool whole = u.slot < 0;
  const float inv = l > 0.0f || l != l ? __fdividef(1.0f, l) : 0.0f;
  const float mul = whole ? inv : 1.0f;
  const bool none = tiles == 0 || (whole && inv == 0.0f);  // zeros, whatever tensor memory holds
  constexpr int kFit = kBytes / 128;                       // fp32 columns of 32 rows that fit
  constexpr int kCols = kFit < kWide ? kFit : kWide;
  constexpr int kLoad = kCols < 32 ? 16 : 32;
  // where the lane's row goes, in elements
  const int64_t mine = whole ? (static_cast<int64_t>(u.first + token) * a.Hq + u.h * G + head) * D
                             : (static_cast<int64_t>(u.slot) * rows + r) * D;
#pragma unroll 1
  for (int c = c0; c < c0 + kWide; c += kCols) {
#pragma unroll 1
    for (int x = 0; x < kCols; x += kLoad) {
      float o[kLoad];
      if (tiles > 0) {
        if constexpr (kLoad == 32) tmem_ld32(taddr + c + x, o);
        else tc::tmem_ld16(taddr + c + x, o);
        tc::tmem_wait_ld();
      }
#pragma unroll
      for (int i = 0; i < kLoad; ++i) o[i] = none ? 0.0f : o[i] * mul;
      if (s_nan[D] != 0) {  // see clear_nan
        const int sees = live ? min(u.len, u.len - u.n + token + 1) : 0;
#pragma unroll
        for (int i = 0; i < kLoad; ++i)
          if (s_nan[c + x + i] < sees) o[i] = __int_as_float(0x7FC00000);
      }
      if (whole) {
#pragma unroll
        for (int i = 0; i < kLoad; i += 8) {
          uint32_t w[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[y]) : "f"(o[i + 2 * y + 1]), "f"(o[i + 2 * y]));
          const int chunk = ((x + i) / 8) ^ (lane % (kCols / 8));
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * (kCols * 2) + chunk * 16), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
        }
      } else {
#pragma unroll
        for (int i = 0; i < kLoad; i += 4) {
          const int chunk = ((x + i) / 4) ^ (lane % (kCols / 4));
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * (kCols * 4) + chunk * 16), "f"(o[i]), "f"(o[i + 1]), "f"(o[i + 2]), "f"(o[i + 3]) : "memory");
        }
      }
    }
    __syncwarp();
    auto drain = [&](auto per_tag) {
      constexpr int per = decltype(per_tag)::value;  // chunks of a row
#pragma unroll 4
      for (int e = 0; e < per; ++e) {
        const int i = (e * 32 + lane) / per, chunk = lane % per;
        const int64_t at = __shfl_sync(0xFFFFFFFFu, mine, i);
        const bool there = __shfl_sync(0xFFFFFFFFu, static_cast<int>(live), i);
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(stage + i * per * 16 + ((chunk ^ (i % per)) << 4)));
        if (there) {
          if (per == kCols / 8) *reinterpret_cast<uint4*>(a.out + at + c + chunk * 8) = v;
          else *reinterpret_cast<uint4*>(p.part + at + c + chunk * 4) = v;
        }
      }
    };
    if (whole) drain(std::integral_constant<int, kCols / 8>{});
    else drain(std::integral_constant<int, kCols / 4>{});
    __syncwarp();
  }
}

// ------------------------------------------------------------------------------- head_dim 256
//
// Both products on 8-bit operands, no conversion of V: p, rounded to f16, is the sum of three e5m2 values
// (split_e5m2), each of what the ones before leave: 11 significant bits. e5m2 has f16's exponents, so all three have the
// factor 1 and one accumulator, down to 2^-17: m stands for 2^11 and moves when a y passes it by 2^4, so a key is
// rounded to 2^-28 of the row's largest whatever stands between. (Two e4m3 parts, a fifth fewer products and 123 us where
// this took 138, end at 2^-14 of it: 5,000 keys 10 nats below one of no value came out 14 to 26% small.)
//
// Sixteen softmax warps, four threads a row with 32 columns each (they exchange their maxima), two score buffers (2 x
// 128 columns of tensor memory, 256 of output), a warp that issues MMAs: 2,610 cycles of products a tile. 4,096 tokens
// (16 / 2 heads): 142 us, 51% of the bf16 rate with the masked half of the diagonal counted out; without the third part's
// product 129, without the arithmetic of the split 130. With f16 probabilities, as below, V alone would take 128 KB of
// shared memory.
struct WideCfg {
  static constexpr int D = 256;
  static constexpr int kSplitC = 4;                      // softmax warpgroups that share the rows, by columns
  static constexpr int kRows = kUnitRows;
  static constexpr int kSoftWarps = 4 * kSplitC;
  static constexpr int kThreads = 32 * (kSoftWarps + 4); // and warps for MMAs, lookups, copies of K, copies of V
  static constexpr int kStages = 2;                      // key tiles in the ring, and value tiles
  static constexpr int kBatch = 4, kBatches = 4, kInfoRing = kBatch * kBatches;  // tiles looked up at a time; kept
  static constexpr int kQ = 2 * Tile<D>::kBytes;         // hi and lo
  static constexpr int kKV = kStages * 2 * Tile<D>::kBytes;
  static constexpr int kAtScale = kQ + kKV;                 // [kInfoRing][kGroups] (ks, log2 vs, 1 / vs)
  static constexpr int kAtRow = kAtScale + kInfoRing * kGroups * 16;
  static constexpr int kAtMax = kAtRow + kInfoRing * kGroups * 4;  // [2][kSplitC][kRows]
  static constexpr int kAtFactor = kAtMax + 2 * kSplitC * kRows * 4;  // [kRows]
  static constexpr int kAtNan = kAtFactor + kRows * 4;   // [D + 1], see clear_nan
  static constexpr int kAtBars = kAtNan + (D + 2) * 4;
  static constexpr int kSmem = 1024 + kAtBars + 8 * (4 * kStages + 2 * kBatches + 8);
  // tensor memory columns
  static constexpr int kS = 0;         // two score buffers of 128
  static constexpr int kO = 256;       // output, D columns
};

__global__ void __launch_bounds__(WideCfg::kThreads, 1)
    attn_prefill_wide_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CacheMaps maps) {
  using C = WideCfg;
  constexpr int D = C::D;
  using TL = Tile<D>;
  constexpr int NC = kTile / C::kSplitC;  // columns (keys) of a softmax thread
  constexpr int NG = NC / kGroup;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + (-smem_addr(smem_raw) & 1023u);
  const uint32_t s_q = smem_addr(smem), s_k = s_q + C::kQ, s_v = s_k + C::kStages * TL::kBytes;
  float4* s_scale = reinterpret_cast<float4*>(smem + C::kAtScale);
  int32_t* s_row = reinterpret_cast<int32_t*>(smem + C::kAtRow);
  float* s_max = reinterpret_cast<float*>(smem + C::kAtMax);
  float* s_factor = reinterpret_cast<float*>(smem + C::kAtFactor);
  int32_t* s_nan = reinterpret_cast<int32_t*>(smem + C::kAtNan);
  const uint32_t bar = s_q + C::kAtBars;
  const uint32_t b_kfull = bar, b_kempty = bar + 8 * C::kStages, b_vfull = bar + 16 * C::kStages,
                 b_vempty = bar + 24 * C::kStages, b_info = bar + 32 * C::kStages, b_infoe = b_info + 8 * C::kBatches,
                 b_s = b_infoe + 8 * C::kBatches, b_p = b_s + 16, b_pv = b_p + 16, b_q = b_pv + 16, b_drain = b_q + 8;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_fail;

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // (known to be the same in a warp)
  const AttnArgs& a = p.a;
  if (tid < 4) prefetch_map(tid == 0 ? &maps.k_page : tid == 1 ? &maps.v_page : tid == 2 ? &maps.k_group : &maps.v_group);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (static_cast<int>(blockIdx.x) >= *reinterpret_cast<volatile int32_t*>(p.counts)) return;
  const PrefillUnit u = p.units[blockIdx.x];
  const int n = u.n, len = u.len;
  const int G = a.Hq / a.H;
  const int rows_all = n * G;  // (below 2^31: the caller's tokens x heads are)
  const int tiles = u.tile1 - u.tile0;

  if (tid <= D) s_nan[tid] = tid < D ? 0x7FFFFFFF : 0;
  if (tid == 0) {
    for (int i = 0; i < 4 * C::kStages + C::kBatches; ++i) mbar_init(bar + 8 * i, 1);
    for (int i = 0; i < C::kBatches; ++i) mbar_init(b_infoe + 8 * i, C::kSoftWarps + 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_s + 8 * i, 1);
      mbar_init(b_p + 8 * i, 32 * C::kSoftWarps);
      mbar_init(b_pv + 8 * i, 1);
    }
    mbar_init(b_q, 32 * C::kSoftWarps);
    mbar_init(b_drain, 1);
    s_fail = 0;
  }
  fence_mbar_init();
  if (warp == C::kSoftWarps) {
    tc::tmem_alloc(&s_tmem, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;

  auto wait = [&](uint32_t b, int parity) { return wait_or_fail(b, parity, &s_fail); };
  auto use = [](int j) { return (j >> 1) & 1; };  // of score buffer j & 1, its barriers' parity

  int copies = 0;  // of a copying warp
  if (warp == C::kSoftWarps + 1) {
    look_up<C>(p, u, tiles, s_scale, s_row, b_info, b_infoe, &s_fail);
  } else if (warp >= C::kSoftWarps + 2) {
    const bool is_v = warp == C::kSoftWarps + 3;
    copies = is_v ? copy_tiles<D, C, C::kStages>(a, u, tiles, &maps.v_page, &maps.v_group, s_v, s_row, b_vfull, b_vempty, b_info, b_infoe, &s_fail)
                  : copy_tiles<D, C, C::kStages>(a, u, tiles, &maps.k_page, &maps.k_group, s_k, s_row, b_kfull, b_kempty, b_info, 0, &s_fail);
  } else if (warp == C::kSoftWarps) {
    // ---- MMAs
    constexpr uint32_t iqk = idesc_f8(128, kTile, false, false), ipv = idesc_f8(128, D, false, true) | kIdescE5m2A;
    bool ok = tiles == 0 || wait(b_q, 0);
    tc::fence_after_sync();
    // descriptors but for their start address (bits 0 .. 13, in 16 bytes), which each MMA adds: the issuing
    // warp shares its scheduler with softmax warps, and a few instructions an MMA are what it gets
    const uint64_t dk = TL::desc(s_k, 16), dq = TL::desc(s_q, 16), dv = TL::desc(s_v, TL::kHalf);
    auto k_off = [](int ks) { return static_cast<uint64_t>((ks / (TL::kRow / 32)) * TL::kHalf + (ks % (TL::kRow / 32)) * 32) >> 4; };
    auto qk = [&](int j) {  // scores of key tile j
      if (lane == 0) {
        const uint32_t d = tmem + C::kS + 128 * (j & 1);
        const uint64_t kt = dk + (j % C::kStages) * (TL::kBytes >> 4);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int ks = 0; ks < D / 32; ++ks)
            mma_f8_ss(d, dq + part * (TL::kBytes >> 4) + k_off(ks), kt + k_off(ks), iqk, part | ks);
        tc::mma_commit(b_s + 8 * (j & 1));
        tc::mma_commit(b_kempty + 8 * (j % C::kStages));
      }
      __syncwarp();
    };
    auto pv = [&](int j) {
      if (lane == 0) {
        const uint32_t pa = tmem + C::kS + 128 * (j & 1);
        const uint64_t vt = dv + (j % C::kStages) * (TL::kBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < kTile / 32; ++ks)
#pragma unroll
          for (int part = 0; part < 3; ++part)
            mma_f8_ts(tmem + C::kO, pa + ks * 32 + part * 8, vt + ks * (32 * TL::kRow >> 4), ipv, (j > 0) | (ks | part));
        tc::mma_commit(b_pv + 8 * (j & 1));
        tc::mma_commit(b_vempty + 8 * (j % C::kStages));
      }
      __syncwarp();
    };
    // V rows past the request's length hold whatever their page holds: 0 * NaN is not 0
    auto clear_tail = [&](int j) {
      const int from = len - (u.tile0 + j) * kTile;
      if (from >= kTile || (from & (kGroup - 1)) == 0) return;
      const int rows = kGroup - (from & (kGroup - 1));
      const uint32_t vt = s_v + (j % C::kStages) * TL::kBytes;
      for (int i = lane; i < rows * (D / 16); i += 32)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + TL::chunk_at(from + i / (D / 16), i % (D / 16))), "r"(0) : "memory");
      tc::fence_async_smem();
      __syncwarp();
    };
    // step by step: scores of tile i, then the products of tile i - 1
#pragma unroll 1
    for (int i = 0; ok && i <= tiles; ++i) {
      const int j = i - 1;
      if (i < tiles) {
        if (!(ok = wait(b_kfull + 8 * (i % C::kStages), (i / C::kStages) & 1))) break;
        qk(i);
      }
      if (j >= 0) {
        if (!(ok = wait(b_vfull + 8 * (j % C::kStages), (j / C::kStages) & 1))) break;
        clear_tail(j);
        if (!(ok = wait(b_p + 8 * (j & 1), use(j)))) break;
        tc::fence_after_sync();
        pv(j);
      }
    }
  } else {
    split_queries<D, C::kRows, C::kSoftWarps>(a, u, G, rows_all, s_q, s_factor);
    tc::fence_async_smem();
    mbar_arrive(b_q);

    // ---- softmax: kSplitC threads a row, NC of the tile's columns each
    const int half = warp / 4;                    // which of the row's threads
    const int r = (warp & 3) * 32 + lane;         // row of the unit
    const int row = u.row0 + r;                   // (token, head) row of the request
    const bool live = row < rows_all;
    const int token = live ? row / G : 0;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int team = 1 + (warp & 3);              // the barrier of the warps that share rows
    bool ok = wait(b_q, 0);
    const float given = s_factor[r];
    const bool finite = given == given;
    const float factor = finite ? given : 0.0f;
    const int sees = live ? min(len, len - n + token + 1) : 0;  // keys this row sees
    // keys before this one are seen by every row of the warp
    const int all_see = __reduce_min_sync(0xFFFFFFFFu, sees);
    const int partial = first_partial(u, G);
    float m = -INFINITY, l = finite || sees <= 0 ? 0.0f : __int_as_float(0x7FC00000);
    // the two warps of a row agree on when to leave; a warp whose wait runs out meets the other until then
    bool left = false;
    for (int j = 0; j < tiles; ++j) {
      const int slot = (j / C::kBatch) % C::kBatches;
      ok = __all_sync(0xFFFFFFFFu, ok && wait(b_info + 8 * slot, (j / C::kInfoRing) & 1) && wait(b_s + 8 * (j & 1), use(j)));
      const uint32_t sc = tmem + C::kS + 128 * (j & 1) + half * NC + lanes;
      const float4* scales = s_scale + (j % C::kInfoRing) * kGroups;
      const int cut = sees - (u.tile0 + j) * kTile - half * NC;      // columns from here on are hidden
      const bool masked = all_see < (u.tile0 + j) * kTile + (half + 1) * NC;
      // 32 scores, -inf where they are hidden. 64 are read twice (for the maximum, for the exponentials)
      // rather than kept: registers for four such warps on a scheduler are worth more.
      auto scores = [&](int c, float (&s)[32]) {
        tmem_ld32(sc + c, s);
        tc::tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (c + i >= cut) s[i] = -INFINITY;
            asm volatile("" : "+f"(s[i]));  // kept behind the branch: as selects these cost every tile
          }
        }
      };
      // the largest exponent of the thread's columns; a page that is none has rows of zeros: its exponents become
      // -infinity by what is added
      float mx = -INFINITY;
      float s[32];
      if (ok) {
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < NC; c += 32) {
          scores(c, s);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float t0 = s[g * kGroup];
#pragma unroll
            for (int i = 1; i + 1 < kGroup; i += 2) t0 = max3(t0, s[g * kGroup + i], s[g * kGroup + i + 1]);
            t0 = fmaxf(t0, s[g * kGroup + kGroup - 1]);
            const float4 e = scales[half * NG + c / kGroup + g];
            mx = fmaxf(mx, fmaf(t0, exponent_scale(e.x, factor), e.y));
          }
        }
      }
      s_max[((j & 1) * C::kSplitC + half) * C::kRows + r] = mx;
      int gone;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
          : "=r"(gone)
          : "r"(static_cast<int>(!ok)), "r"(team), "n"(32 * C::kSplitC)
          : "memory");
      if (gone) {
        left = true;
        break;
      }
#pragma unroll
      for (int i = 1; i < C::kSplitC; ++i) mx = fmaxf(mx, s_max[((j & 1) * C::kSplitC + (half ^ i)) * C::kRows + r]);
      if (__any_sync(0xFFFFFFFFu, mx > m + 4.0f)) {
        const float to = mx > m + 4.0f ? mx : m;  // by the row alone, whatever its neighbours do
        const float root = to == -INFINITY ? 1.0f : ex2_root(m - to), corr = root * root;
        m = to;
        l = l * root * root;
        if (j > 0) {
          ok = __all_sync(0xFFFFFFFFu, wait(b_pv + 8 * ((j - 1) & 1), use(j - 1)));
          if (ok) {
            tc::fence_after_sync();
#pragma unroll 1
            for (int c = half * (D / C::kSplitC); c < (half + 1) * (D / C::kSplitC); c += 32) {
              float o[32];
              tmem_ld32(tmem + C::kO + lanes + c, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= corr;
              tmem_st32(tmem + C::kO + lanes + c, o);
            }
          }
        }
      }
      const float base = m == -INFINITY ? 0.0f : 11.0f - m;
#pragma unroll 1
      for (int c = 0; c < NC; c += 32) {
        float w[24];  // high, middle and low parts of four keys each
        if (NC > 32) scores(c, s);
        if (scales[0].w != 0.0f) l += far_sum(s, scales + half * NG + c / kGroup, factor, base);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          // p * vs comes out of the exponential; the row sum takes vs back by group
          const float4 e = scales[half * NG + c / kGroup + g];
          const float ks = exponent_scale(e.x, factor), add = base + e.y;
          const float2 k2 = make_float2(ks, ks), b2 = make_float2(add, add);
          float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < kGroup; i += 4) {
            uint32_t h[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int at = g * kGroup + i + 2 * y;
              float2 v = fma2(make_float2(s[at], s[at + 1]), k2, b2);
              v.x = ex2(v.x);
              v.y = ex2(v.y);
              sum = add2(sum, v);
              asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[y]) : "f"(v.y), "f"(v.x));
            }
            uint32_t part[3];
            split_e5m2(h, part);
#pragma unroll
            for (int y = 0; y < 3; ++y) w[y * 8 + g * 4 + i / 4] = __uint_as_float(part[y]);
          }
          l = fmaf(sum.x + sum.y, e.z, l);
        }
        tmem_st8(sc + c, w);
        tmem_st8(sc + c + 8, w + 8);
        tmem_st8(sc + c + 16, w + 16);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      if (j >= partial) {
        ok = ok && wait(b_vfull + 8 * (j % C::kStages), (j / C::kStages) & 1);
        if (ok) clear_nan<D, 32 * C::kSoftWarps>(s_v + (j % C::kStages) * TL::kBytes, (u.tile0 + j) * kTile, len, seen_by_all(u, G), tid, s_nan);
        tc::fence_async_smem();
      }
      mbar_arrive(b_p + 8 * (j & 1));
      if (j % C::kBatch == C::kBatch - 1 && lane == 0) mbar_arrive(b_infoe + 8 * slot);  // (the warp has met at the store)
    }
    // epilogue
    if (ok && tiles > 0) ok = wait(b_pv + 8 * ((tiles - 1) & 1), use(tiles - 1));
    ok = __all_sync(0xFFFFFFFFu, ok && !left);
    if (!left) {  // the row's sum from its threads
      s_max[((tiles & 1) * C::kSplitC + half) * C::kRows + r] = l;
      asm volatile("barrier.cta.sync %0, %1;" ::"r"(team), "n"(32 * C::kSplitC) : "memory");
      l = 0.0f;
#pragma unroll
      for (int i = 0; i < C::kSplitC; ++i) l += s_max[((tiles & 1) * C::kSplitC + i) * C::kRows + r];
    }
    if (ok) {
      tc::fence_after_sync();
      if (u.slot >= 0 && live && half == 0) p.ml[static_cast<int64_t>(u.slot) * C::kRows + r] = make_float2(m, l);
      store_rows<D, D / C::kSplitC, C::kQ / C::kSoftWarps>(p, u, C::kRows, r, live, token, row - token * G, G, tiles, l,
                                                           tmem + C::kO + lanes, half * (D / C::kSplitC),
                                                           s_q + warp * (C::kQ / C::kSoftWarps), s_nan);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (s_fail) {  // a wait ran out: leave only once what is in flight has landed
    if (tid == 0 && a.err) atomicOr(a.err, GDN_DEVERR_TIMEOUT);
    if (warp >= C::kSoftWarps + 2)
      for (int i = max(0, copies - C::kStages); i < copies; ++i)
        mbar_wait_bounded((warp == C::kSoftWarps + 2 ? b_kfull : b_vfull) + 8 * (i % C::kStages), (i / C::kStages) & 1);
    if (warp == C::kSoftWarps && lane == 0) {
      tc::mma_commit(b_drain);
      mbar_wait_bounded(b_drain, 0);
    }
    __syncthreads();
  }
  if (warp == C::kSoftWarps) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------- head_dim 64 and 128
//
// Here a key costs half the MMA time and the same softmax, so the softmax and shared memory decide. Probabilities
// are f16 (one conversion for two of them), and a warpgroup converts each tile of V to f16; e4m3 values are exact in f16.
// m stands for 2^7 and moves when a y passes it by 2^8: p <= 2^15, 11 significant bits, and a key is rounded to 2^-32 of
// the row's largest.
//
// Scores of three tiles are in tensor memory (3 x 128 columns, and D of output): Q K of the next tiles runs under
// the softmax. Two warpgroups take the tiles in turn, thread = row, and hand m on; Q K and P V are issued by a thread
// each, so that the waits of one pass under the products of the other. A CTA takes units as they come (the list holds up
// to three times the units that a call has, and a CTA that only finds the list at its end costs as long as any start:
// 8 ragged prompts 312 us then, and 337 with a CTA per place of the list; for head_dim 256 the loop around a unit cost
// more registers than there are). Per tile and 128 rows, the products take
// about 1,110 cycles of the tensor pipe, and nearly as many of shared memory: Q, K and V in f16 as operands, V read
// and written by the conversion, the copies; together 1,400. Measured about 1,950: 300 tokens at 60,000 (32 / 8
// heads of 128) 370 us (366 then), against 198 for the same program without the arithmetic of softmax and conversion, and 301
// with one MMA a product and no conversion (then 371). Not kept: 256 rows (two row tiles, one score buffer each: 402
// us, each tile's chain of softmax and products exposed); sixteen softmax warps (385: a vote between the two threads of a row); p computed before its tile's
// maximum is known and again where that passes (420: twice the registers and code).
template <int D>
struct NarrowCfg {
  static constexpr int kRows = 128;
  static constexpr int kSoftWarps = 8, kConvWarps = 4;
  static constexpr int kThreads = 32 * (kSoftWarps + kConvWarps + 5);  // and warps for Q K, P V, lookups, copies of K and V
  static constexpr int kStagesK = 4, kStagesV = 3, kStagesW = 2, kScores = 3;  // W: V in f16
  static constexpr int kBatch = 4, kBatches = 4, kInfoRing = kBatch * kBatches;
  using TL = Tile<D>;
  using TV = Tile<2 * D>;                                 // V in f16: rows of 2 D bytes
  static constexpr int kQ = 2 * TL::kBytes;               // hi and lo
  static constexpr int kAtK = kQ;
  static constexpr int kAtV = kAtK + kStagesK * TL::kBytes;
  static constexpr int kAtV16 = kAtV + kStagesV * TL::kBytes;
  static constexpr int kAtScale = kAtV16 + kStagesW * TV::kBytes;  // [kInfoRing][kGroups]
  static constexpr int kAtRow = kAtScale + kInfoRing * kGroups * 16;
  static constexpr int kAtFactor = kAtRow + kInfoRing * kGroups * 4;  // [kRows]
  static constexpr int kAtMax = kAtFactor + kRows * 4;             // [3][kRows]: reference, two sums
  static constexpr int kAtNan = kAtMax + 3 * kRows * 4;            // [D + 1], see clear_nan
  static constexpr int kAtBars = kAtNan + (D + 2) * 4;
  static constexpr int kBars = 2 * kStagesK + 2 * kStagesV + kStagesW + 2 * kBatches + 3 * kScores + 3 + kSoftWarps;
  static constexpr int kSmem = 1024 + kAtBars + 8 * kBars;
  static constexpr int kO = 128 * kScores;                // tensor memory: scores of three tiles, then output
};

template <int D>
__global__ void __launch_bounds__(NarrowCfg<D>::kThreads, 1)
    attn_prefill_narrow_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CacheMaps maps) {
  using C = NarrowCfg<D>;
  using TL = typename C::TL;
  using TV = typename C::TV;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ PrefillUnit s_unit;
  __shared__ volatile int s_fail, s_next;
  constexpr int kMma = C::kSoftWarps + C::kConvWarps, kLook = kMma + 2, kCopyK = kMma + 3, kCopyV = kMma + 4;

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // (known to be the same in a warp)
  const AttnArgs& a = p.a;
  if (tid < 4) prefetch_map(tid == 0 ? &maps.k_page : tid == 1 ? &maps.v_page : tid == 2 ? &maps.k_group : &maps.v_group);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int units = *reinterpret_cast<volatile int32_t*>(p.counts);
  if (static_cast<int>(blockIdx.x) >= units) return;
  const int G = a.Hq / a.H;
  if (tid == 0) s_fail = 0;
  if (warp == kMma) {
    tc::tmem_alloc(&s_tmem, 512);
    tc::tmem_relinquish();
  }
  auto wait = [&](uint32_t b, int parity) { return wait_or_fail(b, parity, &s_fail); };

#pragma unroll 1
  for (int next = blockIdx.x;; next = s_next) {
    uint32_t slack = -smem_addr(smem_raw) & 1023u;
    asm volatile("" : "+r"(slack));  // (addresses are worked out per unit: kept from one to the next they cost spills)
    unsigned char* smem = smem_raw + slack;
    const uint32_t s_q = smem_addr(smem), s_k = s_q + C::kAtK, s_v = s_q + C::kAtV, s_v16 = s_q + C::kAtV16;
    float4* s_scale = reinterpret_cast<float4*>(smem + C::kAtScale);
    int32_t* s_row = reinterpret_cast<int32_t*>(smem + C::kAtRow);
    float* s_factor = reinterpret_cast<float*>(smem + C::kAtFactor);
    float* s_max = reinterpret_cast<float*>(smem + C::kAtMax);
    int32_t* s_nan = reinterpret_cast<int32_t*>(smem + C::kAtNan);
    const uint32_t b_kfull = s_q + C::kAtBars, b_kempty = b_kfull + 8 * C::kStagesK, b_vfull = b_kempty + 8 * C::kStagesK,
                   b_vempty = b_vfull + 8 * C::kStagesV, b_wfull = b_vempty + 8 * C::kStagesV, b_info = b_wfull + 8 * C::kStagesW,
                   b_infoe = b_info + 8 * C::kBatches, b_s = b_infoe + 8 * C::kBatches, b_pv = b_s + 8 * C::kScores,
                   b_p = b_pv + 8 * C::kScores, b_q = b_p + 8 * C::kScores, b_drain = b_q + 8, b_turn = b_drain + 16;
    if (tid < static_cast<int>(sizeof(PrefillUnit) / 4)) reinterpret_cast<int*>(&s_unit)[tid] = reinterpret_cast<const int*>(p.units + next)[tid];
    if (tid <= D) s_nan[tid] = tid < D ? 0x7FFFFFFF : 0;
    if (tid < C::kBars) {
      // who arrives: a copy, a commit or one lane, but for what threads and warps release themselves
      const uint32_t b = b_kfull + 8 * tid;
      if (next != static_cast<int>(blockIdx.x)) mbar_inval(b);
      mbar_init(b, b >= b_vempty && b < b_info ? 32 * C::kConvWarps
                   : b >= b_infoe && b < b_s   ? C::kSoftWarps + 1
                   : b >= b_p && b < b_q       ? C::kSoftWarps / 2
                   : b == b_q                  ? 32 * C::kSoftWarps
                                               : 1);
    }
    fence_mbar_init();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    const PrefillUnit& u = s_unit;
    const int n = u.n, len = u.len;
    const int rows_all = n * G;  // (below 2^31: the caller's tokens x heads are)
    const int tiles = u.tile1 - u.tile0;
    // the CTA's next unit, on its way under this one (its readers are past the barrier above)
    if (tid == 32 * kLook) s_next = gridDim.x + atomicAdd(p.counts + 2, 1);

    int copies = 0;  // of a copying warp
    if (warp == kLook) {
      look_up<C>(p, u, tiles, s_scale, s_row, b_info, b_infoe, &s_fail);
    } else if (warp == kCopyK) {
      copies = copy_tiles<D, C, C::kStagesK>(a, u, tiles, &maps.k_page, &maps.k_group, s_k, s_row, b_kfull, b_kempty, b_info, 0, &s_fail);
    } else if (warp == kCopyV) {
      copies = copy_tiles<D, C, C::kStagesV>(a, u, tiles, &maps.v_page, &maps.v_group, s_v, s_row, b_vfull, b_vempty, b_info, b_infoe, &s_fail);
    } else if (warp >= kMma) {
      // ---- MMAs: a thread for Q K and one for P V, so that the waits and commits of one pass under the products of
      // the other. Scores of tile i go where those of i - 3 were, once their probabilities have been multiplied.
      // Descriptors but for their start address, which each MMA adds.
      constexpr uint32_t iqk = idesc_f8(128, kTile, false, false);
      constexpr uint32_t ipv = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | (8u << 24);  // f16 x f16 (MN-major) -> fp32
      const uint64_t dk = TL::desc(s_k, 16), dq = TL::desc(s_q, 16), dv = TV::desc(s_v16, TV::kHalf);
      if (lane == 0 && warp == kMma) {
        bool ok = tiles == 0 || wait(b_q, 0);
        int st = 0, ph = 0, buf = 0, sph = 1;
#pragma unroll 1
        for (int i = 0; ok && i < tiles; ++i) {
          if (!wait(b_kfull + 8 * st, ph) || !wait(b_pv + 8 * buf, sph)) break;
          tc::fence_after_sync();
          const uint64_t kt = dk + st * (TL::kBytes >> 4);
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks)
              mma_f8_ss(tmem + 128 * buf, dq + part * (TL::kBytes >> 4) + ks * 2, kt + ks * 2, iqk, part | ks);
          tc::mma_commit(b_s + 8 * buf);
          tc::mma_commit(b_kempty + 8 * st);
          if (++st == C::kStagesK) st = 0, ph ^= 1;
          if (++buf == C::kScores) buf = 0, sph ^= 1;
        }
        // the barriers are made anew for the next unit: no commit may be on its way
#pragma unroll 1
        for (int i = max(0, tiles - C::kStagesK); i < tiles && !s_fail; ++i) wait(b_kempty + 8 * (i % C::kStagesK), (i / C::kStagesK) & 1);
      } else if (lane == 0) {
        int buf = 0, sph = 0;
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
          if (!wait(b_wfull + 8 * (j & 1), (j >> 1) & 1) || !wait(b_p + 8 * buf, sph)) break;
          tc::fence_after_sync();
          const uint32_t pa = tmem + 128 * buf;
          const uint64_t vt = dv + (j & 1) * (TV::kBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            tc::mma_bf16_ts(tmem + C::kO, pa + (ks >> 1) * 32 + (ks & 1) * 8, vt + ks * (16 * TV::kRow >> 4), ipv, (j > 0) | ks);
          tc::mma_commit(b_pv + 8 * buf);
          if (++buf == C::kScores) buf = 0, sph ^= 1;
        }
#pragma unroll 1
        for (int j = max(0, tiles - C::kScores); j < tiles && !s_fail; ++j) wait(b_pv + 8 * (j % C::kScores), (j / C::kScores) & 1);
      }
      __syncwarp();
    } else if (warp >= C::kSoftWarps) {
      // ---- V to f16: 16-byte chunks of a tile to the threads in turn; keys past the request's length, which hold
      // whatever their page holds, become zero (0 * NaN is not 0)
      const int me = tid - 32 * C::kSoftWarps;
      constexpr int kChunks = D / 16;  // of a key
      const int partial = first_partial(u, G);
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < tiles && ok; ++j) {
        const int st = j % C::kStagesV;
        ok = wait(b_vfull + 8 * st, (j / C::kStagesV) & 1) && (j < 2 || wait(b_pv + 8 * ((j - 2) % C::kScores), ((j - 2) / C::kScores) & 1));
        if (!ok) break;
        const int keys = len - (u.tile0 + j) * kTile;
        // (a thread clears the chunks that it converts)
        if (j >= partial)
          clear_nan<D, 32 * C::kConvWarps>(s_v + st * TL::kBytes, (u.tile0 + j) * kTile, len, seen_by_all(u, G), me, s_nan);
        const uint32_t from = s_v + st * TL::kBytes, to = s_v16 + (j & 1) * TV::kBytes;
#pragma unroll 4
        for (int i = me; i < kTile * kChunks; i += 32 * C::kConvWarps) {
          const int key = i / (8 * kChunks) * 8 + i % 8, c = i / 8 % kChunks;  // (8 keys at a time: no bank twice)
          uint32_t x[4], y[8];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(from + TL::chunk_at(key, c)));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (key >= keys) x[e] = 0;
            asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.rn.f16x2.e4m3x2 %0, lo; cvt.rn.f16x2.e4m3x2 %1, hi;}" : "=r"(y[2 * e]), "=r"(y[2 * e + 1]) : "r"(x[e]));
          }
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + TV::chunk_at(key, 2 * c)), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + TV::chunk_at(key, 2 * c + 1)), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7]) : "memory");
        }
        tc::fence_async_smem();
        mbar_arrive(b_wfull + 8 * (j & 1));
        mbar_arrive(b_vempty + 8 * st);
      }
    } else {
      split_queries<D, C::kRows, C::kSoftWarps>(a, u, G, rows_all, s_q, s_factor);
      tc::fence_async_smem();
      mbar_arrive(b_q);

      // ---- softmax: thread = row; the two warpgroups take the tiles in turn. The reference that both subtract, m, is
      // what the tile before left: warps w and w + 4, which have the same rows, hand it on.
      const int own = warp / 4, pair = warp & 3, r = pair * 32 + lane;  // r: row of the unit
      int sees = 0;                       // keys this row, a (token, head) pair of the request, sees
      if (u.row0 + r < rows_all) sees = min(len, len - n + (u.row0 + r) / G + 1);
      const uint32_t lanes = static_cast<uint32_t>(pair * 32) << 16;
      bool ok = wait(b_q, 0);
      const float given = s_factor[r];
      const bool finite = given == given;
      const float factor = finite ? given : 0.0f;
      const int all_see = __reduce_min_sync(0xFFFFFFFFu, sees);   // keys before this one are seen by every row of the warp
      // a query that is not finite saturates in 8 bits: its row is NaN through its sum
      float m = -INFINITY, l = finite || sees <= 0 ? 0.0f : __int_as_float(0x7FC00000);
      const uint32_t turn = b_turn + 8 * (4 * own + pair), turn_of = b_turn + 8 * (4 * (own ^ 1) + pair);
      // whether any thread of the two warps says so
      auto vote = [&](bool x) {
        uint32_t any;
        asm volatile("{.reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, %2, 64, p; selp.u32 %0, 1, 0, q;}"
                     : "=r"(any) : "r"(static_cast<uint32_t>(x)), "r"(1 + pair) : "memory");
        return any != 0;
      };
      int buf = own, sph = 0;
#pragma unroll 1
      for (int j = own; j < tiles; j += 2) {
        const int slot = (j / C::kBatch) % C::kBatches;
        if (j % C::kBatch < 2) ok = ok && wait(b_info + 8 * slot, (j / C::kInfoRing) & 1);
        ok = ok && wait(b_s + 8 * buf, sph);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t sc = tmem + 128 * buf + lanes;
        const float4* scales = s_scale + (j % C::kInfoRing) * kGroups;
        const int cut = sees - (u.tile0 + j) * kTile;  // columns from here on are hidden
        const bool masked = all_see < (u.tile0 + j + 1) * kTile;
        // the largest exponent of the tile; a page that is none has rows of zeros: its exponents become -infinity by what
        // is added
        auto hide = [&](float (&s)[32], int c) {
          if (masked) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (c + i >= cut) s[i] = -INFINITY;
              asm volatile("" : "+f"(s[i]));  // kept behind the branch: as selects these cost every tile
            }
          }
        };
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < kTile; c += 32) {
          float s[32];
          tmem_ld32(sc + c, s);
          tc::tmem_wait_ld();
          hide(s, c);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float4 e = scales[c / kGroup + g];
            float t0 = s[g * kGroup];
#pragma unroll
            for (int i = 1; i + 1 < kGroup; i += 2) t0 = max3(t0, s[g * kGroup + i], s[g * kGroup + i + 1]);
            mx = fmaxf(mx, fmaf(fmaxf(t0, s[g * kGroup + kGroup - 1]), exponent_scale(e.x, factor), e.y));
          }
        }
        if (j > 0) ok = __all_sync(0xFFFFFFFFu, wait(turn_of, ((j - 1) >> 1) & 1));
        if (!ok) break;
        // the reference follows the row's maximum once that passes it by 2^8 (f16 has the range): by the row alone,
        // whatever its neighbours do
        const float was = j > 0 ? s_max[r] : -INFINITY, to = mx > was + 8.0f ? mx : was;
        const bool scaled = j > 0 && __any_sync(0xFFFFFFFFu, to != was);
        s_max[r] = to;
        __syncwarp();
        if (lane == 0) mbar_arrive(turn);
        if (to != m) {
          const float root = ex2_root(m - to);
          l = l * root * root;
        }
        m = to;
        if (scaled) {
          ok = __all_sync(0xFFFFFFFFu, wait(b_pv + 8 * ((j - 1) % C::kScores), ((j - 1) / C::kScores) & 1));
          if (!ok) break;
          tc::fence_after_sync();
          const float corr = to != was ? ex2(was - to) : 1.0f;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tc::tmem_ld16(tmem + C::kO + lanes + c, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= corr;
            tc::tmem_st16(tmem + C::kO + lanes + c, o);
          }
        }
        // the probabilities: p * vs comes out of the exponential; the row sum takes vs back by group
        const float base = m == -INFINITY ? 0.0f : 7.0f - m;
        if (scales[0].w != 0.0f) {  // (in the loop below, a branch for each group took 4% of the time)
#pragma unroll 1
          for (int c = 0; c < kTile; c += 32) {
            float s[32];
            tmem_ld32(sc + c, s);
            tc::tmem_wait_ld();
            hide(s, c);
            l += far_sum(s, scales + c / kGroup, factor, base);
          }
        }
#pragma unroll 1
        for (int c = 0; c < kTile; c += 32) {
          float cur[32];
          tmem_ld32(sc + c, cur);
          tc::tmem_wait_ld();
          hide(cur, c);
          uint32_t w[16];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float4 e = scales[c / kGroup + g];
            const float ks = exponent_scale(e.x, factor), add = base + e.y;
            const float2 k2 = make_float2(ks, ks), b2 = make_float2(add, add);
            float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kGroup; i += 2) {
              float2 v = fma2(make_float2(cur[g * kGroup + i], cur[g * kGroup + i + 1]), k2, b2);
              v.x = ex2(v.x);
              v.y = ex2(v.y);
              part = add2(part, v);
              asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[(g * kGroup + i) / 2]) : "f"(v.y), "f"(v.x));
            }
            l = fmaf(part.x + part.y, e.z, l);
          }
          tmem_st16u(sc + c, w);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_p + 8 * buf);
        if (j % C::kBatch >= 2 && lane == 0) mbar_arrive(b_infoe + 8 * slot);
        buf += 2;
        if (buf >= C::kScores) buf -= C::kScores, sph ^= 1;
      }
      // the last two products in order: a barrier's parity tells a product only from the one before on it
#pragma unroll 1
      for (int j = max(0, tiles - 2); j < tiles; ++j) ok = ok && wait(b_pv + 8 * (j % C::kScores), (j / C::kScores) & 1);
      if (!vote(!ok)) {
        const float last = tiles > 0 ? s_max[r] : -INFINITY;
        const float root = ex2_root(m - last);
        s_max[(1 + own) * C::kRows + r] = m == last ? l : l * root * root;
        if (!vote(!ok)) {
          tc::fence_after_sync();
          l = s_max[C::kRows + r] + s_max[2 * C::kRows + r];
          const int row = u.row0 + r, token = row / G;
          const bool live = row < rows_all;
          if (u.slot >= 0 && live && own == 0) p.ml[static_cast<int64_t>(u.slot) * C::kRows + r] = make_float2(last, l);
          store_rows<D, D / 2, C::kQ / C::kSoftWarps>(p, u, C::kRows, r, live, token, row - token * G, G, tiles, l,
                                                      tmem + C::kO + lanes, own * (D / 2), s_q + warp * (C::kQ / C::kSoftWarps), s_nan);
        }
      }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (s_fail) {  // a wait ran out: leave only once what is in flight has landed
      if (tid == 0 && a.err) atomicOr(a.err, GDN_DEVERR_TIMEOUT);
      const int stages = warp == kCopyK ? C::kStagesK : C::kStagesV;
      for (int i = max(0, copies - stages); i < copies; ++i)
        mbar_wait_bounded((warp == kCopyK ? b_kfull : b_vfull) + 8 * (i % stages), (i / stages) & 1);
      if (warp >= kMma && warp < kLook && lane == 0) {
        tc::mma_commit(b_drain + 8 * (warp - kMma));
        mbar_wait_bounded(b_drain + 8 * (warp - kMma), 0);
      }
      __syncthreads();
      break;
    }
    if (s_next >= units) break;
  }
  if (warp == kMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(s_tmem, 512);
  }
}

// Joins the key splits of 16 rows of a unit, in order.
template <int D>
__global__ void __launch_bounds__(256) attn_prefill_join_kernel(const __grid_constant__ PrefillParams p) {
  constexpr int kLanes = D / 4;               // threads of a row
  constexpr int kPar = 256 / kLanes;          // rows at a time
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (static_cast<int>(blockIdx.x) >= p.counts[1]) return;
  const PrefillUnit u = p.joins[blockIdx.x];
  const AttnArgs& a = p.a;
  const int first = u.first, n = u.n;
  const int G = a.Hq / a.H;
  const int d4 = threadIdx.x % kLanes;
  for (int i = threadIdx.x / kLanes; i < 16; i += kPar) {
    const int r = blockIdx.y * 16 + i, row = u.row0 + r;
    if (row >= static_cast<int64_t>(n) * G) break;
    float top = -INFINITY;
    for (int s = 0; s < u.splits; ++s) top = fmaxf(top, p.ml[static_cast<int64_t>(u.slot + s) * kUnitRows + r].x);
    float sum = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int s = 0; s < u.splits; ++s) {
      const int64_t at = static_cast<int64_t>(u.slot + s) * kUnitRows + r;
      const float2 e = p.ml[at];
      const float root = e.x == -INFINITY ? (e.y == 0.0f ? 0.0f : 1.0f) : ex2_root(e.x - top), c = root * root;
      const float4 v = *reinterpret_cast<const float4*>(p.part + at * D + d4 * 4);
      sum += e.y * root * root;
      if (e.x != -INFINITY || e.y != 0.0f) {  // (c may be 0 next to a NaN)
        o.x += v.x * c;
        o.y += v.y * c;
        o.z += v.z * c;
        o.w += v.w * c;
      }
    }
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    uint2 st;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.x) : "f"(o.y * inv), "f"(o.x * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.y) : "f"(o.w * inv), "f"(o.z * inv));
    *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(first + row / G) * a.Hq + u.h * G + row % G) * D + d4 * 4) = st;
  }
}

struct PrefillLayout {
  size_t units, joins, ml, part, total;
  int max_units, max_slots;
};
// max_slots: a request has fewer than few_units(d) row tiles x heads to be split, and at most three times
// that then.
PrefillLayout prefill_layout(int T, int B, int max_blocks, int Hq, int H, int d, int bs) {
  const int rows = kUnitRows, G = Hq / H;
  const int64_t tiles = (static_cast<int64_t>(max_blocks) * bs + kTile - 1) / kTile;
  const int64_t row_tiles = H * ((static_cast<int64_t>(T) * G + rows - 1) / rows + B);
  int64_t splits = tiles / kMinSplitTiles;
  if (splits > kMaxSplits) splits = kMaxSplits;
  int64_t slots = 0;
  if (splits > 1 && H < few_units(d)) {
    slots = row_tiles * splits;
    const int64_t most = static_cast<int64_t>(B) * 3 * few_units(d);
    if (slots > most) slots = most;
  }
  PrefillLayout L;
  L.max_units = static_cast<int>(row_tiles + slots < 0x7fffffff ? row_tiles + slots : 0x7fffffff);
  L.max_slots = static_cast<int>(slots);
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  L.units = 256;
  L.joins = up(L.units + static_cast<size_t>(L.max_units) * sizeof(PrefillUnit));
  L.ml = up(L.joins + static_cast<size_t>(slots > 0 ? L.max_units : 0) * sizeof(PrefillUnit));
  L.part = up(L.ml + static_cast<size_t>(slots) * rows * 8);
  L.total = L.part + static_cast<size_t>(slots) * rows * d * 4;
  return L;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kern)(KArgs...), dim3 grid, int threads, int smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D>
cudaError_t launch_prefill_d(const PrefillParams& p, const PrefillLayout& L, const CacheMaps& maps, const Expand4Args* expand, cudaStream_t s) {
  using C = std::conditional_t<D == 256, WideCfg, NarrowCfg<D == 256 ? 128 : D>>;
  auto kern = [] {
    if constexpr (D == 256) return attn_prefill_wide_kernel;
    else return attn_prefill_narrow_kernel<D>;
  }();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  attn_plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess && p.beside) e = launch_cache4_expand(*expand, s);
  if (e != cudaSuccess) return e;
  // head_dim 256: a CTA for each place of the list; otherwise one an SM, which takes units as they come
  const int grid = D == 256 || L.max_units < sm_count() ? L.max_units : sm_count();
  e = launch_after(kern, dim3(grid), C::kThreads, C::kSmem, s, p, maps);
  if (e != cudaSuccess || L.max_slots == 0) return e;
  const int64_t joins = static_cast<int64_t>(p.nb) * few_units(D);
  const int join_grid = static_cast<int>(joins < L.max_units ? joins : L.max_units);
  return launch_after(attn_prefill_join_kernel<D>, dim3(join_grid, C::kRows / 16), 256, 0, s, p);
}

}  // namespace

size_t attn_prefill_workspace(int T, int B, int max_blocks, int Hq, int H, int d, int bs) {
  return prefill_layout(T, B < kBatchPerLaunch ? B : kBatchPerLaunch, max_blocks, Hq, H, d, bs).total;
}

cudaError_t launch_attn_prefill(const AttnArgs& a, const Expand4Args* expand, cudaStream_t s) {
  CacheMaps maps;
  cudaError_t e = encode_cache_maps(&maps, a);
  if (e != cudaSuccess) return e;
  for (int b0 = 0; b0 < a.B; b0 += kBatchPerLaunch) {
    PrefillParams p;
    p.a = a;
    p.fault = attention_test_fault().load(std::memory_order_relaxed);
    p.b0 = b0;
    p.nb = a.B - b0 < kBatchPerLaunch ? a.B - b0 : kBatchPerLaunch;
    p.beside = expand != nullptr && b0 == 0;  // (the pages of all launches)
    const PrefillLayout L = prefill_layout(a.T, p.nb, a.max_blocks, a.Hq, a.H, a.d, a.bs);
    p.max_units = L.max_units;
    p.max_slots = L.max_slots;
    char* ws = static_cast<char*>(a.workspace);
    p.counts = reinterpret_cast<int32_t*>(ws);
    p.units = reinterpret_cast<PrefillUnit*>(ws + L.units);
    p.joins = reinterpret_cast<PrefillUnit*>(ws + L.joins);
    p.ml = reinterpret_cast<float2*>(ws + L.ml);
    p.part = reinterpret_cast<float*>(ws + L.part);
    e = a.d == 64    ? launch_prefill_d<64>(p, L, maps, expand, s)
        : a.d == 128 ? launch_prefill_d<128>(p, L, maps, expand, s)
                     : launch_prefill_d<256>(p, L, maps, expand, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace gdn
