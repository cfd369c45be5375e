// gdn_attn_prefill.cu -- attention of prompt tokens over the 8-bit paged cache, on the
// tcgen05 tensor cores.
//
// Request b has n new tokens (rows cu[b] .. cu[b+1] of q) whose keys and values are already in
// the cache as its last n of len; token i sees keys 0 .. len - n + i. Per (request, kv head) the
// rows of the product are the pairs (token, query head of the group), token-major, so a 128-row
// tile uses each key tile for all G heads.
//
// Both products run on 8-bit operands, straight from the pages: no conversion of K or V, no
// pass through registers. The other operand is split into two e4m3 parts,
//   q = q_hi + q_lo (a row scaled by a power of two so that max |q| lies in [128, 256)),
//   p = p_hi + p_lo (p_hi: p to 4 significant bits, p_lo = e4m3(p - p_hi)),
// and multiplied in two MMAs into the same fp32 accumulator. Four and four significant bits: q is
// a bf16 value (8 bits), so its split is exact down to 2^-18 of the row's largest element, and p
// keeps 8 bits, as a bf16 p would. Two 8-bit MMAs cost what one 16-bit MMA costs, so the
// bound is the dense bf16 rate, with half the shared-memory traffic for K and V.
//
// Scales. A block of keys has one ks: it enters the exponent, exp2(s * ks * factor - m). Its vs
// enters as p * (vs / vs_ref), vs_ref the largest vs seen (within 1.75); the row sum takes p
// without it. The running maximum m moves when a score passes it by 2^4, so that 16 p <= 256
// fits e4m3; the accumulator is rescaled only then.
//
// One CTA per unit: 256 rows (two 128-row tiles) for d <= 128, 128 rows for d = 256, where two
// score buffers take turns instead of two row tiles (tensor memory: 2 x 128 columns of scores,
// 256 columns of output). Warps: one warpgroup of softmax per row tile (thread = row), one warp
// issuing MMAs, one fetching pages by TMA. p overwrites the scores it came from in tensor memory
// and is the A operand of the second product there.
//
// A plan kernel turns the lengths into a list of units, the longest first. A request with few
// rows over a long cache is also cut along the keys, by a rule on its own sizes alone
// (kv_splits), and a third kernel joins the fp32 partial sums in order: results do not depend on
// the rest of the batch.
#include "gdn_cache.cuh"
#include "gdn_internal.h"
#include "gdn_ptx.cuh"
#include "gdn_tc.cuh"

namespace gdn {

namespace {

constexpr int kTile = 128;             // keys of a tile
constexpr int kGroup = 16;             // keys of one TMA box: the smallest block
constexpr int kGroups = kTile / kGroup;
constexpr int kPlanThreads = 1024;
constexpr int kBatchPerLaunch = 2048;
constexpr int kBuckets = 256;
constexpr float kLog2e = 1.4426950408889634f;
// key splits: up to this many units for a request that has fewer than kFewUnits
constexpr int kFewUnits = 76, kSplitUnits = 228, kMaxSplits = 32, kMinSplitTiles = 8;

struct PrefillUnit {
  int b, h, row0, tile0, tile1, slot;  // slot: partial sums' place, or -1: the unit is the whole
  int splits, pad;
};

struct PrefillParams {
  AttnArgs a;
  int b0, nb;
  int rows;                 // rows of a unit
  int max_units, max_slots;
  int32_t* counts;          // [0] units, [1] split tiles
  PrefillUnit* units;       // [max_units]
  PrefillUnit* joins;       // [max_units]: the first split of each split row tile
  float2* ml;               // [max_slots][rows] (maximum, sum)
  float* part;              // [max_slots][rows][d]
};

// How many pieces the key tiles of a request are cut into: the fewest rounds of an assumed 152
// CTAs, counted in tiles with a constant cost per piece.
__host__ __device__ __forceinline__ int kv_splits(int units, int tiles) {
  if (units >= kFewUnits || tiles < 2 * kMinSplitTiles) return 1;
  int best = 1, cost = 0x7fffffff;
  for (int s = 1; s <= kMaxSplits && s * kMinSplitTiles <= tiles && s * units <= kSplitUnits; ++s) {
    const int c = ((units * s + 151) / 152) * ((tiles + s - 1) / s + 4);
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
  const int G = a.Hq / a.H;
  int flags = 0, carry = 0, carry_slot = 0;
  if (tid < kBuckets) s_count[tid] = 0;
  if (tid == 0) s_joins = 0;
  for (int base = 0; base < p.nb; base += kPlanThreads) {
    const int b = base + tid;
    int units = 0, slots = 0;
    if (b < p.nb) {
      int first, n, len;
      request(p, b, first, n, len);
      if (n != a.cu_tokens[p.b0 + b + 1] - a.cu_tokens[p.b0 + b] || len != a.lens[p.b0 + b]) flags = GDN_DEVERR_SEQLENS;
      const int qt = static_cast<int>((static_cast<int64_t>(n) * G + p.rows - 1) / p.rows) * a.H;
      const int s = kv_splits(qt, (len + kTile - 1) / kTile);
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
    int bv = carry, bw = carry_slot;
    for (int i = 0; i < kPlanThreads / 32; ++i) {
      if (i < warp) {
        bv += s_warp[0][i];
        bw += s_warp[1][i];
      }
      carry += s_warp[0][i];
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
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_first[mid] <= u) lo = mid; else hi = mid - 1;
    }
    int first, n, len;
    request(p, lo, first, n, len);
    PrefillUnit d;
    d.b = lo;
    const int qt = static_cast<int>((static_cast<int64_t>(n) * G + p.rows - 1) / p.rows);
    const int s = (s_first[lo + 1] - s_first[lo]) / (qt * a.H);
    const int rem = u - s_first[lo];
    const int piece = rem % s, tile = rem / s;
    d.h = tile % a.H;
    d.row0 = (tile / a.H) * p.rows;
    const int tiles = tiles_of(d.row0, p.rows, n, len, G);
    const int each = (tiles + s - 1) / s;
    d.tile0 = min(piece * each, tiles);
    d.tile1 = min(d.tile0 + each, tiles);
    d.slot = s > 1 ? s_slot[lo] + rem : -1;
    d.splits = s;
    d.pad = 0;
    return d;
  };
  for (int u = tid; u < carry; u += kPlanThreads) {
    const PrefillUnit d = describe(u);
    atomicAdd(&s_count[kBuckets - 1 - min(d.tile1 - d.tile0, kBuckets - 1)], 1);
  }
  __syncthreads();
  if (warp == 0) {  // bucket counts to first places
    int before = 0;
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
  for (int u = tid; u < carry; u += kPlanThreads) {
    const PrefillUnit d = describe(u);
    // (the order within a bucket is free: it decides when a unit runs, not what it computes)
    p.units[atomicAdd(&s_count[kBuckets - 1 - min(d.tile1 - d.tile0, kBuckets - 1)], 1)] = d;
    if (d.splits > 1 && (d.slot - s_slot[d.b]) % d.splits == 0) p.joins[atomicAdd(&s_joins, 1)] = d;
  }
  __syncthreads();
  if (tid == 0) {
    p.counts[0] = carry;
    p.counts[1] = s_joins;
  }
}

// ------------------------------------------------------------------------------------ helpers

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{.reg .b16 x, y; cvt.rn.satfinite.e4m3x2.f32 x, %2, %1; cvt.rn.satfinite.e4m3x2.f32 y, %4, %3; mov.b32 %0, {x, y};}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}

// The 4 leading significant bits, to nearest: v * 2^20 absorbs the rest (T. J. Dekker, "A
// floating-point technique for extending the available precision", 1971).
__device__ __forceinline__ float2 top_bits(float2 v) {
  const float2 t = mul2(v, make_float2(1048577.0f, 1048577.0f));
  const float2 minus = make_float2(-1.0f, -1.0f);
  return fma2(fma2(v, minus, t), minus, t);
}

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(dst), "l"(map), "r"(x), "r"(row), "r"(bar)
      : "memory");
}

#define GDN_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : GDN_R8(r, 0), GDN_R8(r, 8), GDN_R8(r, 16), GDN_R8(r, 24)
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
#undef GDN_R8

// The factor of a score in the exponent. Never zero, so that a masked score (-inf) stays -inf: a
// smaller one moves no exponent (scores are below 2^26).
__device__ __forceinline__ float exponent_scale(float ks, float factor) { return fmaxf(fabsf(ks) * factor, 1e-37f); }

// 8-bit MMAs (kind::f8f6f4, e4m3 x e4m3, fp32 accumulators, 32 elements of K per instruction).
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}
// Instruction descriptor: fp32 D, e4m3 A and B, B optionally MN-major.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Operand tiles are rows of min(d, 128) bytes in the hardware swizzle that TMA writes (128-byte
// rows: 16-byte chunk ^ row mod 8; 64-byte rows: chunk ^ (row / 2) mod 4), 8 rows to an atom;
// d = 256 has two such tiles side by side.
//   K-major (Q, K): the stride offset is the next 8 rows; a K step of 32 is 32 bytes on.
//   MN-major (V, rows are K): the stride offset is the next 8 K rows, the leading offset the next
//   128 bytes of N; a K step of 32 is 32 rows on.
template <int D>
struct Tile {
  static constexpr int kRow = D < 128 ? D : 128;
  static constexpr int kHalf = kTile * kRow;           // one 128-row tile of kRow bytes
  static constexpr int kBytes = kTile * D;
  static __device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lbo) {
    uint64_t d = tc::smem_desc(addr, lbo, 8 * kRow);
    d |= static_cast<uint64_t>(D < 128 ? 4 : 2) << 61;  // 64-byte / 128-byte swizzle
    return d;
  }
  static __device__ __forceinline__ uint64_t k_step(uint32_t tile, int ks) {
    constexpr int per = kRow / 32;
    return desc(tile + (ks / per) * kHalf + (ks % per) * 32, 16);
  }
  static __device__ __forceinline__ uint64_t mn_step(uint32_t tile, int ks) { return desc(tile + ks * 32 * kRow, kHalf); }
  static __device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
    if (D < 128) return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
    return (chunk >> 3) * kHalf + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
  }
};

template <int D>
struct PrefillCfg {
  static constexpr int kTilesM = D == 256 ? 1 : 2;       // row tiles of a unit
  static constexpr int kRows = kTilesM * 128;
  static constexpr int kSoftWarps = 4 * kTilesM;
  static constexpr int kThreads = 32 * (kSoftWarps + 2);
  static constexpr int kStages = D == 256 ? 2 : 3;
  static constexpr int kQ = kTilesM * 2 * Tile<D>::kBytes;  // hi and lo of each row tile
  static constexpr int kKV = kStages * 2 * Tile<D>::kBytes;
  static constexpr int kScales = kStages * kGroups * 2 * 4;
  static constexpr int kSmem = 1024 + kQ + kKV + kScales + 256;
  // tensor memory columns
  static constexpr int kS = 0;         // two score buffers of 128
  static constexpr int kO = 256;       // output, D columns per row tile
};

template <int D>
__global__ void __launch_bounds__(PrefillCfg<D>::kThreads, 1)
    attn_prefill_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
  using C = PrefillCfg<D>;
  using TL = Tile<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + (-smem_addr(smem_raw) & 1023u);
  const uint32_t s_q = smem_addr(smem), s_k = s_q + C::kQ, s_v = s_k + C::kStages * TL::kBytes;
  float* s_scale = reinterpret_cast<float*>(smem + C::kQ + C::kKV);  // [stage][group][ks, vs]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kQ + C::kKV + C::kScales);
  const uint32_t bar = smem_addr(bars);
  // barriers
  const uint32_t b_kfull = bar, b_kempty = bar + 8 * C::kStages, b_vfull = bar + 16 * C::kStages,
                 b_vempty = bar + 24 * C::kStages, b_s = bar + 32 * C::kStages, b_p = b_s + 16, b_pv = b_p + 16,
                 b_q = b_pv + 16, b_drain = b_q + 8;
  static_assert(8 * (4 * C::kStages + 8) <= 256, "barriers fit");
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_fail;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const AttnArgs& a = p.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (static_cast<int>(blockIdx.x) >= *reinterpret_cast<volatile int32_t*>(p.counts)) return;
  const PrefillUnit u = p.units[blockIdx.x];
  int first, n, len;
  request(p, u.b, first, n, len);
  const int G = a.Hq / a.H;
  const int tiles = u.tile1 - u.tile0;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(b_kfull + 8 * i, 1);
      mbar_init(b_kempty + 8 * i, 1);
      mbar_init(b_vfull + 8 * i, 1);
      mbar_init(b_vempty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_s + 8 * i, 1);
      mbar_init(b_p + 8 * i, 128);
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

  // A bounded wait that also gives up once another role has.
  auto wait = [&](uint32_t b, int parity) -> bool {
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(b, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!s_fail) {
      if (mbar_try_wait_sleep(b, parity, 20000u)) return true;
      if (global_ns() - t0 > 1000000000ull) s_fail = 1;
    }
    return false;
  };

  const uint32_t kv_bytes = TL::kBytes;
  if (warp == C::kSoftWarps + 1) {
    // ---- pages: lane g < 8 fetches the 16-key group g of each tile
    const int total_rows = a.num_blocks * a.H * a.bs;  // past the map: zeros
    int done = 0;
    bool ok = true;
    for (int j = 0; j < tiles && ok; ++j) {
      const int st = j % C::kStages, ph = (j / C::kStages) & 1;
      int row = total_rows;
      float ks = -1.0f, vs = 0.0f;
      if (lane < kGroups) {
        const int pos = (u.tile0 + j) * kTile + lane * kGroup;
        if (pos < len) {
          const int page = a.block_table[static_cast<int64_t>(p.b0 + u.b) * a.max_blocks + pos / a.bs];
          if (page >= 0 && page < a.num_blocks) {
            row = (page * a.H + u.h) * a.bs + pos % a.bs;
            ks = a.k_scale[static_cast<int64_t>(page) * a.H + u.h];
            vs = a.v_scale[static_cast<int64_t>(page) * a.H + u.h];
          } else if (a.err) {
            atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);
          }
        }
      }
      ok = wait(b_kempty + 8 * st, ph ^ 1);
      if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
      if (lane == 0) mbar_arrive_expect_tx(b_kfull + 8 * st, kv_bytes);
      __syncwarp();
      if (lane < kGroups)
#pragma unroll
        for (int x = 0; x < D; x += 128)
          tma_rows(s_k + st * TL::kBytes + (x / 128) * TL::kHalf + lane * kGroup * TL::kRow, &kmap, x, row, b_kfull + 8 * st);
      ok = wait(b_vempty + 8 * st, ph ^ 1);
      if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; done = 2 * j + 1; break; }
      if (lane < kGroups) {
        s_scale[(st * kGroups + lane) * 2] = ks;
        s_scale[(st * kGroups + lane) * 2 + 1] = vs;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(b_vfull + 8 * st, kv_bytes);
      __syncwarp();
      if (lane < kGroups)
#pragma unroll
        for (int x = 0; x < D; x += 128)
          tma_rows(s_v + st * TL::kBytes + (x / 128) * TL::kHalf + lane * kGroup * TL::kRow, &vmap, x, row, b_vfull + 8 * st);
      done = 2 * j + 2;
    }
    if (s_fail) {  // leave only once every copy has landed
      for (int i = max(0, done - 2 * C::kStages); i < done; ++i)
        mbar_wait_bounded(((i & 1) ? b_vfull : b_kfull) + 8 * ((i / 2) % C::kStages), ((i / 2) / C::kStages) & 1);
    }
  } else if (warp == C::kSoftWarps) {
    // ---- MMAs
    constexpr uint32_t iqk = idesc_f8(128, kTile, false), ipv = idesc_f8(128, D, true);
    bool ok = tiles == 0 || wait(b_q, 0);
    tc::fence_after_sync();
    auto qk = [&](int j, int t) {  // scores of row tile t, key tile j
      if (lane == 0) {
        const uint32_t d = tmem + C::kS + 128 * (C::kTilesM == 2 ? t : j & 1);
        const uint32_t kt = s_k + (j % C::kStages) * TL::kBytes;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int ks = 0; ks < D / 32; ++ks)
            mma_f8_ss(d, TL::k_step(s_q + (t * 2 + part) * TL::kBytes, ks), TL::k_step(kt, ks), iqk, part | ks);
        tc::mma_commit(b_s + 8 * (C::kTilesM == 2 ? t : j & 1));
        if (t == C::kTilesM - 1) tc::mma_commit(b_kempty + 8 * (j % C::kStages));
      }
      __syncwarp();
    };
    auto pv = [&](int j, int t) {
      if (lane == 0) {
        const uint32_t pa = tmem + C::kS + 128 * (C::kTilesM == 2 ? t : j & 1);
        const uint32_t vt = s_v + (j % C::kStages) * TL::kBytes;
#pragma unroll
        for (int ks = 0; ks < kTile / 32; ++ks)
#pragma unroll
          for (int part = 0; part < 2; ++part)
            mma_f8_ts(tmem + C::kO + t * D, pa + ks * 32 + part * 8, TL::mn_step(vt, ks), ipv, (j > 0) | (ks | part));
        tc::mma_commit(b_pv + 8 * t);
        if (t == C::kTilesM - 1) tc::mma_commit(b_vempty + 8 * (j % C::kStages));
      }
      __syncwarp();
    };
    // V rows past the request's length hold whatever their page holds: 0 * NaN is not 0
    auto clear_tail = [&](int j) {
      const int at = (u.tile0 + j) * kTile;
      const int from = len - at;
      if (from >= kTile || (from & (kGroup - 1)) == 0) return;
      const int rows = kGroup - (from & (kGroup - 1));
      const uint32_t vt = s_v + (j % C::kStages) * TL::kBytes;
      for (int i = lane; i < rows * (D / 16); i += 32) {
        const int row = from + i / (D / 16), c = i % (D / 16);
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + TL::chunk_at(row, c)), "r"(0) : "memory");
      }
      tc::fence_async_smem();
      __syncwarp();
    };
    for (int j = 0; ok && j < tiles; ++j) {
      const int st = j % C::kStages, ph = (j / C::kStages) & 1;
      const int nst = (j + 1) % C::kStages, nph = ((j + 1) / C::kStages) & 1;
      if (j == 0) {
        ok = wait(b_kfull + 8 * st, ph);
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < C::kTilesM; ++t) qk(0, t);
      }
      if (C::kTilesM == 1 && j + 1 < tiles) {
        if (!(ok = wait(b_kfull + 8 * nst, nph))) break;
        qk(j + 1, 0);
      }
#pragma unroll
      for (int t = 0; t < C::kTilesM; ++t) {
        const int x = C::kTilesM == 2 ? t : j & 1;
        const int use = C::kTilesM == 2 ? j : j >> 1;
        if (!(ok = wait(b_p + 8 * x, use & 1))) break;
        if (t == 0) {
          if (!(ok = wait(b_vfull + 8 * st, ph))) break;
          clear_tail(j);
        }
        tc::fence_after_sync();
        pv(j, t);
        if (C::kTilesM == 2 && j + 1 < tiles) {
          if (t == 0 && !(ok = wait(b_kfull + 8 * nst, nph))) break;
          qk(j + 1, t);
        }
      }
    }
    if (s_fail) {  // MMAs in flight read shared memory and write tensor memory: wait for them
      if (lane == 0) {
        tc::mma_commit(b_drain);
        mbar_wait_bounded(b_drain, 0);
      }
      __syncwarp();
    }
  } else {
    // ---- softmax: thread = row
    const int t = warp / 4;                       // row tile
    const int r = tid & 127;                      // row of the tile
    const int row = u.row0 + t * 128 + r;         // (token, head) row of the request
    const int64_t rows_all = static_cast<int64_t>(n) * G;
    const bool live = row < rows_all;
    const int token = live ? row / G : 0;
    const int head = u.h * G + (live ? row % G : 0);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    // query row: scaled to [128, 256) by a power of two and split
    float factor;
    bool finite;
    {
      const uint16_t* qp = a.q + static_cast<int64_t>(first + token) * a.q_stride + static_cast<int64_t>(head) * D;
      uint32_t top = 0;
      for (int c = 0; live && c < D / 8; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(qp + c * 8);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
      }
      const int e = min(max(static_cast<int>(top >> 7), 1), 254);       // 127 + exponent of the largest
      const int down = min(max(127 + 7 - (e - 127), 1), 254);           // * 2^(7 - exponent)
      const float sc = __int_as_float(down << 23);
      // kept positive: the sign of `scale` goes to the query
      factor = fabsf(a.scale) * kLog2e / sc;
      const float put = a.scale < 0.0f ? -sc : sc;
      const uint32_t qh = s_q + (t * 2) * TL::kBytes, ql = qh + TL::kBytes;
      for (int c = 0; c < D / 16; ++c) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint4 w = live ? *reinterpret_cast<const uint4*>(qp + c * 16 + y * 8) : make_uint4(0, 0, 0, 0);
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
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
            hi[y * 2 + i] = e4m3x4(g[0], g[1], g[2], g[3]);
            lo[y * 2 + i] = e4m3x4(f[0], f[1], f[2], f[3]);
          }
        }
        const uint32_t at = TL::chunk_at(r, c);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(qh + at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(ql + at), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
      }
      finite = top < 0x7F80u;
    }
    tc::fence_async_smem();
    mbar_arrive(b_q);

    const int sees = live ? min(len, len - n + token + 1) : 0;  // keys this row sees
    // keys before this one are seen by every row of the warp
    const int all_see = __reduce_min_sync(0xFFFFFFFFu, sees);
    // a query that is not finite saturates in 8 bits: its row is NaN through its sum
    float m = -INFINITY, l = finite || sees <= 0 ? 0.0f : __int_as_float(0x7FC00000), vs_ref = 0.0f;
    bool ok = true;
    for (int j = 0; j < tiles; ++j) {
      const int x = C::kTilesM == 2 ? t : j & 1;
      const int use = C::kTilesM == 2 ? j : j >> 1;
      const int st = j % C::kStages;
      // scales are written before V's copy is armed; V is awaited for them
      ok = wait(b_vfull + 8 * st, (j / C::kStages) & 1) && wait(b_s + 8 * x, use & 1);
      if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
      tc::fence_after_sync();
      const uint32_t sc = tmem + C::kS + 128 * x + lanes;
      float s[kTile];
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tmem_ld32(sc + c, s + c);
      tc::tmem_wait_ld();
      const float* scales = s_scale + st * kGroups * 2;
      const int key0 = (u.tile0 + j) * kTile;
      if (all_see < key0 + kTile) {
        const int cut = sees - key0;
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          if (c >= cut) s[c] = -INFINITY;
      }
      float mx = -INFINITY, vmax = 0.0f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float ks = scales[2 * g];
        vmax = fmaxf(vmax, scales[2 * g + 1]);
        if (ks < 0.0f) {  // a page that is none
#pragma unroll
          for (int c = 0; c < kGroup; ++c) s[g * kGroup + c] = -INFINITY;
        }
        float t0 = s[g * kGroup];
#pragma unroll
        for (int c = 1; c + 1 < kGroup; c += 2) t0 = max3(t0, s[g * kGroup + c], s[g * kGroup + c + 1]);
        t0 = fmaxf(t0, s[g * kGroup + kGroup - 1]);
        mx = fmaxf(mx, t0 * exponent_scale(ks, factor));
      }
      const bool grow_v = vmax > 1.75f * vs_ref;
      if (__any_sync(0xFFFFFFFFu, mx > m + 4.0f) || grow_v) {
        const float to = mx > m + 4.0f ? mx : m;  // by the row alone, whatever its neighbours do
        float corr = to == -INFINITY ? 1.0f : ex2(m - to);
        m = to;
        l *= corr;
        if (grow_v) {
          corr *= vs_ref / vmax;
          vs_ref = vmax;
        }
        if (j > 0) {
          ok = wait(b_pv + 8 * t, (j - 1) & 1);
          if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tc::tmem_ld16(tmem + C::kO + t * D + lanes + c, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= corr;
            tc::tmem_st16(tmem + C::kO + t * D + lanes + c, o);
          }
        }
      }
      const float inv_vs = vs_ref > 0.0f ? 1.0f / vs_ref : 0.0f;
      const float base = m == -INFINITY ? 0.0f : 4.0f - m;
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int c = 0; c < kTile; c += 32) {
        uint32_t w[16];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float ks = exponent_scale(scales[2 * (c / kGroup + g)], factor);
          const float rel = scales[2 * (c / kGroup + g) + 1] * inv_vs;
          const float2 k2 = make_float2(ks, ks), b2 = make_float2(base, base), r2 = make_float2(rel, rel);
#pragma unroll
          for (int i = 0; i < kGroup; i += 4) {
            float2 hi[2], lo[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int e = c + g * kGroup + i + 2 * y;
              float2 v = fma2(make_float2(s[e], s[e + 1]), k2, b2);
              v.x = ex2(v.x);
              v.y = ex2(v.y);
              sum = add2(sum, v);
              v = mul2(v, r2);
              hi[y] = top_bits(v);
              lo[y] = add2(v, make_float2(-hi[y].x, -hi[y].y));
            }
            w[g * 4 + i / 4] = e4m3x4(hi[0].x, hi[0].y, hi[1].x, hi[1].y);
            w[8 + g * 4 + i / 4] = e4m3x4(lo[0].x, lo[0].y, lo[1].x, lo[1].y);
          }
        }
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(w[i]);
        tc::tmem_st16(sc + c, f);
      }
      l += sum.x + sum.y;
      tc::tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(b_p + 8 * x);
    }
    // epilogue
    // (with two score buffers the last two products may both be under way: a wait for the
    // last one's parity alone could pass on the one two before)
    if (C::kTilesM == 1 && ok && tiles > 1) ok = wait(b_pv + 8 * t, (tiles - 2) & 1);
    if (ok && tiles > 0) ok = wait(b_pv + 8 * t, (tiles - 1) & 1);
    if (__all_sync(0xFFFFFFFFu, ok)) {
      tc::fence_after_sync();
      const bool whole = u.slot < 0;
      const float inv = l > 0.0f || l != l ? vs_ref / l : 0.0f;
      const float mul = whole ? inv : vs_ref;
      uint16_t* op = a.out + (static_cast<int64_t>(first + token) * a.Hq + head) * D;
      const int64_t at = static_cast<int64_t>(u.slot) * C::kRows + t * 128 + r;
      float* pp = p.part + at * D;
      for (int c = 0; c < D; c += 16) {
        float o[16];
        if (tiles > 0) {
          tc::tmem_ld16(tmem + C::kO + t * D + lanes + c, o);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0.0f;
        }
        if (live && whole) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(inv == 0.0f ? 0.0f : o[2 * i + 1] * mul), "f"(inv == 0.0f ? 0.0f : o[2 * i] * mul));
          *reinterpret_cast<uint4*>(op + c) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(op + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        } else if (live) {
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(pp + c + i) = make_float4(o[i] * mul, o[i + 1] * mul, o[i + 2] * mul, o[i + 3] * mul);
        }
        __syncwarp();
      }
      if (!whole && live) p.ml[at] = make_float2(m, l);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (tid == 0 && s_fail && a.err) atomicOr(a.err, GDN_DEVERR_TIMEOUT);
  if (warp == C::kSoftWarps) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
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
  int first, n, len;
  request(p, u.b, first, n, len);
  const int G = a.Hq / a.H;
  const int d4 = threadIdx.x % kLanes;
  for (int i = threadIdx.x / kLanes; i < 16; i += kPar) {
    const int r = blockIdx.y * 16 + i, row = u.row0 + r;
    if (row >= static_cast<int64_t>(n) * G) break;
    float top = -INFINITY;
    for (int s = 0; s < u.splits; ++s) top = fmaxf(top, p.ml[static_cast<int64_t>(u.slot + s) * p.rows + r].x);
    float sum = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int s = 0; s < u.splits; ++s) {
      const int64_t at = static_cast<int64_t>(u.slot + s) * p.rows + r;
      const float2 e = p.ml[at];
      const float c = e.x == -INFINITY ? (e.y == 0.0f ? 0.0f : 1.0f) : ex2(e.x - top);
      const float4 v = *reinterpret_cast<const float4*>(p.part + at * D + d4 * 4);
      sum += e.y * c;
      if (c != 0.0f) {
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

int unit_rows(int d) { return d == 256 ? 128 : 256; }

struct PrefillLayout {
  size_t units, joins, ml, part, total;
  int max_units, max_slots;
};
// max_slots: a request has fewer than kFewUnits row tiles x heads to be split, and at most
// kSplitUnits units then.
PrefillLayout prefill_layout(int T, int B, int max_blocks, int Hq, int H, int d, int bs) {
  const int rows = unit_rows(d), G = Hq / H;
  const int64_t tiles = (static_cast<int64_t>(max_blocks) * bs + kTile - 1) / kTile;
  const int64_t row_tiles = H * ((static_cast<int64_t>(T) * G + rows - 1) / rows + B);
  int64_t splits = tiles / kMinSplitTiles;
  if (splits > kMaxSplits) splits = kMaxSplits;
  int64_t slots = 0;
  if (splits > 1 && H < kFewUnits) {
    slots = row_tiles * splits;
    const int64_t most = static_cast<int64_t>(B) * kSplitUnits;
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
cudaError_t launch_prefill_d(const PrefillParams& p, const PrefillLayout& L, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, cudaStream_t s) {
  using C = PrefillCfg<D>;
  cudaError_t e = cudaFuncSetAttribute(attn_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  attn_plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_after(attn_prefill_kernel<D>, dim3(L.max_units), C::kThreads, C::kSmem, s, p, kmap, vmap);
  if (e != cudaSuccess || L.max_slots == 0) return e;
  const int64_t joins = static_cast<int64_t>(p.nb) * kFewUnits;
  const int grid = static_cast<int>(joins < L.max_units ? joins : L.max_units);
  return launch_after(attn_prefill_join_kernel<D>, dim3(grid, C::kRows / 16), 256, 0, s, p);
}

}  // namespace

size_t attn_prefill_workspace(int T, int B, int max_blocks, int Hq, int H, int d, int bs) {
  return prefill_layout(T, B < kBatchPerLaunch ? B : kBatchPerLaunch, max_blocks, Hq, H, d, bs).total;
}

cudaError_t launch_attn_prefill(const AttnArgs& a, cudaStream_t s) {
  CUtensorMap kmap, vmap;
  const int64_t rows = static_cast<int64_t>(a.num_blocks) * a.H * a.bs;
  cudaError_t e = encode_cache_map(&kmap, a.k_cache, rows, a.d, kGroup);
  if (e == cudaSuccess) e = encode_cache_map(&vmap, a.v_cache, rows, a.d, kGroup);
  if (e != cudaSuccess) return e;
  for (int b0 = 0; b0 < a.B; b0 += kBatchPerLaunch) {
    PrefillParams p;
    p.a = a;
    p.b0 = b0;
    p.nb = a.B - b0 < kBatchPerLaunch ? a.B - b0 : kBatchPerLaunch;
    p.rows = unit_rows(a.d);
    const PrefillLayout L = prefill_layout(a.T, p.nb, a.max_blocks, a.Hq, a.H, a.d, a.bs);
    p.max_units = L.max_units;
    p.max_slots = L.max_slots;
    char* ws = static_cast<char*>(a.workspace);
    p.counts = reinterpret_cast<int32_t*>(ws);
    p.units = reinterpret_cast<PrefillUnit*>(ws + L.units);
    p.joins = reinterpret_cast<PrefillUnit*>(ws + L.joins);
    p.ml = reinterpret_cast<float2*>(ws + L.ml);
    p.part = reinterpret_cast<float*>(ws + L.part);
    e = a.d == 64    ? launch_prefill_d<64>(p, L, kmap, vmap, s)
        : a.d == 128 ? launch_prefill_d<128>(p, L, kmap, vmap, s)
                     : launch_prefill_d<256>(p, L, kmap, vmap, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace gdn
