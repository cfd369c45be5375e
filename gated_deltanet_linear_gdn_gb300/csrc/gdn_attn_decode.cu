// gdn_attn_decode.cu -- attention of single tokens over the 8-bit paged cache.
//
// Per request b (len keys), kv head h and the G query heads that share it:
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),  k_j = ks * byte, v_j = vs * byte
// with one ks, vs per (block, kv head). Bound by memory: every cached byte is read once
// (2 d bytes per token and kv head) for 4 G operations per byte.
//
// Split. A (request, kv head) is cut into units of 256, 512 or 1,024 keys by its OWN length
// (unit_keys), never by the batch: a row's result depends on its own inputs alone, bit for bit,
// as for every other call of the library. A persistent grid walks the units; a unit's 16-key
// groups are dealt to the CTA's warps. A request of one unit is finished in the kernel, a longer
// one leaves fp32 partial sums (with their maximum and sum) that a second, programmatically
// dependent kernel joins in unit order.
//
// A warp works on its own: it fetches its groups by TMA into a private ring (rows of d bytes,
// hardware swizzle), so nothing in the loop waits for another warp, and the next unit's keys are
// in flight while this one is joined. Groups are 16 keys because the smallest block is 16 tokens:
// a group never crosses a block, so it has one page, one ks and one vs.
//
// Products on the warp-level f16 tensor instruction (16 x 8 x 16). A decode step has at most 8
// (or 16) query rows per kv head; the 128-row tcgen05 tile would be over 90% padding, and the
// kernel needs 4 G operations per byte, a few percent of even the warp-level rate. The keys are the
// 16-row operand and the query heads the 8-wide one, so G <= 8 wastes nothing:
//   S^T[key, head] = K Q^T,  O^T[d, head] = V^T P^T.
// Both operands come from the bytes with exact conversions (e4m3 -> f16). Any order of the d
// (and of the keys) is right for a sum, so the fragments are taken in the order in which one
// 16-byte load per lane delivers them: lane (r, j) reads the d-chunks j, j+4, .. of its key for
// S^T, and the d-chunk r of keys 2j, 2j^5 (+8) for O^T. group_key() orders the keys so that with
// the swizzle both loads are free of bank conflicts.
//
// Precision. Queries are scaled per head by a power of two (largest element in [1, 2)) and are
// then exact in f16 down to 2^-24 of that element. Maxima, sums and accumulators are fp32. P is
// rounded to f16 (11 bits; the output is bf16, 8 bits); it is taken relative to a running maximum
// that moves only when a score passes it by 2^8, so P <= 2^8, and vs enters relative to the
// largest vs seen within 2^4: |P| < 2^13 stays in f16's range.
#include <cudaTypedefs.h>

#include "gdn_cache.cuh"
#include "gdn_internal.h"
#include "gdn_ptx.cuh"

namespace gdn {

cudaError_t encode_cache_map(CUtensorMap* map, const uint8_t* cache, int64_t total_rows, int d, int rows) {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
  if (e != cudaSuccess) return e;
  if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(total_rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(d < 128 ? d : 128), static_cast<cuuint32_t>(rows)};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
      map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(cache), dims, strides, box, step,
      CU_TENSOR_MAP_INTERLEAVE_NONE, d < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {

constexpr int kGroup = 16;          // keys of one group
constexpr int kMaxUnitKeys = 1024;
constexpr int kBatchPerLaunch = 2048;  // requests of one launch (their unit counts stay in shared memory)
constexpr float kLog2e = 1.4426950408889634f;

// Keys of one unit of a request of `len` keys.
__host__ __device__ __forceinline__ int unit_keys(int len) {
  return len <= 4096 ? 256 : len <= 8192 ? 512 : kMaxUnitKeys;
}
__host__ __device__ __forceinline__ int units_of(int len) {
  const int u = unit_keys(len);
  return (len + u - 1) / u;
}
// The most units that any length up to `cap` has.
int64_t most_units(int64_t cap) {
  if (cap <= 4096) return (cap + 255) / 256;
  return cap <= 16384 ? 16 : (cap + kMaxUnitKeys - 1) / kMaxUnitKeys;
}

// The key, within a group, of fragment row r (0..7; rows 8..15 are 8 keys on). With 128-byte
// rows and the hardware swizzle (16-byte chunk ^ (row mod 8)), rows r and r + 1 have to differ in
// chunk bit 2 for S^T's loads and rows 0, 2, 4, 6 in chunk bits 1, 2 for O^T's.
__device__ __forceinline__ int group_key(int r) { return (r & 6) ^ ((r & 1) * 5); }

template <int D>
__device__ __forceinline__ uint32_t tile_at(int key, int chunk) {  // byte of a 16-byte chunk of a row
  if (D == 64) return key * 64 + ((chunk ^ ((key >> 1) & 3)) << 4);
  return (chunk >> 3) * (kGroup * 128) + key * 128 + (((chunk & 7) ^ (key & 7)) << 4);
}

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(dst), "l"(map), "r"(x), "r"(row), "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
// the low and the high e4m3 pair of a word as f16 pairs
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float bf2f_(uint32_t h) { return __uint_as_float(h << 16); }

struct DecodeParams {
  AttnArgs a;
  int heads;      // query heads of one unit: min(G, 16)
  int chunks;     // units' head chunks per kv head: ceil(G / 16)
  int b0, nb;     // the launch's requests
  int32_t* pre;   // workspace: [nb + 1] units before request b (of one kv head and chunk)
  float2* ml;     // [units][heads] (maximum, sum) of a unit that is one of several
  float* part;    // [units][heads][D]
};

template <int D, int NT, int NW>
struct DecodeCfg {
  static constexpr int kThreads = 32 * NW;
  static constexpr int kStage = 2 * kGroup * D;                  // a group's keys and values
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kRing = NW * kStages * kStage;
  static constexpr int kHeadStride = D + 4;                      // floats; padded against bank conflicts
  static constexpr int kJoin = NW * 8 * kHeadStride * 4;
  static constexpr int kSlots = kMaxUnitKeys / (kGroup * NW);    // a warp's group slots of the longest unit
  static constexpr int kInfo = NW * 64 * 16;
  static constexpr int kMl = NW * (8 * NT * 2 + 1) * 4;
  static constexpr int kFixed = kRing + kJoin + kInfo + ((kMl + 15) & ~15) + NW * kStages * 8;  // then pre[nb + 1]
  static constexpr int kAlign = 1024;                            // the swizzle repeats every 1,024 bytes
  static_assert(kSlots <= 32, "a batch of 32 lanes covers whole units");
};

// One unit of the launch: request, kv head, head chunk, its first key and the keys it holds.
struct Unit {
  int b, h, chunk, first, keys, index, count;  // index: the unit's place in its request's `count`
};

__device__ __forceinline__ Unit find_unit(const int32_t* pre, int nb, int HC, int chunks, int f,
                                          const int32_t* lens, int cap) {
  int lo = 0, hi = nb - 1;  // the last request whose units start at or before f and that has some
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(pre[mid]) * HC <= f) lo = mid; else hi = mid - 1;
  }
  Unit u;
  u.b = lo;
  u.count = pre[lo + 1] - pre[lo];
  const int rem = f - pre[lo] * HC;
  const int hc = rem / u.count;
  u.index = rem % u.count;
  u.h = hc / chunks;
  u.chunk = hc % chunks;
  const int len = min(max(lens[lo], 0), cap);
  const int uk = unit_keys(len);
  u.first = u.index * uk;
  u.keys = min(uk, len - u.first);
  return u;
}

template <int D, int NT, int NW>
__global__ void __launch_bounds__(32 * NW) attn_decode_kernel(const __grid_constant__ DecodeParams p,
                                                              const __grid_constant__ CUtensorMap kmap,
                                                              const __grid_constant__ CUtensorMap vmap) {
  using C = DecodeCfg<D, NT, NW>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + (-smem_addr(smem_raw) & (C::kAlign - 1));
  unsigned char* ring = smem;
  float* join = reinterpret_cast<float*>(smem + C::kRing);
  int4* info = reinterpret_cast<int4*>(smem + C::kRing + C::kJoin);
  float* s_m = reinterpret_cast<float*>(smem + C::kRing + C::kJoin + C::kInfo);  // [NW][8 NT]
  float* s_l = s_m + NW * 8 * NT;
  float* s_vs = s_l + NW * 8 * NT;                                               // [NW]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kFixed - NW * C::kStages * 8);
  int32_t* pre = reinterpret_cast<int32_t*>(smem + C::kFixed);                    // [nb + 1]
  __shared__ int32_t s_scan[NW];

  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, j = lane & 3;
  const int cap = a.max_blocks * a.bs;
  const int32_t* lens = a.lens + p.b0;

  if (lane == 0)
    for (int s = 0; s < C::kStages; ++s) mbar_init(smem_addr(&bars[warp * C::kStages + s]), 1);
  fence_mbar_init();
  // units before each request
  {
    int carry = 0, flags = 0;
    for (int base = 0; base < p.nb; base += C::kThreads) {
      const int b = base + tid;
      int len = 0;
      if (b < p.nb) {
        len = lens[b];
        if (len < 0 || len > cap) flags = GDN_DEVERR_SEQLENS;
        len = min(max(len, 0), cap);
      }
      int v = units_of(len);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += x;
      }
      if (lane == 31) s_scan[warp] = v;
      __syncthreads();
      int before = carry;
      for (int w = 0; w < warp; ++w) before += s_scan[w];
      if (b < p.nb) pre[b + 1] = before + v;
      for (int w = 0; w < NW; ++w) carry += s_scan[w];
      __syncthreads();
    }
    if (tid == 0) pre[0] = 0;
    if (flags && a.err && blockIdx.x == 0) atomicOr(a.err, flags);
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = tid; b <= p.nb; b += C::kThreads) p.pre[b] = pre[b];

  const int HC = a.H * p.chunks;
  const int units = pre[p.nb] * HC;
  const int G = a.Hq / a.H;
  const int mine = units > static_cast<int>(blockIdx.x)
                       ? (units - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x)
                       : 0;
  const int nslots = mine * C::kSlots;  // this warp's group slots, empty ones among them
  int4* my_info = info + warp * 64;
  const uint32_t my_ring = smem_addr(ring) + warp * C::kStages * C::kStage;
  const uint32_t my_bars = smem_addr(bars) + warp * C::kStages * 8;
  int next = 0, issued = 0, consumed = 0;  // the slot to fetch next; groups fetched and used
  bool ok = true;

  // Fetches ahead: every free stage gets the warp's next group. Slot n is group (n % kSlots) * NW + warp of
  // the CTA's unit n / kSlots; 32 slots are looked up at a time, one per lane.
  auto fetch = [&](int at) {
    while (ok && next < nslots && issued - consumed < C::kStages && next < ((at >> 5) + 2) * 32) {
      if ((next & 31) == 0) {
        const int n = next + lane;
        int4 e = make_int4(0, 0, 0, 0);  // row of the cache, keys, ks, vs
        if (n < nslots) {
          const Unit u = find_unit(pre, p.nb, HC, p.chunks, blockIdx.x + (n / C::kSlots) * gridDim.x, lens, cap);
          const int key = ((n % C::kSlots) * NW + warp) * kGroup;
          if (key < u.keys) {
            const int pos = u.first + key;
            const int page = a.block_table[static_cast<int64_t>(p.b0 + u.b) * a.max_blocks + pos / a.bs];
            if (page >= 0 && page < a.num_blocks) {
              e.x = (page * a.H + u.h) * a.bs + pos % a.bs;
              e.y = min(kGroup, u.keys - key);
              e.z = __float_as_int(a.k_scale[static_cast<int64_t>(page) * a.H + u.h]);
              e.w = __float_as_int(a.v_scale[static_cast<int64_t>(page) * a.H + u.h]);
            } else if (a.err) {
              atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);  // a page that is none: its tokens are not seen
            }
          }
        }
        my_info[n & 63] = e;
        __syncwarp();
      }
      const int4 e = my_info[next & 63];
      if (e.y > 0) {
        const int s = issued % C::kStages;
        if (lane == 0) {
          const uint32_t dst = my_ring + s * C::kStage, bar = my_bars + s * 8;
          mbar_arrive_expect_tx(bar, C::kStage);
#pragma unroll
          for (int x = 0; x < D; x += 128) {
            tma_rows(dst + x * kGroup, &kmap, x, e.x, bar);
            tma_rows(dst + kGroup * D + x * kGroup, &vmap, x, e.x, bar);
          }
        }
        ++issued;
      }
      ++next;
    }
  };

  for (int k = 0; k < mine; ++k) {
    fetch(k * C::kSlots);
    const int f = blockIdx.x + k * gridDim.x;
    const Unit u = find_unit(pre, p.nb, HC, p.chunks, f, lens, cap);
    const int head0 = u.h * G + u.chunk * 16;             // the unit's first query head
    const int heads = min(p.heads, G - u.chunk * 16);

    // queries: B fragments of Q^T, scaled per head to [1, 2)
    uint32_t qf[NT][D / 16][2];
    float qexp[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int hd = nt * 8 + r;
      const uint16_t* qp = a.q + static_cast<int64_t>(p.b0 + u.b) * a.q_stride + static_cast<int64_t>(head0 + hd) * D;
      uint4 raw[D / 64][2];
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          raw[c][x] = hd < heads ? *reinterpret_cast<const uint4*>(qp + (j + 4 * c) * 16 + x * 8) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw[c][x].x, raw[c][x].y, raw[c][x].z, raw[c][x].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
        }
      }
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const int ex = min(max(static_cast<int>(top >> 7), 1), 254) - 127;  // exponent of the largest element
      // a subnormal or non-finite largest element only loses the exact scaling, not its value
      const float down = __int_as_float((min(max(127 - ex, 1), 254)) << 23);
      qexp[nt] = 1.0f / down;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint32_t w[8] = {raw[c][0].x, raw[c][0].y, raw[c][0].z, raw[c][0].w,
                               raw[c][1].x, raw[c][1].y, raw[c][1].z, raw[c][1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          qf[nt][c * 4 + i / 2][i & 1] = pack_f16(bf2f_(w[i] & 0xFFFFu) * down, bf2f_(w[i] >> 16) * down);
      }
    }
    // the factor of heads 2j, 2j + 1
    float hf[NT][2], m[NT][2], l[NT][2];
    float acc[NT][D / 16][4];
    float vs_ref = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        hf[nt][x] = __shfl_sync(0xFFFFFFFFu, qexp[nt], (2 * j + x) * 4) * a.scale * kLog2e;
        m[nt][x] = -INFINITY;
        l[nt][x] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[nt][i][x] = 0.0f;
    }

    for (int i = 0; i < C::kSlots; ++i) {
      const int at = k * C::kSlots + i;
      fetch(at);
      const int4 e = my_info[at & 63];
      const int valid = e.y;
      if (valid == 0) continue;
      const int st = consumed % C::kStages;
      if (ok && !mbar_wait_bounded(my_bars + st * 8, (consumed / C::kStages) & 1)) ok = false;
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        ok = false;
        break;
      }
      const uint32_t kt = my_ring + st * C::kStage, vt = kt + kGroup * D;
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[nt][x] = 0.0f;
      const int key = group_key(r);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint4 ka = lds128(kt + tile_at<D>(key, j + 4 * c));
        const uint4 kb = lds128(kt + tile_at<D>(key + 8, j + 4 * c));
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t a0, a1, a2, a3;
          to_f16(wa[x], a0, a2);
          to_f16(wb[x], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], a0, a1, a2, a3, qf[nt][c * 4 + x][0], qf[nt][c * 4 + x][1]);
        }
      }
      const float ks = __int_as_float(e.z), vs = __int_as_float(e.w);
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[nt][x] *= hf[nt][x & 1] * ks;
          if (key + (x & 2) * 4 >= valid) s[nt][x] = -INFINITY;
          above |= s[nt][x] > m[nt][x & 1] + 8.0f;
        }
      if (__any_sync(0xFFFFFFFFu, above)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float t = fmaxf(s[nt][x], s[nt][x + 2]);
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 16));
            t = t > m[nt][x] + 8.0f ? t : m[nt][x];  // by the head alone, whatever the others do
            const float corr = t == -INFINITY ? 1.0f : ex2(m[nt][x] - t);
            m[nt][x] = t;
            l[nt][x] *= corr;
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
              acc[nt][q][x] *= corr;
              acc[nt][q][x + 2] *= corr;
            }
          }
      }
      if (vs > vs_ref * 16.0f) {
        const float down = vs_ref / vs;
        vs_ref = vs;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int q = 0; q < D / 16; ++q)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[nt][q][x] *= down;
      }
      const float rel = vs_ref > 0.0f ? __fdividef(vs, vs_ref) : 0.0f;
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          pr[x] = ex2(s[nt][x] - m[nt][x & 1]);
          l[nt][x & 1] += pr[x];
          pr[x] *= rel;
        }
        pb[nt][0] = transpose8x8(pack_f16(pr[0], pr[1]));
        pb[nt][1] = transpose8x8(pack_f16(pr[2], pr[3]));
      }
      // values: keys past the last one hold whatever the page holds, and 0 * NaN is not 0
      const int ke = 2 * j, ko = (2 * j) ^ 5;
      const bool cut = valid < kGroup;
      if (D >= 128) {
#pragma unroll
        for (int hh = 0; hh < D / 128; ++hh) {
          uint4 v[4];
          v[0] = lds128(vt + tile_at<D>(ke, hh * 8 + r));
          v[1] = lds128(vt + tile_at<D>(ko, hh * 8 + r));
          v[2] = lds128(vt + tile_at<D>(ke + 8, hh * 8 + r));
          v[3] = lds128(vt + tile_at<D>(ko + 8, hh * 8 + r));
          if (cut) {
            const uint4 z = make_uint4(0, 0, 0, 0);
            if (ke >= valid) v[0] = z;
            if (ko >= valid) v[1] = z;
            if (ke + 8 >= valid) v[2] = z;
            if (ko + 8 >= valid) v[3] = z;
          }
          const uint32_t w[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w},
                                    {v[2].x, v[2].y, v[2].z, v[2].w}, {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t a0, a1, a2, a3;
              to_f16(__byte_perm(w[0][x], w[1][x], y ? 0x7362 : 0x5140), a0, a1);
              to_f16(__byte_perm(w[2][x], w[3][x], y ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816(acc[nt][hh * 8 + x * 2 + y], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
            }
        }
      } else {
        uint2 v[4];
        const uint32_t sub = (r & 1) * 8;
        v[0] = lds64(vt + tile_at<D>(ke, r >> 1) + sub);
        v[1] = lds64(vt + tile_at<D>(ko, r >> 1) + sub);
        v[2] = lds64(vt + tile_at<D>(ke + 8, r >> 1) + sub);
        v[3] = lds64(vt + tile_at<D>(ko + 8, r >> 1) + sub);
        if (cut) {
          const uint2 z = make_uint2(0, 0);
          if (ke >= valid) v[0] = z;
          if (ko >= valid) v[1] = z;
          if (ke + 8 >= valid) v[2] = z;
          if (ko + 8 >= valid) v[3] = z;
        }
        const uint32_t w[4][2] = {{v[0].x, v[0].y}, {v[1].x, v[1].y}, {v[2].x, v[2].y}, {v[3].x, v[3].y}};
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t a0, a1, a2, a3;
            to_f16(__byte_perm(w[0][x], w[1][x], y ? 0x7362 : 0x5140), a0, a1);
            to_f16(__byte_perm(w[2][x], w[3][x], y ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(acc[nt][x * 2 + y], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
          }
      }
      __syncwarp();  // the stage is free: its next copy may start
      ++consumed;
    }

    // join the CTA's warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float t = l[nt][x];
        t += __shfl_xor_sync(0xFFFFFFFFu, t, 4);
        t += __shfl_xor_sync(0xFFFFFFFFu, t, 8);
        t += __shfl_xor_sync(0xFFFFFFFFu, t, 16);
        if (r == 0) {
          s_m[warp * 8 * NT + nt * 8 + 2 * j + x] = m[nt][x];
          s_l[warp * 8 * NT + nt * 8 + 2 * j + x] = t;
        }
      }
    if (lane == 0) s_vs[warp] = vs_ref;
    constexpr int DPT = D >= 128 ? 16 : 8;  // consecutive d of one lane in each 128 (or 64) of D
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float* o = join + (warp * 8 + 2 * j + x) * C::kHeadStride + r * DPT;
#pragma unroll
        for (int q = 0; q < D / 16; q += 2) {
          const int at = (q / (DPT / 2)) * 128 + (q % (DPT / 2)) * 2;
          *reinterpret_cast<float4*>(o + at) = make_float4(acc[nt][q][x], acc[nt][q][x + 2], acc[nt][q + 1][x], acc[nt][q + 1][x + 2]);
        }
      }
      __syncthreads();
      for (int e = tid; e < 8 * D / 4; e += C::kThreads) {
        const int hd = e / (D / 4), d4 = e % (D / 4) * 4;
        if (nt * 8 + hd >= heads) continue;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, s_m[w * 8 * NT + nt * 8 + hd]);
        float sum = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float mw = s_m[w * 8 * NT + nt * 8 + hd];
          const float lw = s_l[w * 8 * NT + nt * 8 + hd];
          // a warp without keys has m = -inf, l = 0; with only NaN scores m = -inf, l = NaN
          const float c = mw == -INFINITY ? (lw == 0.0f ? 0.0f : 1.0f) : ex2(mw - top);
          sum += lw * c;
          const float cv = c * s_vs[w];
          const float4 v = *reinterpret_cast<const float4*>(join + (w * 8 + hd) * C::kHeadStride + d4);
          o.x += v.x * cv;
          o.y += v.y * cv;
          o.z += v.z * cv;
          o.w += v.w * cv;
        }
        const int head = nt * 8 + hd;
        if (u.count == 1) {
          const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
          uint2 st;
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.x) : "f"(o.y * inv), "f"(o.x * inv));
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.y) : "f"(o.w * inv), "f"(o.z * inv));
          *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(p.b0 + u.b) * a.Hq + head0 + head) * D + d4) = st;
        } else {
          const int64_t at = static_cast<int64_t>(f) * p.heads + head;
          *reinterpret_cast<float4*>(p.part + at * D + d4) = o;
          if (d4 == 0) p.ml[at] = make_float2(top, sum);
        }
      }
      __syncthreads();
    }
  }
  if (!ok && lane == 0) {
    // a copy that did not come: leave once those in flight have landed
    for (; consumed < issued; ++consumed)
      mbar_wait_bounded(my_bars + (consumed % C::kStages) * 8, (consumed / C::kStages) & 1);
    if (a.err) atomicOr(a.err, GDN_DEVERR_TIMEOUT);
  }
}

// Joins the units of one request, kv head and query head in unit order; an empty request gets zeros.
template <int D>
__global__ void __launch_bounds__(128) attn_decode_join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kLanes = D / 4, kRows = 128 / kLanes;
  __shared__ float4 s_o[kRows][kLanes];
  __shared__ float s_sum[kRows], s_top[4];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const AttnArgs& a = p.a;
  const int HC = a.H * p.chunks, G = a.Hq / a.H;
  const int b = blockIdx.x / HC, hc = blockIdx.x % HC, head = blockIdx.y;
  const int qh = (hc / p.chunks) * G + (hc % p.chunks) * 16 + head;
  if ((hc % p.chunks) * 16 + head >= G) return;
  const int first = p.pre[b], n = p.pre[b + 1] - first;
  if (n == 1) return;
  const int tid = threadIdx.x, d4 = tid % kLanes, row = tid / kLanes;
  const int64_t f = static_cast<int64_t>(first) * HC + static_cast<int64_t>(hc) * n;
  const float2* ml = p.ml + f * p.heads + head;
  const float* part = p.part + (f * p.heads + head) * D;
  float top = -INFINITY;
  for (int i = tid; i < n; i += 128) top = fmaxf(top, ml[static_cast<int64_t>(i) * p.heads].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  __syncthreads();
  top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
  float sum = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int i = row; i < n; i += kRows) {
    const float2 e = ml[static_cast<int64_t>(i) * p.heads];
    const float c = e.x == -INFINITY ? (e.y == 0.0f ? 0.0f : 1.0f) : ex2(e.x - top);
    const float4 v = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(i) * p.heads * D + d4 * 4);
    sum += e.y * c;
    o.x += v.x * c;
    o.y += v.y * c;
    o.z += v.z * c;
    o.w += v.w * c;
  }
  s_o[row][d4] = o;
  if (d4 == 0) s_sum[row] = sum;
  __syncthreads();
  if (row != 0) return;
#pragma unroll
  for (int i = 1; i < kRows; ++i) {
    const float4 v = s_o[i][d4];
    sum += s_sum[i];
    o.x += v.x;
    o.y += v.y;
    o.z += v.z;
    o.w += v.w;
  }
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  uint2 st;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.x) : "f"(o.y * inv), "f"(o.x * inv));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.y) : "f"(o.w * inv), "f"(o.z * inv));
  *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(p.b0 + b) * a.Hq + qh) * D + d4 * 4) = st;
}

struct DecodeLayout {
  size_t pre, ml, part, total;
};
DecodeLayout decode_layout(int nb, int max_blocks, int Hq, int H, int d, int bs) {
  const int G = Hq / H, heads = G < 16 ? G : 16, chunks = (G + 15) / 16;
  const size_t units = static_cast<size_t>(nb) * H * chunks * most_units(static_cast<int64_t>(max_blocks) * bs);
  DecodeLayout L;
  L.pre = 0;
  L.ml = (static_cast<size_t>(nb + 1) * 4 + 255) & ~static_cast<size_t>(255);
  L.part = (L.ml + units * heads * 8 + 255) & ~static_cast<size_t>(255);
  L.total = L.part + units * heads * d * 4;
  return L;
}

template <int D, int NT, int NW>
cudaError_t launch_decode_d(DecodeParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s) {
  using C = DecodeCfg<D, NT, NW>;
  auto kern = attn_decode_kernel<D, NT, NW>;
  const int smem = C::kAlign + C::kFixed + (p.nb + 1) * 4;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int per_sm = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, C::kThreads, smem);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  const int64_t most = static_cast<int64_t>(p.nb) * p.a.H * p.chunks *
                       most_units(static_cast<int64_t>(p.a.max_blocks) * p.a.bs);
  const int grid = static_cast<int>(most < static_cast<int64_t>(per_sm) * sm_count() ? most : per_sm * sm_count());
  kern<<<grid, C::kThreads, smem, s>>>(p, kmap, vmap);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.nb * p.a.H * p.chunks, p.heads, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_join_kernel<D>, p);
}

}  // namespace

size_t attn_decode_workspace(int B, int max_blocks, int Hq, int H, int d, int bs) {
  return decode_layout(B < kBatchPerLaunch ? B : kBatchPerLaunch, max_blocks, Hq, H, d, bs).total;
}

cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t s) {
  CUtensorMap kmap, vmap;
  const int64_t rows = static_cast<int64_t>(a.num_blocks) * a.H * a.bs;
  cudaError_t e = encode_cache_map(&kmap, a.k_cache, rows, a.d, kGroup);
  if (e == cudaSuccess) e = encode_cache_map(&vmap, a.v_cache, rows, a.d, kGroup);
  if (e != cudaSuccess) return e;
  const int G = a.Hq / a.H;
  DecodeParams p;
  p.a = a;
  p.heads = G < 16 ? G : 16;
  p.chunks = (G + 15) / 16;
  for (int b0 = 0; b0 < a.B; b0 += kBatchPerLaunch) {
    p.b0 = b0;
    p.nb = a.B - b0 < kBatchPerLaunch ? a.B - b0 : kBatchPerLaunch;
    const DecodeLayout L = decode_layout(p.nb, a.max_blocks, a.Hq, a.H, a.d, a.bs);
    char* ws = static_cast<char*>(a.workspace);
    p.pre = reinterpret_cast<int32_t*>(ws + L.pre);
    p.ml = reinterpret_cast<float2*>(ws + L.ml);
    p.part = reinterpret_cast<float*>(ws + L.part);
    const bool wide = p.heads > 8;
    if (a.d == 64) e = wide ? launch_decode_d<64, 2, 8>(p, kmap, vmap, s) : launch_decode_d<64, 1, 8>(p, kmap, vmap, s);
    else if (a.d == 128) e = wide ? launch_decode_d<128, 2, 8>(p, kmap, vmap, s) : launch_decode_d<128, 1, 8>(p, kmap, vmap, s);
    else e = wide ? launch_decode_d<256, 2, 4>(p, kmap, vmap, s) : launch_decode_d<256, 1, 4>(p, kmap, vmap, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace gdn
