// gdn_attn4_decode.cu -- attention of single tokens over the 4-bit paged cache.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),  k_j, v_j = code * 2^(e - 127) by groups of 32 of the head
//
// Bound by memory on paper (17 / 32 bytes a value, read once), and next to that by instructions: no tensor-core operand is 4
// bits with a scale by groups of V's rows, so every code passes through registers once. 16 keys of a head of 256 (8,192
// values, 4.35 KB) are 187 clocks of an SM's share of the memory's rate, so the design counts instructions:
//   - codes become f16 pairs by one conversion of a byte (exact), straight into the operand registers of the warp-level
//     product, m16n8k16: keys (or d) on the 16-row side, query heads on the 8-column side, so that groups of up to 8 heads
//     waste nothing. A byte of K has two elements of a key, a byte of V one element of two keys: the pairs that the two
//     products' operands want.
//   - a scale is never multiplied with a value. K's enters after a group's 32 elements, on the 16 x 8 scores; V's is
//     multiplied with the probabilities, once for a group's 32 d. Both are made once for a step, four a lane, and shared.
//   - the tensor cores behind tcgen05 would want the same conversion and then a second trip through shared memory, which at
//     this rate is full: 3 bytes a value and 40 values a clock are 120 of its 128 bytes a clock. The warp-level product's
//     rate suffices: 0.5 a clock and SM, and these 16 keys are 32 of them.
// The ALU does 2 conversions a clock and SM, 128 of them for 16 keys of 256; about 540 instructions in all (K 170, V 130,
// scales 70, copies 60, softmax and the rest), 2.2 issued a clock: 240 clocks where the copies alone would take 190.
//
// A CTA of four warps takes a unit's tiles in turn, one step of each warp to a tile: 16 keys of a head of 256, 32 of 128, 64 of
// 64 (the same bytes; what a step costs besides is the same). A warp has the scores of its own keys, and then the quarter of d
// of all the tile's keys: the probabilities, as operands, and the scales of V go through shared memory. So an output is in
// registers once (a first version in which each warp had all d of its own keys needed 64 registers for it and joined four
// outputs at a unit's end: 274 us for the largest case). Two barriers a tile; the first carries the vote whether a running
// maximum moves. Copies (cp.async, a warp's own keys two tiles ahead, values one) run beside that; 16-byte pieces of a row
// change places so that no operand load has a bank twice.
//
// Queries are f16, scaled by a power of two per head so that the largest element lies in [2^14, 2^15): exact for bf16
// values down to 2^-31 of it. Probabilities x V's largest scale of the key are f16: 11 significant bits, and 2^-34 of the
// row's largest.
//
// Scales of V: with x the exponent of a score and e that of the key's largest scale of V, m is the running maximum of x + e
// and stands for 2^9; it moves when an x + e passes it by 2^5. p 2^e goes into the product, next to 2^(e_group - e), and p
// itself into the sum: 2^(kTop - e) for the row's largest, so that next to a scale of V of 2^101 or more what counts may be a
// subnormal number, which the exponential does not give. It is added by itself where such a scale has set a running maximum.
//
// Split: units of a request's own length (gdn_attn_units.cuh), joined by a second, programmatically dependent kernel in unit
// order.
//
// Measured: 256 requests of 7,000 to 8,192 tokens (16 / 2 heads of 256) 204 us, 5.2 TB/s (copies alone 158 without partial sums
// and join); 64 of 1 to 8,192 (28 / 4 of 128) 46 us; 2 of 131,071 38 us; one of 4,097 12.6 us; 128 of 4,096 (32 / 8 of 64) 91 us, 3.1
// TB/s. Groups of 16 heads (NT = 2), 64 requests of 7,000 to 8,192: 94 us at 256 (8 heads 66), 57 at 128 (41); of 32, two chunks that
// read the cache once each, 94 at 128.
#include "gdn_attn.cuh"
#include "gdn_attn_units.cuh"
#include "gdn_cache4.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kRise = 5.0f;          // log2 of what a score may pass the running maximum by
constexpr float kTop = 9.0f;           // log2 of what the running maximum stands for
// log2 of the scales of V next to which a p of the sum that is not below 2^-34 of the largest may be below 2^-126 (from 2^101 on). A
// byte behind a request's keys may set this off, too: up to 2^90 what is added is below half a step of any sum.
constexpr float kFarAbove = 90.0f;

// Small units shorten the chain that a small batch waits for, and cost a large one partial sums and the start of a pipeline;
// a unit of 256 keys of 256, 512 of 128 or 1,024 of 64 is the same 70 KB. 256 requests of about 8,000 tokens (16 / 2 heads of
// 256) 214 us in up to 24 of the smaller ones and 204 in up to 12, one of 4,097 10.9 and 12.6; 128 of 4,096 (32 / 8 of 64) 101 us
// from 512 keys on and 91 from 1,024.
template <int D>
using Units = UnitRule<D == 256 ? 8 : D == 128 ? 9 : 10, D == 256 ? 10 : 11, 12>;
static_assert(kWarps == 4 && (1 << 11) / 16 / kWarps <= 32, "a lane for each 16 of a warp's keys of a unit");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
  return r;
}
// c += a b, 16 x 16 by 16 x 8, f16 in, fp32 sums; and the first of a chain, a b
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// whether one of four bytes is 255
__device__ __forceinline__ bool has_255(uint32_t w) { return ((~w - 0x01010101u) & w & 0x80808080u) != 0; }

// whether one of four bytes is 192 or more
__device__ __forceinline__ bool has_192(uint32_t w) { return (w & (w << 1) & 0x80808080u) != 0; }

// A score is summed up times its query's power of two, up to 2^26 (elements below 2^15, codes up to 6, 256 of them). With a scale
// of K of 2^65 or more among a warp's keys, their scales are lowered by as much until that power is out again: up to 2^127 no
// score is infinite that is not so itself. (The raising stands in the branch of a request's last keys: in a branch of its own,
// or as another factor, 207 and 209 us for the largest case; here 204.5, and 205.3 before.)
constexpr float kLower = 0x1p-26f;

// Scales from four bytes each of K and of V; the largest scale of V of the first two's and of the last two's key (one key or two).
struct FourScales {
  uint32_t k[4];  // fp32 2^(e - 127)
  uint32_t v[2];  // f16 pairs 2^(e - top)
  __device__ __forceinline__ static uint32_t without_255(uint32_t w) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (((w >> 8 * j) & 255u) == 255u) w &= ~(255u << 8 * j);
    return w;
  }
  __device__ __forceinline__ void make(uint32_t kw, uint32_t vw, int top0, int top1) {
    k[0] = (kw << 23) & 0x7F800000u;
    k[1] = (kw << 15) & 0x7F800000u;
    k[2] = (kw << 7) & 0x7F800000u;
    k[3] = (kw >> 1) & 0x7F800000u;
    // 25 + e - top is the exponent field of 2^(e - top + 10), times 2^-10 (rounded to an f16 subnormal where that is one)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t add = static_cast<uint32_t>(256 + 25 - (j ? top1 : top0)) * 0x10001u;
      const uint32_t t = max_u16x2(__byte_perm(vw, 0, j ? 0x4342 : 0x4140) + add, 0x01000100u);
      v[j] = mul_f16x2((t & 0x001F001Fu) << 10, 0x14001400u);
    }
  }
  __device__ __forceinline__ void lower() {
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = __float_as_uint(__uint_as_float(k[j]) * kLower);
  }
  __device__ __forceinline__ void mark(uint32_t kw, uint32_t vw) {  // NaN for 255
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (((kw >> 8 * j) & 255u) == 255u) k[j] = 0x7FC00000u;
      if (((vw >> 8 * j) & 255u) == 255u) v[j / 2] = (v[j / 2] & (j % 2 ? 0xFFFFu : 0xFFFF0000u)) | (j % 2 ? 0x7E000000u : 0x7E00u);
    }
  }
};

template <class T, int N>
__device__ __forceinline__ void load_words(const unsigned char* p, T (&v)[N]) {
  static_assert((N == 2 || N == 4) && sizeof(T) == 4, "8 or 16 bytes");
  if constexpr (N == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    v[0] = reinterpret_cast<const T&>(u.x);
    v[1] = reinterpret_cast<const T&>(u.y);
    v[2] = reinterpret_cast<const T&>(u.z);
    v[3] = reinterpret_cast<const T&>(u.w);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = reinterpret_cast<const T&>(u.x);
    v[1] = reinterpret_cast<const T&>(u.y);
  }
}

// NT: query heads of a unit by eights, 1 or 2. A warp's step has 16 keys of a head of 256, 32 of 128, 64 of 64: the same bytes,
// and what a step costs besides is the same.
template <int D, int NT>
struct Cfg {
  static constexpr int kT = 256 / D, kStep = 16 * kT;       // 16-row tiles of a step, its keys
  static constexpr int kTileKeys = kStep * kWarps;
  static constexpr int kG = D / kGroup4;                    // groups of a head
  static constexpr int kM = D / 16 / kWarps;                // 16-row tiles of O^T a warp has
  static constexpr int kRowK = D / 2, kRowV = D;            // bytes of a key, of a key pair's values
  static constexpr int kKeys = kStep * kRowK + 2 * kStep * kG;  // a warp's keys of a tile, and the scales of its keys and values
  static constexpr int kValues = kTileKeys / 2 * kRowV;     // a tile's values
  static constexpr int kScaleK = kStep * kG * 4, kScaleV = 16 * kG * 2;  // of a warp's keys, of 16 keys' values, as the products want them
  static constexpr int kAtV = kWarps * 2 * kKeys, kAtSk = kAtV + 2 * kValues, kAtSv = kAtSk + kWarps * kScaleK, kAtP = kAtSv + kWarps * kT * kScaleV,
                       kAtQ = kAtP + kWarps * kT * NT * 256, kAtFactor = kAtQ + NT * kG * 512, kAtMax = kAtFactor + 64, kAtSum = kAtMax + kWarps * 64,
                       kAtLens = kAtSum + kWarps * 64;
  // CTAs of an SM. One more costs registers, and with them instructions that are computed again: 256 requests of about 8,000
  // tokens (D = 256, 8 heads) 204 us with 4, 213 with 5 and 216 with 3. 16 heads: 3 and 4 the same.
  static constexpr int kCtas = NT == 2 ? 3 : 4;
  static constexpr int smem_of(int nb) { return 128 + kAtLens + 4 * (nb + nb / kCoarse + 2); }
  static_assert(kKeys % 128 == 0 && kAtP % 16 == 0 && kStep * kG == 128, "alignment: a place in a row is changed by bits of the address; 4 scales a lane");
  // Where 16 bytes lie in a row, as bits of the address to change: no bank twice for eight rows' (four pairs') operand words
  // of one group.
  static __device__ __forceinline__ uint32_t swap_k(int row) { return (D == 256 ? row & 7 : D == 128 ? row >> 1 & 3 : row >> 2 & 1) << 4; }
  static __device__ __forceinline__ uint32_t swap_v(int row) { return (D == 64 ? row & 2 : 2 * (row & 3)) << 4; }
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtas) attn4_decode_kernel(const __grid_constant__ DecodeParams p, int sms) {
  using C = Cfg<D, NT>;
  using Walk = WalkOf<Units<D>>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + (-smem_addr(smem_raw) & 127u);
  __shared__ int32_t s_scan[kWarps];
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int g = lane >> 2, c = lane & 3;
  unsigned char* my_keys = smem + warp * 2 * C::kKeys;       // the warp's two stages of keys
  unsigned char* values = smem + C::kAtV;                    // the CTA's two stages of values
  unsigned char* my_k = smem + C::kAtSk + warp * C::kScaleK; // scales of the warp's keys: [key][group] fp32
  unsigned char* all_v = smem + C::kAtSv;                    // scales of the tile's values: [16 keys][pair][group], f16 pairs
  unsigned char* all_p = smem + C::kAtP;                     // the tile's probabilities as operands: [16 keys][n][lane]
  unsigned char* all_q = smem + C::kAtQ;                     // queries as operands: [n][group][lane]
  float* s_factor = reinterpret_cast<float*>(smem + C::kAtFactor);
  float* s_max = reinterpret_cast<float*>(smem + C::kAtMax);  // [head][warp]
  float* s_sum = reinterpret_cast<float*>(smem + C::kAtSum);  // [head][warp]
  int32_t* lens = reinterpret_cast<int32_t*>(smem + C::kAtLens);
  int32_t* tsum = lens + p.nb;
  constexpr int kPart = C::kG < 4 ? C::kG : 4;               // groups whose scales of K a load takes
  const int cap = a.max_blocks * a.bs, shift = 31 - __clz(a.bs), G = a.Hq / a.H;

  // where the lane's 16 bytes of a copy of 512 go: the swap of a row is that of the copy's first row and that of the row in it
  const uint32_t to_keys = smem_addr(my_keys) + lane * 16 / C::kRowK * C::kRowK + (lane * 16 % C::kRowK ^ C::swap_k(lane * 16 / C::kRowK));
  const uint32_t to_values = smem_addr(values) + warp * (C::kStep / 2 * C::kRowV) + lane * 16 / C::kRowV * C::kRowV + (lane * 16 % C::kRowV ^ C::swap_v(lane * 16 / C::kRowV));
  const uint32_t my_scales = smem_addr(my_keys) + C::kStep * C::kRowK + lane * 16;
  // the lane's words: of group 0 of key g and of key pair c, at the group of the warp's first d
  const uint32_t word_k = g * C::kRowK + (c * 4 ^ C::swap_k(g)), word_v = c * C::kRowV + ((warp * C::kM / 2 * 32) ^ C::swap_v(c)) + g * 4;

  // lengths, and tiles before every kCoarse-th request
  {
    int carry = 0, flags = 0;
    for (int at = 0; at < p.nb; at += kThreads) {
      const int b = at + tid;
      int len = b < p.nb ? a.lens[p.b0 + b] : 0;
      if (len < 0 || len > cap) flags = GDN_DEVERR_SEQLENS;
      len = min(max(len, 0), cap);
      if (b < p.nb) lens[b] = len;
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
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        carry += s_scan[w];
      }
      if (b < p.nb && b % kCoarse == 0) tsum[b / kCoarse] = before + v - own;
      __syncthreads();
    }
    if (tid == 0) tsum[(p.nb + kCoarse - 1) / kCoarse] = carry;
    if (flags && a.err && blockIdx.x == 0) atomicOr(a.err, flags);
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel may take its place

  Walk w;
  w.lens = lens;
  w.tsum = tsum;
  w.nb = p.nb;
  w.H = a.H;
  w.chunks = p.chunks;
  // A full grid's CTAs are dealt to the SMs in turn: an SM's get neighbouring shares, so that what shares are rounded to (whole
  // units) adds up to one unit an SM and not one a CTA.
  const int per_sm = gridDim.x / sms;
  w.start(per_sm * sms == static_cast<int>(gridDim.x) ? blockIdx.x % sms * per_sm + blockIdx.x / sms : blockIdx.x, gridDim.x);
  int held = -1;  // the head of q that shared memory holds
#pragma unroll 1
  for (; w.more(); w.next()) {
    const int head0 = w.h * G + w.chunk * 16, heads = min(p.heads, G - w.chunk * 16), keys = w.keys();
    const int tiles = (keys + C::kTileKeys - 1) / C::kTileKeys;
    // the row of the cache that each 16 of the warp's keys start at, one to a lane; -1: no such page, or no key
    int row = -1;
    {
      const int at = lane / C::kT * C::kTileKeys + warp * C::kStep + lane % C::kT * 16, pos = w.first() + at;
      if (at < keys) {
        const int page = a.block_table[static_cast<int64_t>(p.b0 + w.b) * a.max_blocks + (pos >> shift)];
        if (page >= 0 && page < a.num_blocks) row = ((page * a.H + w.h) << shift) + (pos & (a.bs - 1));
        else if (a.err) atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);
      }
    }
    auto row_of = [&](int t, int i) { return __shfl_sync(0xFFFFFFFFu, row, (t * C::kT + i) & 31); };  // of the tile's i-th 16
    auto fetch_keys = [&](int t) {  // of the warp, into its stage t & 1
      const uint32_t to = to_keys + (t & 1) * C::kKeys;
#pragma unroll
      for (int i = 0; i < C::kT; ++i) {
        const int from = row_of(t, i);
        if (t < tiles && from >= 0) {
          const uint8_t* k = a.k_cache + static_cast<int64_t>(from) * C::kRowK + lane * 16;
#pragma unroll
          for (int x = 0; x < D / 64; ++x) cp_async16((to ^ C::swap_k(x * (512 / C::kRowK))) + (i * (D / 64) + x) * 512, k + x * 512);
        }
      }
      const int from = row_of(t, lane % 8 / C::kG);
      if (lane < 16 && t < tiles && from >= 0)  // 16 bytes each: K's scales, V's
        cp_async16(my_scales + (t & 1) * C::kKeys, (lane < 8 ? reinterpret_cast<const uint8_t*>(a.k_scale) : reinterpret_cast<const uint8_t*>(a.v_scale)) + static_cast<int64_t>(from) * C::kG + lane % C::kG * 16);
      cp_async_commit();
    };
    auto fetch_values = [&](int t) {  // the warp's part of stage t & 1
      const uint32_t to = to_values + (t & 1) * C::kValues;
#pragma unroll
      for (int i = 0; i < C::kT; ++i) {
        const int from = row_of(t, i);
        if (t < tiles && from >= 0) {
          const uint8_t* v = a.v_cache + static_cast<int64_t>(from) * (D / 2) + lane * 16;
#pragma unroll
          for (int x = 0; x < D / 64; ++x) cp_async16((to ^ C::swap_v(x * (512 / C::kRowV))) + (i * (D / 64) + x) * 512, v + x * 512);
        }
      }
      cp_async_commit();
    };
    fetch_keys(0);
    fetch_values(0);
    fetch_keys(1);

    // queries as the second operand of K's product: for each eight heads and group, a lane's four registers
    const int wanted = w.b * a.Hq + head0;
    if (wanted != held) {
      held = wanted;
      constexpr int kLanes = D / 8, kAtOnce = kThreads / kLanes;
      for (int h0 = 0; h0 < 8 * NT; h0 += kAtOnce) {
        const int h = h0 + tid / kLanes, e = tid % kLanes;  // 8 elements of a head
        uint4 u = make_uint4(0, 0, 0, 0);
        if (h < heads)
          u = *reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(p.b0 + w.b) * a.q_stride + static_cast<int64_t>(head0 + h) * D + e * 8);
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const int field = min(max(static_cast<int>(top >> 7), 15), 254);  // 127 + exponent of the largest
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - (field - 127)) << 23);  // * 2^(14 - exponent)
        const float put = a.scale < 0.0f ? -up : up;                                                // the factor is kept positive
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_f16(__uint_as_float(x[i] << 16) * put, __uint_as_float(x[i] & 0xFFFF0000u) * put);
        if (h >= 8 * NT) continue;  // (a head of 64 takes 8 lanes, and all of them 16 heads)
        *reinterpret_cast<uint4*>(all_q + ((h / 8) * C::kG + e / 4) * 512 + ((h % 8) * 4 + e % 4) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
        // a query that is not finite makes its head NaN through its factor
        if (e == 0)
          s_factor[h] = top < 0x7F80u ? fabsf(a.scale) * kLog2e * __uint_as_float(static_cast<uint32_t>(field - 14) << 23) : __int_as_float(0x7FC00000);
      }
      __syncthreads();
    }

    float o[C::kM][NT][4], m[NT][2], l[NT][2], fac[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[n][j] = -INFINITY;
        l[n][j] = 0.0f;
        fac[n][j] = s_factor[n * 8 + 2 * c + j];
      }
#pragma unroll
    for (int t = 0; t < C::kM; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[t][n][j] = 0.0f;

    bool far = false;  // a running maximum was set next to a scale of V above 2^kFarAbove
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
      if (t == 0) cp_async_wait<2>();  // (behind the first keys: their values, the next keys; later ones came before values)
      __syncwarp();
      const unsigned char* st = my_keys + (t & 1) * C::kKeys;
      const int live = keys - t * C::kTileKeys - warp * C::kStep;  // how many of the warp's keys the request has
      // their scales, four a lane: half of a key's groups (D = 256), a key's, or two keys'
      int e_own;
      {
        const int key = D == 256 ? lane >> 1 : D == 128 ? lane : 2 * lane;
        const unsigned char* raw = st + C::kStep * C::kRowK;
        const uint32_t kw = reinterpret_cast<const uint32_t*>(raw)[lane], vw = reinterpret_cast<const uint32_t*>(raw + 128)[lane];
        const int key_live = row_of(t, key / 16) >= 0 ? live : 0;  // (a page that is none: no key)
        const bool nan = has_255(kw) | has_255(vw);
        // (of the keys that the request has: what lies behind them changes no bit)
        const bool high = __any_sync(0xFFFFFFFFu, has_192(key < key_live ? D == 64 && key + 1 >= key_live ? kw & 0xFFFFu : kw : 0u));
        FourScales sc;
        int top0, top1;
        {
          const uint32_t w = nan ? sc.without_255(vw) : vw;
          const uint32_t lo = __byte_perm(w, 0, 0x4140), hi = __byte_perm(w, 0, 0x4342);
          if constexpr (D == 64) {
            top0 = max(lo & 0xFFFFu, lo >> 16);
            top1 = max(hi & 0xFFFFu, hi >> 16);
            top1 = min(max(top1, kBias4 + kLeastScale), 253);
          } else {
            const uint32_t m = max_u16x2(lo, hi);
            top0 = max(m & 0xFFFFu, m >> 16);
            if constexpr (D == 256) top0 = max(top0, __shfl_xor_sync(0xFFFFFFFFu, top0, 1));
          }
          top0 = min(max(top0, kBias4 + kLeastScale), 253);
          if constexpr (D != 64) top1 = top0;
        }
        e_own = D == 64 ? ((top0 - kBias4) & 0xFFFF) | (top1 - kBias4) << 16 : top0 - kBias4;
        sc.make(kw, vw, top0, top1);
        if (high) sc.lower();
        if (nan) sc.mark(kw, vw);
        if (key + (D == 64) >= key_live) {
          sc.v[1] = 0;
          if (D != 64 || key >= key_live) sc.v[0] = 0;
        }
        *reinterpret_cast<uint4*>(my_k + lane * 16) = make_uint4(sc.k[0], sc.k[1], sc.k[2], sc.k[3]);  // [key][group]
        __syncwarp();
        // scores of keys 16 i + g and 16 i + g + 8, heads 2 c and 2 c + 1
        float s[C::kT][NT][4];
#pragma unroll
        for (int i = 0; i < C::kT; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][n][j] = 0.0f;
        const uint32_t keys_at = smem_addr(st) + word_k;  // (rows that are 8 apart have the same swap)
#pragma unroll
        for (int gr = 0; gr < C::kG; gr += kPart) {
          float k0[C::kT][kPart], k1[C::kT][kPart];
#pragma unroll
          for (int i = 0; i < C::kT; ++i) {
            load_words(my_k + ((16 * i + g) * C::kG + gr) * 4, k0[i]);
            load_words(my_k + ((16 * i + g + 8) * C::kG + gr) * 4, k1[i]);
          }
#pragma unroll
          for (int z = 0; z < kPart; ++z) {
            const uint32_t at = keys_at ^ (gr + z) * 16;
            uint4 q[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) q[n] = *reinterpret_cast<const uint4*>(all_q + (n * C::kG + gr + z) * 512 + lane * 16);
#pragma unroll
            for (int i = 0; i < C::kT; ++i) {
              uint32_t x[4], y[4];
              e2m1x8(lds32(at + i * 16 * C::kRowK), x);
              e2m1x8(lds32(at + (i * 16 + 8) * C::kRowK), y);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float r[4];
                mma0(r, x[0], y[0], x[1], y[1], q[n].x, q[n].y);
                mma(r, x[2], y[2], x[3], y[3], q[n].z, q[n].w);
                s[i][n][0] = fmaf(r[0], k0[i][z], s[i][n][0]);
                s[i][n][1] = fmaf(r[1], k0[i][z], s[i][n][1]);
                s[i][n][2] = fmaf(r[2], k1[i][z], s[i][n][2]);
                s[i][n][3] = fmaf(r[3], k1[i][z], s[i][n][3]);
              }
            }
          }
        }
        __syncwarp();  // the keys have been read
        fetch_keys(t + 2);
        // the largest scale of V of each of the lane's keys, as floats
        float e[C::kT][2];
#pragma unroll
        for (int i = 0; i < C::kT; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int k = 16 * i + g + 8 * j;
            int x = __shfl_sync(0xFFFFFFFFu, e_own, D == 256 ? 2 * k : D == 128 ? k : k >> 1);
            if (D == 64) x = g & 1 ? x >> 16 : static_cast<int16_t>(x);
            e[i][j] = __int_as_float(0x4B400000 + x) - 12582912.0f;
          }
        // the exponents x; their largest x + e of each head, and what that passes the running maxima by, at most
        float above = -INFINITY, most[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) most[n][j] = -INFINITY;
#pragma unroll
        for (int i = 0; i < C::kT; ++i) {
          const int seen = row_of(t, i) >= 0 ? live - 16 * i : 0;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][n][j] *= fac[n][j & 1];
          if (seen < 16 || high) {  // the request's last keys, a page that is none; scales that were lowered
            if (high) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][n][j] *= 1.0f / kLower;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (g + (j & 2) * 4 >= seen) s[i][n][j] = -INFINITY;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) most[n][j] = fmaxf(most[n][j], fmaxf(s[i][n][j] + e[i][0], s[i][n][2 + j] + e[i][1]));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) above = fmaxf(above, most[n][j] - m[n][j]);  // (-inf - -inf is left out)
        // from here on every warp is done with the tile before: its values, their scales and the probabilities are free
        if (__syncthreads_or(above > kRise)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float top = most[n][j];
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
              if (g == 0) s_max[(n * 8 + 2 * c + j) * kWarps + warp] = top;
            }
          float largest = e[0][0];
#pragma unroll
          for (int i = 0; i < C::kT; ++i) largest = max3(largest, e[i][0], e[i][1]);
          far |= __syncthreads_or(largest > kFarAbove) != 0;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float corr[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 v = *reinterpret_cast<const float4*>(s_max + (n * 8 + 2 * c + j) * kWarps);
              const float top = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
              const float to = top > m[n][j] + kRise ? top : m[n][j];  // by the head alone, whatever the others do
              const float root = to == -INFINITY ? 1.0f : ex2_root(m[n][j] - to);
              m[n][j] = to;
              l[n][j] = l[n][j] * root * root;
              corr[j] = root * root;
            }
#pragma unroll
            for (int x = 0; x < C::kM; ++x) {
              o[x][n][0] *= corr[0];
              o[x][n][1] *= corr[1];
              o[x][n][2] *= corr[0];
              o[x][n][3] *= corr[1];
            }
          }
        }
        fetch_values(t + 1);
        // p 2^e, keys' rows turned into columns, and p into the sum: from its own exponent, as p 2^e is 0 next to a scale 2^126
        // times as large
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float from[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) from[j] = m[n][j] == -INFINITY ? 0.0f : m[n][j] - kTop;
#pragma unroll
          for (int i = 0; i < C::kT; ++i) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              x[j] = ex2(s[i][n][j] + (e[i][0] - from[j]));
              x[2 + j] = ex2(s[i][n][2 + j] + (e[i][1] - from[j]));
              l[n][j] += ex2(s[i][n][j] - from[j]) + ex2(s[i][n][2 + j] - from[j]);
            }
            *reinterpret_cast<uint2*>(all_p + (((warp * C::kT + i) * NT + n) * 32 + lane) * 8) =
                make_uint2(transpose8(pack_f16(x[0], x[1])), transpose8(pack_f16(x[2], x[3])));
          }
        }
        if (far) {  // what the sum has lost below 2^-126
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float from = m[n][j] == -INFINITY ? 0.0f : m[n][j] - kTop;
#pragma unroll
              for (int i = 0; i < C::kT; ++i)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const float x = s[i][n][2 * z + j] - from;
                  if (x < -126.0f) l[n][j] += ex2(x + 64.0f) * 0x1p-64f;
                }
            }
        }
        // V's scales: keys 2 j and 2 j + 1 side by side, [j][group]. Where they are two lanes', the even key's lane writes the
        // first half of its groups, the odd one the second.
        uint32_t* put = reinterpret_cast<uint32_t*>(all_v + warp * (C::kT * C::kScaleV)) + (key >> 1) * C::kG;
        if constexpr (D == 64) {
          *reinterpret_cast<uint2*>(put) = make_uint2(__byte_perm(sc.v[0], sc.v[1], 0x5410), __byte_perm(sc.v[0], sc.v[1], 0x7632));
        } else {
          const bool odd = key & 1;
          const uint32_t mine_v = odd ? sc.v[1] : sc.v[0], got = __shfl_xor_sync(0xFFFFFFFFu, odd ? sc.v[0] : sc.v[1], D == 256 ? 2 : 1);
          const uint32_t lo = odd ? got : mine_v, hi = odd ? mine_v : got;
          *reinterpret_cast<uint2*>(put + (D == 256 ? (lane & 1) * 4 : 0) + (odd ? 2 : 0)) = make_uint2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
        }
      }
      cp_async_wait<2>();  // (behind these values: the keys of the tile after the next, the next values)
      __syncthreads();
      // O^T: the warp's d, all keys of the tile
      {
        const uint32_t values_at = smem_addr(values) + (t & 1) * C::kValues + word_v;  // (pairs c and c + 4 have the same swap)
#pragma unroll
        for (int sub = 0; sub < kWarps * C::kT; ++sub) {  // 16 keys
          uint2 pr[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) pr[n] = *reinterpret_cast<const uint2*>(all_p + ((sub * NT + n) * 32 + lane) * 8);
          const unsigned char* sv = all_v + sub * C::kScaleV + (c * C::kG + warp * C::kM / 2) * 4;
          uint32_t v0[2], v1[2];
          if constexpr (C::kM == 4) {
            load_words(sv, v0);
            load_words(sv + 4 * C::kG * 4, v1);
          } else {
            v0[0] = *reinterpret_cast<const uint32_t*>(sv);
            v1[0] = *reinterpret_cast<const uint32_t*>(sv + 4 * C::kG * 4);
          }
#pragma unroll
          for (int z = 0; z < (C::kM + 1) / 2; ++z) {
            const uint32_t at = (values_at ^ z * 32) + sub * (8 * C::kRowV);
            uint32_t lo = lds32(at), hi = lds32(at + 4 * C::kRowV);
            if constexpr (C::kM == 1) {  // half of a group
              lo >>= (warp & 1) * 16;
              hi >>= (warp & 1) * 16;
            }
            uint32_t x[4], y[4];
            e2m1x8(lo, x);
            e2m1x8(hi, y);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t b0 = mul_f16x2(pr[n].x, v0[z]), b1 = mul_f16x2(pr[n].y, v1[z]);
              mma(o[2 * z][n], x[0], x[1], y[0], y[1], b0, b1);
              if constexpr (C::kM > 1) mma(o[2 * z + 1][n], x[2], x[3], y[2], y[3], b0, b1);
            }
          }
        }
      }
    }
    cp_async_wait<0>();
    // the unit's sums, over the lanes and the warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][j] += __shfl_xor_sync(0xFFFFFFFFu, l[n][j], x);
        if (g == 0) s_sum[(n * 8 + 2 * c + j) * kWarps + warp] = l[n][j];
      }
    __syncthreads();
    const int64_t f = ((static_cast<int64_t>(w.b) * a.H + w.h) * p.chunks + w.chunk) * p.each + w.index;
    const bool alone = w.count == 1;
    uint16_t* out = a.out + (static_cast<int64_t>(p.b0 + w.b) * a.Hq + head0) * D;
    float* part = p.part + f * p.heads * D;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int h = n * 8 + 2 * c + j;
        const float4 l4 = *reinterpret_cast<const float4*>(s_sum + h * kWarps);
        const float sum = (l4.x + l4.y) + (l4.z + l4.w), inv = sum > 0.0f || sum != sum ? __fdividef(1.0f, sum) : 0.0f;
        if (h < heads) {
          if (!alone && warp == 0 && g == 0) p.ml[f * p.heads + h] = make_float2(m[n][j], sum);
          if constexpr (C::kM == 1) {  // d of the warp's half of a group: 4 g + 0 and 1, or 2 and 3
            const int d = (warp >> 1) * 32 + g * 4 + (warp & 1) * 2;
            if (alone) *reinterpret_cast<uint32_t*>(out + h * D + d) = pack_bf16(o[0][n][j] * inv, o[0][n][2 + j] * inv);
            else *reinterpret_cast<float2*>(part + h * D + d) = make_float2(o[0][n][j], o[0][n][2 + j]);
          } else {
#pragma unroll
            for (int z = 0; z < C::kM / 2; ++z) {
              const int d = (warp * C::kM / 2 + z) * 32 + g * 4;
              const float4 v = make_float4(o[2 * z][n][j], o[2 * z][n][2 + j], o[2 * z + 1][n][j], o[2 * z + 1][n][2 + j]);
              if (alone) *reinterpret_cast<uint2*>(out + h * D + d) = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
              else *reinterpret_cast<float4*>(part + h * D + d) = v;
            }
          }
        }
      }
    __syncthreads();  // sums, scales, probabilities and the last values have been read
  }
}

// Joins the units of one request, kv head and head chunk in unit order; an empty request gets zeros. The units' weights are
// made once for a head, in shared memory; a thread then has four d of a head. Up to kJoinFew units it takes in order; more are
// taken by kJoinRows4 threads, unit u by u mod kJoinRows4, whose sums are taken in order then. The whole call (16 / 2 heads of 256)
// with kJoinFew 8, 16 and 32: one request of 32,768 keys (32 units) 18.8, 18.8, 21.4 us; one of 24,000 25.1, 24.8, 26.8; 512 of up to
// 3,000 (12 units) 149, 123, 124, as eight makes a join of all requests wide.
constexpr int kJoinFew = 16, kJoinRows4 = 16;
static_assert(kJoinFew <= 32, "a lane for each unit");
constexpr int kJoinUnits = 1024;  // weights that are kept at a time

template <int D>
__global__ void __launch_bounds__(256) attn4_join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kLanes = D / 4;  // threads of a head
  __shared__ float s_w[kJoinUnits];
  __shared__ float s_red[16];
  __shared__ float4 s_o[kJoinRows4][16];
  const AttnArgs& a = p.a;
  const int HC = a.H * p.chunks, G = a.Hq / a.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / HC, hc = blockIdx.x - b * HC, h = hc / p.chunks, chunk = hc - h * p.chunks;
  const int heads = min(p.heads, G - chunk * 16);
  const int n = Units<D>::count(min(max(a.lens[p.b0 + b], 0), a.max_blocks * a.bs));
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (by every CTA: this kernel's end stands for the call's)
  if (n == 1) return;
  const int64_t f = static_cast<int64_t>(blockIdx.x) * p.each * p.heads;
  const float2* ml = p.ml + f;
  const float4* part = reinterpret_cast<const float4*>(p.part + f * D);
  uint16_t* out = a.out + (static_cast<int64_t>(p.b0 + b) * a.Hq + h * G + chunk * 16) * D;
  const int step = p.heads * kLanes;  // vectors of a unit
  // A unit's weight by its root: a sum is multiplied with it twice. (Without keys m = -inf, l = 0; with only NaN scores
  // m = -inf, l = NaN.)
  auto root_of = [](float2 e, float top) { return e.x == -INFINITY ? (e.y == 0.0f ? 0.0f : 1.0f) : ex2_root(e.x - top); };
  auto inverse = [](float l) { return l > 0.0f || l != l ? __fdividef(1.0f, l) : 0.0f; };
  auto fma4 = [](float4& o, const float4& v, float w) {
    o.x = fmaf(v.x, w, o.x);
    o.y = fmaf(v.y, w, o.y);
    o.z = fmaf(v.z, w, o.z);
    o.w = fmaf(v.w, w, o.w);
  };
  auto store = [&](int i, const float4& o, float inv) {
    *reinterpret_cast<uint2*>(out + i * 4) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  };
  if (n <= kJoinFew) {
    const int i = blockIdx.y * 256 + tid, first = blockIdx.y * (256 / kLanes);  // the block's heads
    if (first >= heads) return;
#pragma unroll
    for (int in = warp; in < 256 / kLanes; in += 8) {  // a head, a lane for each unit
      float2 e = make_float2(-INFINITY, 0.0f);
      if (first + in < heads && lane < n) e = ml[lane * p.heads + first + in];
      float top = e.x;
#pragma unroll
      for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
      const float root = root_of(e, top);
      float l = e.y * root * root;
#pragma unroll
      for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
      s_w[in * 32 + lane] = root * root;
      if (lane == 0) s_red[in] = inverse(l);
    }
    __syncthreads();
    if (i >= heads * kLanes) return;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int u = 0; u < n; ++u) fma4(o, part[static_cast<int64_t>(u) * step + i], s_w[tid / kLanes * 32 + u]);
    store(i, o, s_red[tid / kLanes]);
    return;
  }
  const int row = tid / 16, in = tid % 16;
#pragma unroll 1
  for (int i0 = blockIdx.y * 16; i0 < heads * kLanes; i0 += gridDim.y * 16) {  // 16 lanes of one head
    const float2* e = ml + i0 / kLanes;
    float top = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (int u = tid; u < n; u += 256) top = fmaxf(top, e[static_cast<int64_t>(u) * p.heads].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    if (lane == 0) s_red[warp] = top;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 8; ++x) top = fmaxf(top, s_red[x]);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int u0 = 0; u0 < n; u0 += kJoinUnits) {
      const int here = min(kJoinUnits, n - u0);
#pragma unroll 1
      for (int u = tid; u < here; u += 256) {
        const float2 x = e[static_cast<int64_t>(u0 + u) * p.heads];
        const float root = root_of(x, top);
        l += x.y * root * root;
        s_w[u] = root * root;
      }
      __syncthreads();
#pragma unroll 8
      for (int u = row; u < here; u += kJoinRows4) fma4(o, part[static_cast<int64_t>(u0 + u) * step + i0 + in], s_w[u]);
      __syncthreads();
    }
    s_o[row][in] = o;
#pragma unroll
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
    if (lane == 0) s_red[8 + warp] = l;
    __syncthreads();
    if (row == 0) {
#pragma unroll
      for (int x = 1; x < kJoinRows4; ++x) fma4(o, s_o[x][in], 1.0f);
      l = 0.0f;
#pragma unroll
      for (int x = 0; x < 8; ++x) l += s_red[8 + x];
      store(i0 + in, o, inverse(l));
    }
    __syncthreads();
  }
}

template <int D, int NT>
cudaError_t launch_d(DecodeParams& p, cudaStream_t s) {
  using C = Cfg<D, NT>;
  auto kern = attn4_decode_kernel<D, NT>;
  const int smem = C::smem_of(p.nb);
  // the same for every call: the limit is the kernel's, whichever thread sets it last
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem_of(kBatchPerLaunch));
  if (e != cudaSuccess) return e;
  int per_sm = kSmemPerSm / (smem + 256 + 1024);  // (256: what the kernel declares itself)
  if (per_sm > C::kCtas) per_sm = C::kCtas;       // (registers for as many by its launch bounds)
  if (per_sm < 1) per_sm = 1;
  const int64_t most = static_cast<int64_t>(p.nb) * p.a.H * p.chunks * p.each;
  const int grid = static_cast<int>(most < static_cast<int64_t>(per_sm) * sm_count() ? most : per_sm * sm_count());
  kern<<<grid, kThreads, smem, s>>>(p, sm_count());
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // The join, a programmatic dependent: four d of a head to a thread, or to kJoinRows4 of them where requests may have many
  // units; of those CTAs no more than fill the GPU (512 x 32, most of them for requests of few units, took 27 us, and 512 x 2 eight).
  cudaLaunchConfig_t cfg = {};
  const int pairs = p.nb * p.a.H * p.chunks, few = (p.heads * D + 1023) / 1024;
  int wide = p.heads * D / 64;
  if (wide > 16 * sm_count() / pairs) wide = 16 * sm_count() / pairs;
  cfg.gridDim = dim3(pairs, p.each > kJoinFew && wide > few ? wide : few, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn4_join_kernel<D>, p);
}

template <int D>
cudaError_t launch_all(const AttnArgs& a, cudaStream_t s) {
  const int G = a.Hq / a.H;
  DecodeParams p;
  p.a = a;
  p.fault = 0;
  p.heads = G < 16 ? G : 16;
  p.chunks = (G + 15) / 16;
  p.each = static_cast<int>(Units<D>::most(static_cast<int64_t>(a.max_blocks) * a.bs));
  const int most = attn_decode_batch(a.max_blocks, a.Hq, a.H, a.bs);  // (not 0: the caller has checked)
  const int launches = (a.B + most - 1) / most, per = (a.B + launches - 1) / launches;
  for (int b0 = 0; b0 < a.B; b0 += per) {
    p.b0 = b0;
    p.nb = a.B - b0 < per ? a.B - b0 : per;
    const DecodeLayout L = decode_layout<Units<D>>(p.nb, a.max_blocks, a.Hq, a.H, D, a.bs);
    char* ws = static_cast<char*>(a.workspace);
    p.ml = reinterpret_cast<float2*>(ws);
    p.part = reinterpret_cast<float*>(ws + L.part);
    const cudaError_t e = p.heads <= 8 ? launch_d<D, 1>(p, s) : launch_d<D, 2>(p, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t attn4_decode_workspace(int B, int max_blocks, int Hq, int H, int d, int bs) {
  const int most = attn_decode_batch(max_blocks, Hq, H, bs), nb = B < most ? B : most;
  return d == 64    ? decode_layout<Units<64>>(nb, max_blocks, Hq, H, d, bs).total
         : d == 128 ? decode_layout<Units<128>>(nb, max_blocks, Hq, H, d, bs).total
                    : decode_layout<Units<256>>(nb, max_blocks, Hq, H, d, bs).total;
}

cudaError_t launch_attn4_decode(const AttnArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_all<64>(a, s) : a.d == 128 ? launch_all<128>(a, s) : launch_all<256>(a, s);
}

}  // namespace gdn
