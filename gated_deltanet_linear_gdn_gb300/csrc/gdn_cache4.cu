// gdn_cache4.cu -- the 4-bit paged cache: its writer, its read-back, and the pages of prompts as 8-bit ones.
//
// Format. e2m1 codes (a sign and 0, 0.5, 1, 1.5, 2, 3, 4, 6) in groups of 32 along the head; a group has one byte e and its
// values are code * 2^(e - 127). A power of two for a scale makes both directions exact but for the one rounding to a code:
// value * 2^(127 - e) is exact in fp32, and code * 2^(e - 127) a bf16 value, but for 2^128 and above: what is larger than
// 1.75 * 2^127 (byte 253, code 4) and the codes of a foreign cache's 253 and 254 read back infinite.
//
// Writer. Per token, head and group, with a the largest |x| of the finite values: e the least with a <= 7 * 2^(e - 127), at
// least 63. (Up to 7 rounds to 6 by no more than the half step that 4 to 6 have anyway, so a limit of 6 would only make
// every group between 6 and 7 twice as coarse.) Tokens do not touch one another: nothing that was written is rounded again,
// a token may be written in any step, and the order of a call's tokens does not matter.
//
// V's bytes hold the same element of two neighbouring tokens, so that the attention's product over tokens finds its operand
// pairs as they lie. The token with the even slot writes for both where the next one follows it in the call; a token alone
// changes its half of the bytes by atomics (each bit has one writer, so the result has no order).
//
// Bound by memory, 2 bytes read and 17 / 32 written a value (the read-back the other way round); next to that the read-back by
// instructions (181 to a thread's 16 values, 2.9 issued a clock, the ALU at 59%), the writer by waiting for its loads (164, 2.1 a
// clock, the ALU at 52%). 131,071 tokens (2 heads of 256) read back in 58 us, 5.9 TB/s (61 with three CTAs an SM, of 67
// registers); 26,734 tokens of prompts (8 heads of 128, 139 MB) written in 30 us, 4.7 TB/s, and read back in 27; 256 single
// tokens 2.1 and 2.4 us.
#include "gdn_attn.cuh"
#include "gdn_cache4.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// 16 elements of a token's head, as a thread has them: two lanes make a group.
struct Sixteen {
  uint4 a, b;
  __device__ __forceinline__ void load(const uint16_t* p) {
    a = *reinterpret_cast<const uint4*>(p);
    b = *reinterpret_cast<const uint4*>(p + 8);
  }
  __device__ __forceinline__ void word(int i, uint32_t& w) const { w = i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w; }
  // The byte of the group's scale. |x| orders like its bits, two at a time; from 0x7F80 on it is not finite.
  __device__ __forceinline__ uint32_t group_byte() const {
    uint32_t m = 0, w;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      word(i, w);
      asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w & 0x7FFF7FFFu));
    }
    m = max(m & 0xFFFFu, m >> 16);
    uint32_t all = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    if (__any_sync(0xFFFFFFFFu, all >= 0x7F80u)) {  // an infinity or NaN: once more over the finite values
      if (m >= 0x7F80u) {
        const bool nan = m > 0x7F80u;
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          word(i, w);
          const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
          m = max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
        }
        if (nan) m = 0xFFFFu;
      }
      all = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      if (all == 0xFFFFu) return kNaN4;
    }
    // the largest = 2^(E - 127) * (1 + M / 128) <= 1.75 * 2^2 * 2^(e - 127)
    const int e = static_cast<int>(all >> 7) - 2 + ((all & 127u) > 96u);
    return max(e, kLeastByte4);
  }
  // values 8 i .. 8 i + 7 times r
  __device__ __forceinline__ void scaled(int i, float r, float (&f)[8]) const {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t w;
      word(4 * i + x, w);
      const float2 v = mul2(make_float2(bf_lo(w), bf_hi(w)), make_float2(r, r));
      f[2 * x] = v.x;
      f[2 * x + 1] = v.y;
    }
  }
};
// 2^(127 - byte), which a value is multiplied with (of a group with NaN, anything: its codes mean nothing)
__device__ __forceinline__ float down_by(uint32_t byte) { return __uint_as_float((254u - min(byte, 253u)) << 23); }

// Rows of the cache, (block, head, offset), are fewer than 2^31: everything but the address itself is in 32 bits.
struct Rows {
  uint32_t of_block, of_head;  // rows of a block; the head's first one in it
  int shift, mask;
  __device__ __forceinline__ Rows(const Cache4& c, int h) {
    of_block = c.H * c.bs;
    of_head = h * c.bs;
    shift = 31 - __clz(c.bs);
    mask = c.bs - 1;
  }
  __device__ __forceinline__ uint32_t of(int slot) const { return static_cast<uint32_t>(slot >> shift) * of_block + static_cast<uint32_t>(slot & mask) + of_head; }
};
__device__ __forceinline__ uint64_t wide(uint32_t a, uint32_t b) { return static_cast<uint64_t>(a) * b; }

// grid: (tokens, keys or values). A CTA has `at_once` tokens, or of a long call (N = 2) twice as many: of keys each thread has two
// that are at_once apart, of values two neighbours. A thread has 16 elements of a head.
// (Four CTAs an SM, 64 registers: with the 70 that the compiler takes by itself, 26,734 tokens of 8 heads of 128 written and read
// back took 62.6 us instead of 58.0.)
template <int N>
__global__ void __launch_bounds__(kThreads, 4) cache4_append_kernel(const __grid_constant__ Append4Args a, int per, int at_once) {
  const Cache4& c = a.c;
  const int lt = threadIdx.x / per, j0 = threadIdx.x - lt * per;
  const int sixteens = 27 - __clz(c.d), all = c.H << sixteens, groups = c.d / kGroup4;  // (log2 of a head's sixteens)
  const int cap = c.num_blocks * c.bs;
  // (below: the same number of turns of every loop for all threads, as lanes exchange their groups' maxima)
  if (blockIdx.y == 0) {
    const int64_t first = static_cast<int64_t>(blockIdx.x) * at_once * N + lt;
#pragma unroll 1
    for (int j = j0; j - j0 < all; j += per) {
      const int h = j >> sixteens, e = j - (h << sixteens);  // the head, and which 16 of it
      const Rows rows(c, h);
      int slot[N];
      Sixteen u[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t t = first + static_cast<int64_t>(i) * at_once;
        slot[i] = lt < at_once && t < a.T && j < all ? a.slot_map[t] : -1;
        if (slot[i] >= cap) {
          if (j == 0 && a.err) atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);
          slot[i] = -1;
        }
        u[i].a = u[i].b = make_uint4(0, 0, 0, 0);
        if (slot[i] >= 0) u[i].load(a.k + t * a.k_stride + j * 16);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t byte = u[i].group_byte(), row = rows.of(slot[i]);
        const float down = down_by(byte);
        float f[8];
        uint2 codes;
        u[i].scaled(0, down, f);
        codes.x = to_e2m1x8(f);
        u[i].scaled(1, down, f);
        codes.y = to_e2m1x8(f);
        if (slot[i] >= 0) {
          *reinterpret_cast<uint2*>(c.k + wide(row, c.d / 2) + e * 8) = codes;
          if (e % 2 == 0) c.k_scale[wide(row, groups) + e / 2] = static_cast<uint8_t>(byte);
        }
      }
    }
    return;
  }
  const int64_t t = N * (static_cast<int64_t>(blockIdx.x) * at_once + lt);
  auto slot_at = [&](int64_t t) {
    const int s = t >= 0 && t < a.T ? a.slot_map[t] : -1;
    return s < cap ? s : -1;
  };
#pragma unroll 1
  for (int j = j0; j - j0 < all; j += per) {
    const int h = j >> sixteens, e = j - (h << sixteens);
    const Rows rows(c, h);
    // Writes token t, at `slot` (negative: nothing), and the next one with it where that is the pair's other half.
    auto put = [&](int slot, bool pair, const Sixteen& u, const Sixteen& w) {
      const uint32_t row = rows.of(slot), byte = u.group_byte(), byte2 = w.group_byte();
      const float down = down_by(byte);
      uint8_t* sc = c.v_scale + wide(row, groups) + e / 2;
      uint4* to = reinterpret_cast<uint4*>(c.v + wide(row / 2, c.d) + e * 16);
      float f[8], y[8];
      uint32_t codes[4];
      if (pair) {
        const float down2 = down_by(byte2);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          u.scaled(z, down, f);
          w.scaled(z, down2, y);
          codes[2 * z] = to_e2m1x8({f[0], y[0], f[1], y[1], f[2], y[2], f[3], y[3]});
          codes[2 * z + 1] = to_e2m1x8({f[4], y[4], f[5], y[5], f[6], y[6], f[7], y[7]});
        }
        *to = make_uint4(codes[0], codes[1], codes[2], codes[3]);
        if (e % 2 == 0) sc[groups] = static_cast<uint8_t>(byte2);
      } else if (slot >= 0) {
        const uint32_t own = (slot & 1) ? 0xF0F0F0F0u : 0x0F0F0F0Fu;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          u.scaled(z, down, f);
          codes[2 * z] = to_e2m1x8({f[0], f[0], f[1], f[1], f[2], f[2], f[3], f[3]});
          codes[2 * z + 1] = to_e2m1x8({f[4], f[4], f[5], f[5], f[6], f[6], f[7], f[7]});
        }
        // (atomics: the neighbour may be written by another thread of this call, where the two do not follow each other)
        uint32_t* word = reinterpret_cast<uint32_t*>(to);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          atomicAnd(word + z, ~own);
          atomicOr(word + z, codes[z] & own);
        }
      }
      if (slot >= 0 && e % 2 == 0) *sc = static_cast<uint8_t>(byte);
    };
    // of two tokens that follow each other in a run one writes: the one at an even slot, for the next one, too; the other is
    // written by it or by the thread before
    int slot0 = -1, slot1 = -1;
    bool pair0 = false, pair1 = false;
    if (lt < at_once && t < a.T && j < all) {
      const int before = slot_at(t - 1), s0 = slot_at(t), s1 = slot_at(t + 1), after = N == 2 ? slot_at(t + 2) : -1;
      slot0 = (s0 & 1) && before == s0 - 1 ? -1 : s0;
      slot1 = N == 1 || ((s1 & 1) && s0 == s1 - 1) ? -1 : s1;
      pair0 = slot0 >= 0 && !(s0 & 1) && s1 == s0 + 1;
      pair1 = slot1 >= 0 && !(s1 & 1) && after == s1 + 1;
    }
    const uint16_t* src = a.v + t * a.v_stride + j * 16;
    Sixteen u, w;
    auto load = [&](const uint16_t* p, bool one, bool two) {
      u.a = u.b = w.a = w.b = make_uint4(0, 0, 0, 0);
      if (one) u.load(p);
      if (two) w.load(p + a.v_stride);
    };
    const bool first0 = slot0 >= 0, both = first0 && slot1 >= 0;  // (both: tokens of no run, or of two)
    load(first0 ? src : src + a.v_stride, first0 || slot1 >= 0, first0 ? pair0 : pair1);
    put(first0 ? slot0 : slot1, first0 ? pair0 : pair1, u, w);
    if (__any_sync(0xFFFFFFFFu, both)) {
      load(src + a.v_stride, both, both && pair1);
      put(both ? slot1 : -1, both && pair1, u, w);
    }
  }
}

// Eight values (f16 pairs) times 2^(byte - 127) as bf16. Exact: a code has two significant bits.
__device__ __forceinline__ uint4 scaled_bf16(const uint32_t (&h)[4], float s) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    asm("{.reg .b16 x, y; mov.b32 {x, y}, %2; cvt.f32.f16 %0, x; cvt.f32.f16 %1, y;}" : "=f"(lo), "=f"(hi) : "r"(h[i]));
    const float2 v = mul2(make_float2(lo, hi), make_float2(s, s));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(v.y), "f"(v.x));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// 2^(byte - 127), the least of them a subnormal
__device__ __forceinline__ float group_scale(uint32_t byte) {
  return __uint_as_float(byte == kNaN4 ? 0x7FC00000u : byte == 0 ? 0x00400000u : byte << 23);
}

__global__ void __launch_bounds__(kThreads, 4) cache4_read_kernel(const __grid_constant__ Read4Args a, int per, int at_once, int rounds) {
  const Cache4& c = a.c;
  const bool is_v = blockIdx.y != 0;
  const int lt = threadIdx.x / per, j0 = threadIdx.x - lt * per;
  const int sixteens = 27 - __clz(c.d), all = c.H << sixteens, groups = c.d / kGroup4;
  const int cap = c.num_blocks * c.bs;
  uint16_t* x = is_v ? a.v : a.k;
  const int64_t stride = is_v ? a.v_stride : a.k_stride, first = static_cast<int64_t>(blockIdx.x) * at_once * rounds + lt;
  const uint8_t* scales = is_v ? c.v_scale : c.k_scale;
  if (lt >= at_once) return;
  // a thread has two eights of a head, half a head apart: what a warp stores at a time is in one piece
  constexpr int kFlight = 4;
#pragma unroll 1
  for (int j = j0; j < all; j += per) {
    const int h = j >> sixteens, e = j - (h << sixteens);  // the head, and which eight of its first half
    const Rows rows(c, h);
    const uint8_t* codes = is_v ? c.v + e * 8 : c.k + e * 4;
    uint16_t* out = x + first * stride + h * c.d + e * 8;
    int slot[kFlight], next[kFlight];
    auto look = [&](int r0) {
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int64_t t = first + static_cast<int64_t>(r0 + i) * at_once;
        next[i] = r0 + i < rounds && t < a.T ? a.slot_map[t] : -1;
      }
    };
    look(0);
#pragma unroll 1
    for (int r0 = 0; r0 < rounds; r0 += kFlight) {
      uint32_t byte[kFlight][2];
      uint2 raw[kFlight][2];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        slot[i] = next[i];
        if (slot[i] >= cap) {
          if (j == 0 && a.err && !is_v) atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);
          slot[i] = -1;
        }
        if (slot[i] < 0) continue;
        const uint32_t row = rows.of(slot[i]);
        const uint8_t* sc = scales + wide(row, groups) + e / 4;
        byte[i][0] = sc[0];
        byte[i][1] = sc[groups / 2];
        if (is_v) {
          const uint8_t* v = codes + wide(row / 2, c.d);
          raw[i][0] = *reinterpret_cast<const uint2*>(v);
          raw[i][1] = *reinterpret_cast<const uint2*>(v + c.d / 2);
        } else {
          const uint8_t* k = codes + wide(row, c.d / 2);
          raw[i][0].x = *reinterpret_cast<const uint32_t*>(k);
          raw[i][1].x = *reinterpret_cast<const uint32_t*>(k + c.d / 4);
        }
      }
      look(r0 + kFlight);  // (on its way under what follows)
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        if (slot[i] < 0) continue;
        uint16_t* to = out + static_cast<int64_t>((r0 + i) * at_once) * stride;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          uint32_t f[4];
          if (is_v) {  // of each byte the half of the slot's token
            const uint32_t pick = (slot[i] & 1) ? 0x7632u : 0x5410u;
            uint32_t y[4];
            e2m1x8(raw[i][z].x, y);
            f[0] = __byte_perm(y[0], y[1], pick);
            f[1] = __byte_perm(y[2], y[3], pick);
            e2m1x8(raw[i][z].y, y);
            f[2] = __byte_perm(y[0], y[1], pick);
            f[3] = __byte_perm(y[2], y[3], pick);
          } else {
            e2m1x8(raw[i][z].x, f);
          }
          *reinterpret_cast<uint4*>(to + z * (c.d / 2)) = scaled_bf16(f, group_scale(byte[i][z]));
        }
      }
    }
  }
}

// Tokens that a CTA has at a time, and how often, by the CTAs an SM that one round would make: more loads in flight a thread
// against fewer CTAs. Measured (8 heads of 128, 4 tokens a CTA; read back in 1, 2, 4, 8 rounds): 256 tokens 2.5, 2.7, 3.2, 4.9 us;
// 1,024 (1.7 CTAs an SM) 3.6, 3.1, 3.3, 4.8; 3,500 (5.8) 7.7, 5.7, 4.7, 6.1; 14,000 (23) 28.3, 19.4, 15.4, 16.5; 26,734 (44) 52.3,
// 35.2, 27.4, 26.5. Written in 1 and 2: 256 tokens 2.1, 2.3; 1,024 2.8, 2.6; 26,734 42.0, 30.0. 2 heads of 64 and of 256 turn at
// the same counts of CTAs.
struct Shape {
  int per, at_once, rounds;
  dim3 grid;
};
Shape shape_of(int T, int H, int d, int most) {
  const int all = H * d / 16;
  Shape s;
  s.per = all < kThreads ? all : kThreads;
  s.at_once = kThreads / s.per;
  const int64_t ctas = (static_cast<int64_t>(T) + s.at_once - 1) / s.at_once;
  const int64_t sms = sm_count();
  const int rounds = ctas <= sms ? 1 : ctas <= 3 * sms ? 2 : ctas < 32 * sms ? 4 : 8;
  s.rounds = rounds < most ? rounds : most;
  s.grid = dim3(static_cast<unsigned>((ctas + s.rounds - 1) / s.rounds), 2);
  return s;
}

// ------------------------------------------------------------------------ pages of prompts, in 8 bits
//
// The prompt attention multiplies e4m3 tiles with one scale to a page and head, so that its operands go from memory to the
// tensor cores untouched. A page of 4-bit values is such a tile almost without a rounding: with 2^m the page's largest scale
// a value is code * 2^(e - m + 6) times 2^(m - 6), at most 6 * 64 = 384, and exact in e4m3 down to groups of 2^-14 times the
// page's largest; below that it is rounded to 2^-9, 2^-18 of the page's largest value. A page is read once (17 / 32 bytes a
// value) and written once (1 byte); the products that follow are the call's time.

// An f16 pair times an f16 pair, as two e4m3 bytes.
__device__ __forceinline__ uint32_t mul_e4m3(uint32_t h, uint32_t s) {
  uint32_t r;
  asm("{.reg .b32 x; .reg .b16 y; mul.rn.f16x2 x, %1, %2; cvt.rn.satfinite.e4m3x2.f16x2 y, x; mov.b32 %0, {y, 0};}"
      : "=r"(r)
      : "r"(h), "r"(s));
  return r;
}
// 2^(6 + d) as f16 bits for d <= 0 (below 2^-14, where every code is below half of e4m3's least value: 0)
__device__ __forceinline__ uint32_t f16_scale(int byte, int top) {
  if (byte == kNaN4) return 0x7E00u;
  const int e = 21 + byte - top;
  return e > 0 ? static_cast<uint32_t>(e) << 10 : 0u;
}

// An item is a page's keys or values of one head; a team of TS warps has it.
template <int TS>
__global__ void __launch_bounds__(kThreads, 4) cache4_expand_kernel(const __grid_constant__ Expand4Args a) {
  extern __shared__ int32_t s_first[];  // [B + 1]: pages before each request
  __shared__ int32_t s_warp[kThreads / 32];
  __shared__ int32_t s_top[kThreads / 32];
  constexpr int kTeams = kThreads / 32 / TS, kLanes = 32 * TS;
  const Cache4& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, team = warp / TS, in = tid - team * kLanes;
  const int cap = a.max_blocks * c.bs, block = 31 - __clz(c.bs);
  // pages of the requests that have new tokens, in a range of rows that there is (the attention takes no others). One that there is
  // no room for gets a table of no pages, as those behind it
  auto pages_of = [&](int b) {
    const int len = min(max(a.lens[b], 0), cap), from = a.cu_tokens[b], to = a.cu_tokens[b + 1];
    return from >= 0 && to > from && to <= a.T ? (len + c.bs - 1) >> block : 0;
  };
  {
    int carry = 0;
    bool refused = false;
    for (int at = 0; at < a.B; at += kThreads) {
      const int b = at + tid, pages = b < a.B ? pages_of(b) : 0;
      long long v = pages;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += y;
      }
      // (saturated: what is past `held` is refused, whatever it is)
      if (lane == 31) s_warp[warp] = static_cast<int32_t>(min(v, 0x3FFFFFFFll));
      __syncthreads();
      long long before = carry, total = carry;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
      }
      const long long end = before + v;
      if (b < a.B) {
        refused |= pages > 0 && end > a.held;
        s_first[b + 1] = static_cast<int32_t>(min(end, static_cast<long long>(a.held)));
      }
      carry = static_cast<int32_t>(min(total, 0x3FFFFFFFll));
      __syncthreads();
    }
    if (tid == 0) s_first[0] = 0;
    __syncthreads();
    if (refused && a.err && blockIdx.x == 0) atomicOr(a.err, GDN_DEVERR_BLOCKS);
  }
  auto fits = [&](int b, int pages) { return s_first[b + 1] - s_first[b] == pages; };
#pragma unroll 1
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int pages = pages_of(b);
    if (fits(b, pages)) continue;
    for (int j = tid; j < pages; j += kThreads) a.table[static_cast<int64_t>(b) * a.max_blocks + j] = -1;
  }
  const int groups = c.d / kGroup4, H2 = 2 * c.H;
  const int64_t items = static_cast<int64_t>(s_first[a.B]) * H2;
#pragma unroll 1
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kTeams + team; item < items; item += static_cast<int64_t>(gridDim.x) * kTeams) {
    const int page = static_cast<int>(item / H2), hk = static_cast<int>(item - static_cast<int64_t>(page) * H2);
    const bool is_v = hk >= c.H;
    const int h = is_v ? hk - c.H : hk;
    int lo = 0, hi = a.B - 1;  // the last request that starts at or before the page
#pragma unroll 1
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_first[mid] <= page) lo = mid; else hi = mid - 1;
    }
    const int b = lo, j = page - s_first[b];
    if (!fits(b, pages_of(b))) continue;
    const int keys = min(c.bs, min(max(a.lens[b], 0), cap) - (j << block));
    const int from = a.block_table[static_cast<int64_t>(b) * a.max_blocks + j];
    const bool good = from >= 0 && from < c.num_blocks && keys > 0;
    if (hk == 0 && in == 0) a.table[static_cast<int64_t>(b) * a.max_blocks + j] = good ? page : -1;
    if (!good) continue;
    const int64_t of_head = static_cast<int64_t>(from) * c.H + h, to_head = static_cast<int64_t>(page) * c.H + h;
    const uint8_t* sc = (is_v ? c.v_scale : c.k_scale) + of_head * c.bs * groups;
    uint8_t* dst = (is_v ? a.v : a.k) + to_head * c.bs * c.d;
    // the team's part in registers, 128 values a lane, between the largest scale and the conversion
    auto page_top = [&](int top) {
      top = __reduce_max_sync(0xFFFFFFFFu, top);
      if constexpr (TS > 1) {
        if (lane == 0) s_top[warp] = top;
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + team), "n"(kLanes) : "memory");
#pragma unroll
        for (int w = 0; w < TS; ++w) top = max(top, s_top[team * TS + w]);
      }
      // K's scale of the page stays a normal number, V's what the attention takes as it is: of smaller values, 2^-99 and its
      // multiples remain
      top = max(top, is_v ? kBias4 + 6 + kLeastScale : 16);
      if (in == 0) (is_v ? a.v_scale : a.k_scale)[to_head] = __uint_as_float(static_cast<uint32_t>(top - 6) << 23);
      return top;
    };
    auto finite = [](int e) { return e == kNaN4 ? 0 : e; };
    if (!is_v) {
      const uint2* src = reinterpret_cast<const uint2*>(c.k + of_head * c.bs * (c.d / 2));
      const int live = keys * groups * 2;  // half groups
      uint2 u[8];
      int byte[8], top = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int i = in + q * kLanes;
        u[q] = make_uint2(0, 0);
        byte[q] = 0;
        if (i < live) {
          u[q] = src[i];
          byte[q] = sc[i / 2];
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) top = max(top, finite(byte[q]));
      top = page_top(top);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int i = in + q * kLanes;
        if (i >= c.bs * groups * 2) break;
        const uint32_t s = f16_scale(byte[q], top) * 0x10001u;
        uint32_t y[4], o[4];
        e2m1x8(u[q].x, y);
        o[0] = mul_e4m3(y[0], s) | (mul_e4m3(y[1], s) << 16);
        o[1] = mul_e4m3(y[2], s) | (mul_e4m3(y[3], s) << 16);
        e2m1x8(u[q].y, y);
        o[2] = mul_e4m3(y[0], s) | (mul_e4m3(y[1], s) << 16);
        o[3] = mul_e4m3(y[2], s) | (mul_e4m3(y[3], s) << 16);
        *reinterpret_cast<uint4*>(dst + i * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(c.v + of_head * c.bs / 2 * c.d);
      const int vectors = 27 - __clz(c.d);  // log2 of the 16-byte vectors of a pair of tokens, d bytes
      uint4 u[4];
      int even_byte[4], odd_byte[4], top = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = in + q * kLanes, pair = i >> vectors, group = (i - (pair << vectors)) / 2, t = 2 * pair;
        u[q] = make_uint4(0, 0, 0, 0);
        even_byte[q] = odd_byte[q] = 0;
        if (t < keys) {
          u[q] = src[i];
          even_byte[q] = sc[t * groups + group];
          if (t + 1 < keys) odd_byte[q] = sc[(t + 1) * groups + group];
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) top = max(top, max(finite(even_byte[q]), finite(odd_byte[q])));
      top = page_top(top);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = in + q * kLanes, pair = i >> vectors, x0 = (i - (pair << vectors)) * 16, t = 2 * pair;
        if (t >= c.bs) break;
        // (a token past the last: a scale of 0)
        const uint32_t s = (t < keys ? f16_scale(even_byte[q], top) : 0u) | (t + 1 < keys ? f16_scale(odd_byte[q], top) << 16 : 0u);
        const uint32_t w[4] = {u[q].x, u[q].y, u[q].z, u[q].w};
        uint32_t even[4], odd[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t y[4];
          e2m1x8(w[x], y);  // (even token, odd token) of four elements
          const uint32_t p = mul_e4m3(y[0], s) | (mul_e4m3(y[1], s) << 16), q2 = mul_e4m3(y[2], s) | (mul_e4m3(y[3], s) << 16);
          even[x] = __byte_perm(p, q2, 0x6420);
          odd[x] = __byte_perm(p, q2, 0x7531);
        }
        *reinterpret_cast<uint4*>(dst + t * c.d + x0) = make_uint4(even[0], even[1], even[2], even[3]);
        *reinterpret_cast<uint4*>(dst + (t + 1) * c.d + x0) = make_uint4(odd[0], odd[1], odd[2], odd[3]);
      }
    }
    if constexpr (TS > 1) asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + team), "n"(kLanes) : "memory");  // s_top is written anew
  }
  // The kernel runs beside the call's plan (it needs nothing of it), and the attention's prologue beside this one's end; that
  // this one is done stands for the plan, too.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace

cudaError_t launch_cache4_append(const Append4Args& a, cudaStream_t s) {
  const Shape sh = shape_of(a.T, a.c.H, a.c.d, 2);
  auto kern = sh.rounds == 2 ? cache4_append_kernel<2> : cache4_append_kernel<1>;
  kern<<<sh.grid, kThreads, 0, s>>>(a, sh.per, sh.at_once);
  return cudaGetLastError();
}

cudaError_t launch_cache4_read(const Read4Args& a, cudaStream_t s) {
  const Shape sh = shape_of(a.T, a.c.H, a.c.d, 8);
  cache4_read_kernel<<<sh.grid, kThreads, 0, s>>>(a, sh.per, sh.at_once, sh.rounds);
  return cudaGetLastError();
}

cudaError_t launch_cache4_expand(const Expand4Args& a, cudaStream_t s) {
  // warps of an item: one for each 4,096 values
  const int size = a.c.bs * a.c.d, ts = size >= 32768 ? 8 : size >= 16384 ? 4 : size >= 8192 ? 2 : 1, teams = kThreads / 32 / ts;
  // eight CTAs an SM, two rounds of those that fit: with four, prompts over pages of 16 (4 heads of 64, 20,000 keys) 37.4 us for 39.4
  // and 64 tokens at 131,000 (2 heads of 256) 180 for 178; with 64, 39.3 and 185
  const int64_t items = (static_cast<int64_t>(a.held) * a.c.H * 2 + teams - 1) / teams, most = 8 * static_cast<int64_t>(sm_count());
  const int grid = static_cast<int>(items < most ? items : most);
  auto kern = ts == 8 ? cache4_expand_kernel<8> : ts == 4 ? cache4_expand_kernel<4> : ts == 2 ? cache4_expand_kernel<2> : cache4_expand_kernel<1>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = (a.B + 1) * sizeof(int32_t);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace gdn
