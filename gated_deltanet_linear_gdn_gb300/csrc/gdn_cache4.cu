// gdn_cache4.cu -- the 4-bit paged cache: its writer, its read-back, and the pages of prompts as 8-bit ones.
//
// Format. e2m1 codes (a sign and 0, 0.5, 1, 1.5, 2, 3, 4, 6) in groups of 32 along the head; a group has one byte e and its
// values are code * 2^(e - 127). A power of two for a scale makes both directions exact but for the one rounding to a code:
// value * 2^(127 - e) is exact in fp32, and code * 2^(e - 127) is a bf16 value.
//
// Writer. Per token, head and group, with a the largest |x| of the finite values: e the least with a <= 7 * 2^(e - 127), at
// least 63. (Up to 7 rounds to 6 by no more than the half step that 4 to 6 have anyway, so a limit of 6 would only make
// every group between 6 and 7 twice as coarse.) Tokens do not touch one another: nothing that was written is rounded again,
// a token may be written in any step, and the order of tokens does not matter but for the two that share V's bytes.
//
// V's bytes hold the same element of two neighbouring tokens, so that the attention's product over tokens finds its operand
// pairs as they lie. The token with the even slot writes for both where the next one follows it in the call; a token alone
// keeps its neighbour's half.
//
// Bound by memory, 2 bytes read and 17 / 32 written a value (the read-back the other way round).
#include "gdn_cache4.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// The byte of a group's scale, from the eight bf16 values that each of the group's four lanes has.
__device__ __forceinline__ uint32_t group_byte(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t top = 0, nan = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;  // |x| orders like its bits, from 0x7F80 on not finite
    top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    nan |= (lo > 0x7F80u) | (hi > 0x7F80u);
  }
  uint32_t m = top | (nan << 16);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const uint32_t n = __shfl_xor_sync(0xFFFFFFFFu, m, o);
    m = max(m & 0xFFFFu, n & 0xFFFFu) | ((m | n) & 0x10000u);
  }
  if (m >> 16) return kNaN4;
  // top = 2^(E - 127) * (1 + M / 128) <= 1.75 * 2^2 * 2^(e - 127)
  const int e = static_cast<int>(m >> 7) - 2 + ((m & 127u) > 96u);
  return max(e, kLeastByte4);
}
// 2^(127 - byte), which a value is multiplied with (of a group with NaN, anything: its codes mean nothing)
__device__ __forceinline__ float down_by(uint32_t byte) { return __uint_as_float((254u - min(byte, 253u)) << 23); }

__device__ __forceinline__ void scaled(const uint4& u, float r, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf_lo(w[i]) * r;
    f[2 * i + 1] = bf_hi(w[i]) * r;
  }
}

// Four bits each of two words side by side: byte i = (element i of a, element i of b).
__device__ __forceinline__ uint2 interleave(uint32_t a, uint32_t b) {
  auto spread = [](uint32_t x) {  // 16 bits: four bits to each byte
    x = (x | (x << 8)) & 0x00FF00FFu;
    return (x | (x << 4)) & 0x0F0F0F0Fu;
  };
  return make_uint2(spread(a & 0xFFFFu) | (spread(b & 0xFFFFu) << 4), spread(a >> 16) | (spread(b >> 16) << 4));
}

// grid: (tokens, keys or values). A CTA has `at_once` tokens at a time, `rounds` times; a thread has 8 elements of a head.
__global__ void __launch_bounds__(kThreads) cache4_append_kernel(const __grid_constant__ Append4Args a, int per, int at_once, int rounds) {
  const Cache4& c = a.c;
  const bool is_v = blockIdx.y != 0;
  const int lt = threadIdx.x / per, j0 = threadIdx.x - lt * per;
  const int chunks = 31 - __clz(c.d >> 3), all = c.H << chunks, groups = c.d / kGroup4;  // chunks: log2 of a head's
  const int cap = c.num_blocks * c.bs, block = 31 - __clz(c.bs);
  const uint16_t* x = is_v ? a.v : a.k;
  const int64_t stride = is_v ? a.v_stride : a.k_stride, first = static_cast<int64_t>(blockIdx.x) * at_once * rounds + lt;
  uint8_t* scales = is_v ? c.v_scale : c.k_scale;
#pragma unroll 1
  for (int j = j0; j - j0 < all; j += per) {  // (the same number of turns for all threads: per divides all, or is the CTA)
#pragma unroll 2
    for (int r = 0; r < rounds; ++r) {
      const int64_t t = first + static_cast<int64_t>(r) * at_once;
      int slot = -1, next = -1;
      bool mine = lt < at_once && t < a.T && j < all;
      if (mine) {
        slot = a.slot_map[t];
        if (slot >= cap && j == 0 && a.err && !is_v) atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);
        mine = slot >= 0 && slot < cap;
        if (mine && is_v) {
          if (slot & 1) {
            mine = !(t > 0 && a.slot_map[t - 1] == slot - 1);  // the token before writes for both
          } else if (t + 1 < a.T && a.slot_map[t + 1] == slot + 1) {
            next = slot + 1;
          }
        }
      }
      const uint16_t* src = x + t * stride + j * 8;
      uint4 u = make_uint4(0, 0, 0, 0), w = u;
      if (mine) u = *reinterpret_cast<const uint4*>(src);
      if (mine && next >= 0) w = *reinterpret_cast<const uint4*>(src + stride);
      const uint32_t byte = group_byte(u);
      float f[8];
      scaled(u, down_by(byte), f);
      const uint32_t codes = to_e2m1x8(f);
      const int h = j >> chunks, e = j - (h << chunks);  // the head, and which 8 of its elements
      const int blk = slot >> block, off = slot & (c.bs - 1);
      const int64_t of_head = static_cast<int64_t>(blk) * c.H + h;
      uint8_t* sc = scales + (of_head * c.bs + off) * groups + e / 4;
      if (!is_v) {
        if (mine) *reinterpret_cast<uint32_t*>(c.k + (of_head * c.bs + off) * (c.d / 2) + e * 4) = codes;
      } else {
        const uint32_t byte2 = group_byte(w);
        uint2* put = reinterpret_cast<uint2*>(c.v + (of_head * c.bs + off) / 2 * c.d + e * 8);
        if (mine && next >= 0) {
          scaled(w, down_by(byte2), f);
          *put = interleave(codes, to_e2m1x8(f));
          if (e % 4 == 0) sc[groups] = static_cast<uint8_t>(byte2);
        } else if (mine) {
          const uint2 was = *put, got = (slot & 1) ? interleave(0, codes) : interleave(codes, 0);
          const uint32_t keep = (slot & 1) ? 0x0F0F0F0Fu : 0xF0F0F0F0u;
          *put = make_uint2((was.x & keep) | got.x, (was.y & keep) | got.y);
        }
      }
      if (mine && e % 4 == 0) *sc = static_cast<uint8_t>(byte);
    }
  }
}

// Eight codes of a group as bf16. Every value is exact: a code has two significant bits.
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t byte) {
  // 2^(byte - 127), the least of them a subnormal
  const float s = byte == kNaN4 ? __uint_as_float(0x7FC00000u) : byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
  uint32_t h[4], o[4];
  e2m1x8(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    asm("{.reg .b16 x, y; mov.b32 {x, y}, %2; cvt.f32.f16 %0, x; cvt.f32.f16 %1, y;}" : "=f"(lo), "=f"(hi) : "r"(h[i]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(hi * s), "f"(lo * s));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(kThreads) cache4_read_kernel(const __grid_constant__ Read4Args a, int per, int at_once, int rounds) {
  const Cache4& c = a.c;
  const bool is_v = blockIdx.y != 0;
  const int lt = threadIdx.x / per, j0 = threadIdx.x - lt * per;
  const int chunks = 31 - __clz(c.d >> 3), all = c.H << chunks, groups = c.d / kGroup4;
  const int cap = c.num_blocks * c.bs, block = 31 - __clz(c.bs);
  uint16_t* x = is_v ? a.v : a.k;
  const int64_t stride = is_v ? a.v_stride : a.k_stride, first = static_cast<int64_t>(blockIdx.x) * at_once * rounds + lt;
  const uint8_t* scales = is_v ? c.v_scale : c.k_scale;
  if (lt >= at_once) return;
#pragma unroll 1
  for (int j = j0; j < all; j += per) {
    const int h = j >> chunks, e = j - (h << chunks);
#pragma unroll 4
    for (int r = 0; r < rounds; ++r) {
      const int64_t t = first + static_cast<int64_t>(r) * at_once;
      if (t >= a.T) continue;
      const int slot = a.slot_map[t];
      if (slot >= cap && j == 0 && a.err && !is_v) atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);
      if (slot < 0 || slot >= cap) continue;
      const int blk = slot >> block, off = slot & (c.bs - 1);
      const int64_t at = (static_cast<int64_t>(blk) * c.H + h) * c.bs + off;
      const uint32_t byte = scales[at * groups + e / 4];
      uint32_t codes;
      if (!is_v) {
        codes = *reinterpret_cast<const uint32_t*>(c.k + at * (c.d / 2) + e * 4);
      } else {
        const uint2 two = *reinterpret_cast<const uint2*>(c.v + at / 2 * c.d + e * 8);
        auto gather = [](uint32_t y) {  // the low four bits of each byte, side by side
          y &= 0x0F0F0F0Fu;
          y = (y | (y >> 4)) & 0x00FF00FFu;
          return (y | (y >> 8)) & 0xFFFFu;
        };
        const int up = (slot & 1) * 4;
        codes = gather(two.x >> up) | (gather(two.y >> up) << 16);
      }
      *reinterpret_cast<uint4*>(x + t * stride + j * 8) = values8(codes, byte);
    }
  }
}

// Tokens that a CTA has at a time, and how often: one round while they are few.
struct Shape {
  int per, at_once, rounds;
  dim3 grid;
};
Shape shape_of(int T, int H, int d) {
  const int all = H * d / 8;
  Shape s;
  s.per = all < kThreads ? all : kThreads;
  s.at_once = kThreads / s.per;
  const int64_t ctas = (static_cast<int64_t>(T) + s.at_once - 1) / s.at_once;
  s.rounds = ctas >= 16 * sm_count() ? 4 : 1;
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

__global__ void __launch_bounds__(kThreads) cache4_expand_kernel(const __grid_constant__ Expand4Args a) {
  extern __shared__ int32_t s_first[];  // [B + 1]: pages before each request
  __shared__ int32_t s_warp[kThreads / 32];
  __shared__ int32_t s_top[kThreads / 32];
  const Cache4& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = a.max_blocks * c.bs, block = 31 - __clz(c.bs);
  // pages of the requests that have new tokens; one that there is no room for counts as empty
  {
    int carry = 0, flags = 0;
    for (int at = 0; at < a.B; at += kThreads) {
      const int b = at + tid;
      int len = 0;
      if (b < a.B) {
        len = a.lens[b];
        if (len < 0 || len > cap) flags |= GDN_DEVERR_SEQLENS;
        len = min(max(len, 0), cap);
        if (a.cu_tokens[b + 1] <= a.cu_tokens[b]) len = 0;
      }
      const int pages = (len + c.bs - 1) >> block;
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
      const bool fits = end <= a.held;
      if (b < a.B) {
        if (!fits && pages > 0) flags |= GDN_DEVERR_BLOCKS;
        s_first[b + 1] = static_cast<int32_t>(min(end, static_cast<long long>(a.held)));
        if (blockIdx.x == 0) a.new_lens[b] = fits ? len : 0;
      }
      carry = static_cast<int32_t>(min(total, 0x3FFFFFFFll));
      __syncthreads();
    }
    if (tid == 0) s_first[0] = 0;
    __syncthreads();
    if (flags && a.err && blockIdx.x == 0) atomicOr(a.err, flags);
  }
  const int groups = c.d / kGroup4, H2 = 2 * c.H;
  const int64_t items = static_cast<int64_t>(s_first[a.B]) * H2;
#pragma unroll 1
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
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
    const int keys = min(c.bs, min(max(a.lens[b], 0), cap) - (j << block));
    const int from = a.block_table[static_cast<int64_t>(b) * a.max_blocks + j];
    const bool good = from >= 0 && from < c.num_blocks && keys > 0;
    if (hk == 0 && tid == 0) a.table[static_cast<int64_t>(b) * a.max_blocks + j] = good ? page : -1;
    if (!good) continue;
    const int64_t of_head = static_cast<int64_t>(from) * c.H + h;
    const uint8_t* sc = (is_v ? c.v_scale : c.k_scale) + of_head * c.bs * groups;
    // the page's largest scale
    int top = 0;
    for (int i = tid; i < keys * groups; i += kThreads) {
      const int e = sc[i];
      if (e != kNaN4) top = max(top, e);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = max(top, s_top[w]);
    top = max(top, 16);  // (the page's scale stays a normal number)
    const int64_t to_head = static_cast<int64_t>(page) * c.H + h;
    if (tid == 0) (is_v ? a.v_scale : a.k_scale)[to_head] = __uint_as_float(static_cast<uint32_t>(top - 6) << 23);
    uint8_t* dst = (is_v ? a.v : a.k) + to_head * c.bs * c.d;
    if (!is_v) {
      const uint4* src = reinterpret_cast<const uint4*>(c.k + of_head * c.bs * (c.d / 2));
      for (int i = tid; i < c.bs * groups; i += kThreads) {  // a group
        uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (i < keys * groups) {
          const uint4 u = src[i];
          const uint32_t s = f16_scale(sc[i], top) * 0x10001u, w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t y[4];
            e2m1x8(w[x], y);
            o[2 * x] = mul_e4m3(y[0], s) | (mul_e4m3(y[1], s) << 16);
            o[2 * x + 1] = mul_e4m3(y[2], s) | (mul_e4m3(y[3], s) << 16);
          }
        }
        uint4* put = reinterpret_cast<uint4*>(dst + i * kGroup4);
        put[0] = make_uint4(o[0], o[1], o[2], o[3]);
        put[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(c.v + of_head * c.bs / 2 * c.d);
      const int vectors = 27 - __clz(c.d);  // log2 of the 16-byte vectors of a pair of tokens, d bytes
      for (int i = tid; i < (c.bs / 2) << vectors; i += kThreads) {  // 16 elements of two tokens
        const int pair = i >> vectors, x0 = (i - (pair << vectors)) * 16, t = 2 * pair;
        uint32_t even[4] = {0, 0, 0, 0}, odd[4] = {0, 0, 0, 0};
        if (t < keys) {
          const uint4 u = src[i];
          const uint32_t s = f16_scale(sc[t * groups + x0 / kGroup4], top) |
                             (t + 1 < keys ? f16_scale(sc[(t + 1) * groups + x0 / kGroup4], top) << 16 : 0u);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t y[4];
            e2m1x8(w[x], y);  // (even token, odd token) of four elements
            uint32_t z[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) z[q] = mul_e4m3(y[q], s);
            const uint32_t p = z[0] | (z[1] << 16), q = z[2] | (z[3] << 16);
            even[x] = __byte_perm(p, q, 0x6420);
            odd[x] = __byte_perm(p, q, 0x7531);
          }
        }
        *reinterpret_cast<uint4*>(dst + t * c.d + x0) = make_uint4(even[0], even[1], even[2], even[3]);
        *reinterpret_cast<uint4*>(dst + (t + 1) * c.d + x0) = make_uint4(odd[0], odd[1], odd[2], odd[3]);
      }
    }
    __syncthreads();  // s_top is written anew
  }
}

}  // namespace

cudaError_t launch_cache4_append(const Append4Args& a, cudaStream_t s) {
  const Shape sh = shape_of(a.T, a.c.H, a.c.d);
  cache4_append_kernel<<<sh.grid, kThreads, 0, s>>>(a, sh.per, sh.at_once, sh.rounds);
  return cudaGetLastError();
}

cudaError_t launch_cache4_read(const Read4Args& a, cudaStream_t s) {
  const Shape sh = shape_of(a.T, a.c.H, a.c.d);
  cache4_read_kernel<<<sh.grid, kThreads, 0, s>>>(a, sh.per, sh.at_once, sh.rounds);
  return cudaGetLastError();
}

cudaError_t launch_cache4_expand(const Expand4Args& a, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(a.held) * a.c.H * 2, most = 8 * static_cast<int64_t>(sm_count());
  const int grid = static_cast<int>(items < most ? items : most);
  cache4_expand_kernel<<<grid, kThreads, (a.B + 1) * sizeof(int32_t), s>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn
