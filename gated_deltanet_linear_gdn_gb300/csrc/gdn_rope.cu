// gdn_rope.cu -- rotary positions: pairs of a head's elements turned by position x frequency, and the tables of
// frequencies that long contexts use.
//
//   (x1, x2) -> f (x1 cos a - x2 sin a, x2 cos a + x1 sin a),  a = position * w_i
//
// An angle of a far position has to be taken modulo a turn before it is rounded to fp32 (at position 10^6 an fp32 product
// is off by 0.03). So a frequency is kept as a fraction of a turn in 64 bits, w_i / (2 pi) * 2^64: position times that,
// modulo 2^64, is one integer product without rounding, its upper half the angle to 2^-32 of a turn. As an fp32 number that is off
// by up to 2^-26 of a turn (between a quarter and a half of one), what the sine's own rounding amounts to. The table is off by
// 2^-55 of a turn (it is made from doubles), at position 2^31 2^-24.
//
// Bound by memory: an element is read and written once. Sines and cosines are made once for a token, in shared memory, for all
// heads of q and k. 31,779 tokens (40 heads of 128, all of them turned) 95.5 us, 6.8 TB/s: the rate of a copy; 64 tokens 2.2 us. In
// place the same 95.5; a quarter of 18 heads of 256 36.9 us, 4.0 TB/s in pieces of 128 bytes (85.8 out of place); 64 tokens 2.0 us.
#include <math.h>

#include "gdn_internal.h"
#include "gdn_rope.cuh"

namespace gdn {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWide = 256;

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float first(float a, float b, float2 cs) { return a * cs.x - b * cs.y; }
__device__ __forceinline__ float second(float a, float b, float2 cs) { return b * cs.x + a * cs.y; }

// Rows as vectors of 16 bytes, rot_dim a multiple of 16: a CTA has one token, a thread one item of its rows: two vectors with
// eight pairs (the half layout's two halves of them, or twice four neighbours), or two that are only copied. The item's sines
// and cosines stay in registers for all of its rows (read from shared memory for each row they kept that at 91%, 123 us for
// 31,779 tokens of 40 heads of 128).
template <bool INTER>
__global__ void __launch_bounds__(kRopeWide) rope_wide_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float s_angle[];  // cosines, sines: [2][rot / 2]
  constexpr int kFlight = 3;          // rows that a thread loads at a time
  const int tid = threadIdx.x, half = a.rot / 2, eights = a.rot / 16;  // (rotated items)
  const int64_t t = blockIdx.x;
  const int at_once = blockDim.x / a.items, row0 = tid / a.items, item = tid - row0 * a.items;
  const bool turns = item < eights;
  // the item's vectors, in elements
  const int at = !turns ? item * 16 : item * 8, to = !turns ? at + 8 : at + half;
  const bool two = to < a.d;
  const int rows = row0 < at_once ? a.Hq + a.H : 0;
  const uint16_t* q = a.q + t * a.q_stride;
  const uint16_t* k = a.k + t * a.k_stride - static_cast<int64_t>(a.Hq) * a.d;
  uint4 u[kFlight], v[kFlight];
  auto load = [&](int r0) {
#pragma unroll
    for (int y = 0; y < kFlight; ++y) {
      const int r = r0 + y * at_once;
      if (r >= rows) break;
      const uint16_t* src = (r < a.Hq ? q : k) + r * a.d;
      u[y] = *reinterpret_cast<const uint4*>(src + at);
      if (two) v[y] = *reinterpret_cast<const uint4*>(src + to);
    }
  };
  const int pos = a.positions[t];
  load(row0);  // (on its way under the sines)
  if (pos < 0) return;  // a padded step's row
  for (int i = tid; i < half; i += blockDim.x) {
    const uint64_t turn = a.turns[i] * static_cast<uint32_t>(pos) + 0x80000000ull;
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
    s_angle[i] = c * a.factor;
    s_angle[half + i] = s * a.factor;
  }
  __syncthreads();
  float2 cs[8];
  if (turns) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = INTER ? (j < 4 ? item * 4 + j : (item + eights) * 4 + j - 4) : item * 8 + j;
      cs[j] = make_float2(s_angle[i], s_angle[half + i]);
    }
  }
  uint16_t* q_out = a.q_out + t * a.q_out_stride;
  uint16_t* k_out = a.k_out + t * a.k_out_stride - static_cast<int64_t>(a.Hq) * a.d;
#pragma unroll 1
  for (int r0 = row0; r0 < rows; r0 += kFlight * at_once) {
    if (r0 != row0) load(r0);
#pragma unroll
    for (int y = 0; y < kFlight; ++y) {
      const int r = r0 + y * at_once;
      if (r >= rows) break;
      uint32_t p[4] = {u[y].x, u[y].y, u[y].z, u[y].w}, w[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
      if (turns) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float pa = bf_lo(p[j]), pb = bf_hi(p[j]), wa = bf_lo(w[j]), wb = bf_hi(w[j]);
          if constexpr (INTER) {
            p[j] = pack(first(pa, pb, cs[j]), second(pa, pb, cs[j]));
            w[j] = pack(first(wa, wb, cs[4 + j]), second(wa, wb, cs[4 + j]));
          } else {
            p[j] = pack(first(pa, wa, cs[2 * j]), first(pb, wb, cs[2 * j + 1]));
            w[j] = pack(second(pa, wa, cs[2 * j]), second(pb, wb, cs[2 * j + 1]));
          }
        }
      }
      uint16_t* dst = (r < a.Hq ? q_out : k_out) + r * a.d;
      *reinterpret_cast<uint4*>(dst + at) = make_uint4(p[0], p[1], p[2], p[3]);
      if (two) *reinterpret_cast<uint4*>(dst + to) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Any sizes, strides and alignment: an item is one pair, or two elements that are only copied. A CTA has a few tokens. Two bytes at
// a time: 62 of 128 elements turned for 31,779 tokens of 40 heads 247 us (131 in place), 62 of 256 for 64 tokens of 18 heads 13 us.
template <bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float2 s_cs[];  // [tokens of the CTA][rot / 2]
  __shared__ int32_t s_pos[kRopeTokens];
  const int tid = threadIdx.x, half = a.rot / 2, rows = a.Hq + a.H;
  const int t0 = blockIdx.x * kRopeTokens, here = min(kRopeTokens, a.T - t0), total = here * rows * a.items;
  if (tid < here) s_pos[tid] = a.positions[t0 + tid];
  __syncthreads();
  for (int i = tid; i < here * half; i += kRopeThreads) {
    const int t = i / half;
    const uint64_t turn = a.turns[i - t * half] * static_cast<uint32_t>(s_pos[t]) + 0x80000000ull;
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f, &s, &c);
    s_cs[i] = make_float2(c * a.factor, s * a.factor);
  }
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < total; i += kRopeThreads) {
    // (i x the divisor is below 2^32, so the product with its reciprocal is exact; 2^32 / 1 is not a 32-bit number)
    const int row_all = a.items == 1 ? i : __umulhi(i, a.by_items), item = i - row_all * a.items;
    const int t = rows == 1 ? row_all : __umulhi(row_all, a.by_rows), row = row_all - t * rows;
    if (s_pos[t] < 0) continue;  // a padded step's row
    const bool is_k = row >= a.Hq, turns = item < half;
    const int h = is_k ? row - a.Hq : row;
    const int64_t tok = t0 + t;
    const uint16_t* src = (is_k ? a.k + tok * a.k_stride : a.q + tok * a.q_stride) + h * a.d;
    uint16_t* dst = (is_k ? a.k_out + tok * a.k_out_stride : a.q_out + tok * a.q_out_stride) + h * a.d;
    const int at = INTER || !turns ? item * 2 : item, to = INTER || !turns ? at + 1 : at + half;
    const bool two = to < a.d;
    const uint32_t u = src[at], v = two ? src[to] : 0u;
    uint32_t w = u | (v << 16);
    if (turns) {
      const float2 cs = s_cs[t * half + item];
      w = pack(first(bf_lo(u), bf_lo(v), cs), second(bf_lo(u), bf_lo(v), cs));
    }
    dst[at] = static_cast<uint16_t>(w);
    if (two) dst[to] = static_cast<uint16_t>(w >> 16);
  }
}

uint32_t reciprocal(uint32_t n) { return static_cast<uint32_t>(((uint64_t{1} << 32) + n - 1) / n); }

}  // namespace

cudaError_t launch_rope(RopeArgs a, cudaStream_t s) {
  const bool in_place = (a.Hq == 0 || (a.q_out == a.q && a.q_out_stride == a.q_stride)) &&
                        (a.H == 0 || (a.k_out == a.k && a.k_out_stride == a.k_stride));
  auto aligned = [](const void* p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0; };
  const bool wide = a.rot % 16 == 0 && a.d % 8 == 0 && aligned(a.q, a.q_stride) && aligned(a.k, a.k_stride) &&
                    aligned(a.q_out, a.q_out_stride) && aligned(a.k_out, a.k_out_stride);
  const int per = wide ? 16 : 2;
  a.items = in_place ? a.rot / per : a.rot / per + (a.d - a.rot + per - 1) / per;
  a.by_items = reciprocal(a.items);
  a.by_rows = reciprocal(a.Hq + a.H);
  const int half = a.rot / 2;
  if (wide) {
    // Threads of a token: few tokens want short turns over their heads, many want each thread to have several rows for its sines.
    // With 256, 128 and 64: 8 tokens of 136 heads of 128 2.9, 3.2, 4.8 us; 256 of 40 2.7, 2.6, 2.8 and of 136 3.9, 4.2, 5.1; 1,024 of
    // 40 5.6, 3.8, 4.0; 1,536 9.1, 6.5, 6.1; 8,192 41.5, 27.4, 27.0.
    const int threads = a.T <= kRopeFew ? kRopeWide : a.T <= kRopeMany ? 128 : 64;
    auto kern = a.interleaved ? rope_wide_kernel<true> : rope_wide_kernel<false>;
    kern<<<a.T, threads, 2 * half * sizeof(float), s>>>(a);
  } else {
    auto kern = a.interleaved ? rope_kernel<true> : rope_kernel<false>;
    kern<<<(a.T + kRopeTokens - 1) / kRopeTokens, kRopeThreads, kRopeTokens * half * sizeof(float2), s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace gdn

// ------------------------------------------------------------------------------------ C ABI

namespace {

bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1) == 0; }

constexpr double kPi = 3.14159265358979323846;

}  // namespace

extern "C" {

gdn_status gdn_rope_frequencies(int32_t rot_dim, double base, gdn_rope_scaling scaling, double factor,
                                int32_t trained_len, double* host_freqs, float* host_factor) {
  if (rot_dim <= 0 || rot_dim % 2 != 0 || !host_freqs || !host_factor) return GDN_ERR_INVALID_ARG;
  if (rot_dim > gdn::kRopeMaxDim) return GDN_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !isfinite(base)) return GDN_ERR_INVALID_ARG;
  if (scaling < GDN_ROPE_PLAIN || scaling > GDN_ROPE_YARN) return GDN_ERR_INVALID_ARG;
  if (scaling != GDN_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return GDN_ERR_INVALID_ARG;
  if (scaling == GDN_ROPE_YARN && trained_len <= 0) return GDN_ERR_INVALID_ARG;
  const int half = rot_dim / 2;
  if (scaling == GDN_ROPE_NTK && rot_dim > 2) base *= pow(factor, rot_dim / (rot_dim - 2.0));
  if (!isfinite(base)) return GDN_ERR_INVALID_ARG;  // (all but the first pair would stand still)
  *host_factor = scaling == GDN_ROPE_YARN ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
  // YARN: the (real) index of the pair that turns `turns` times over the trained length
  auto index = [&](double turns) { return rot_dim * log(trained_len / (2.0 * kPi * turns)) / (2.0 * log(base)); };
  double lo = 0.0, hi = 0.0;
  if (scaling == GDN_ROPE_YARN) {
    lo = fmax(floor(index(32.0)), 0.0);
    hi = fmin(ceil(index(1.0)), rot_dim - 1.0);
  }
  for (int i = 0; i < half; ++i) {
    double w = pow(base, -2.0 * i / rot_dim);
    if (scaling == GDN_ROPE_LINEAR) w /= factor;
    if (scaling == GDN_ROPE_YARN) {
      const double mix = fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
      w = w / factor * mix + w * (1.0 - mix);
    }
    host_freqs[i] = w;
  }
  return GDN_OK;
}

gdn_status gdn_rope_turns(const double* host_freqs, int32_t count, uint64_t* host_turns) {
  if (count <= 0 || !host_freqs || !host_turns) return GDN_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (!isfinite(host_freqs[i])) return GDN_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    const double turn = host_freqs[i] / (2.0 * kPi), part = turn - floor(turn);
    // part * 2^64, rounded; a part that rounds up to a whole turn is none
    const double scaled = part * 18446744073709551616.0;
    host_turns[i] = scaled >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(scaled);
  }
  return GDN_OK;
}

gdn_status gdn_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const int32_t* positions,
                    int32_t total_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                    int32_t rot_dim, gdn_rope_layout layout, const uint64_t* turns, float factor, void* q_out,
                    int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  if (total_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0 || num_q_heads + static_cast<int64_t>(num_kv_heads) == 0)
    return GDN_ERR_INVALID_ARG;
  if (head_dim <= 0 || rot_dim <= 0 || rot_dim % 2 != 0 || rot_dim > head_dim) return GDN_ERR_INVALID_ARG;
  if (layout != GDN_ROPE_HALVES && layout != GDN_ROPE_INTERLEAVED) return GDN_ERR_INVALID_ARG;
  if (!(factor == factor) || factor - factor != 0.0f) return GDN_ERR_INVALID_ARG;  // finite
  if (head_dim > gdn::kRopeMaxDim || num_q_heads > 1024 || num_kv_heads > 1024 || total_tokens > 0x7fffffff - gdn::kRopeTokens)
    return GDN_ERR_UNSUPPORTED;
  if (total_tokens == 0) return GDN_OK;
  if (!positions || !turns || (num_q_heads > 0 && (!q || !q_out)) || (num_kv_heads > 0 && (!k || !k_out)))
    return GDN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(positions) & 3) != 0 || (reinterpret_cast<uintptr_t>(turns) & 7) != 0 || !aligned2(q) ||
      !aligned2(k) || !aligned2(q_out) || !aligned2(k_out))
    return GDN_ERR_INVALID_ARG;
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim, k_row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (num_q_heads > 0 && (q_stride < q_row || q_out_stride < q_row)) return GDN_ERR_INVALID_ARG;
  if (num_kv_heads > 0 && (k_stride < k_row || k_out_stride < k_row)) return GDN_ERR_INVALID_ARG;
  gdn::RopeArgs a{};
  a.positions = positions;
  a.turns = turns;
  a.T = total_tokens;
  a.Hq = num_q_heads;
  a.H = num_kv_heads;
  a.d = head_dim;
  a.rot = rot_dim;
  a.interleaved = layout == GDN_ROPE_INTERLEAVED;
  a.factor = factor;
  if (num_q_heads > 0) {
    a.q = static_cast<const uint16_t*>(q);
    a.q_out = static_cast<uint16_t*>(q_out);
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
  }
  if (num_kv_heads > 0) {
    a.k = static_cast<const uint16_t*>(k);
    a.k_out = static_cast<uint16_t*>(k_out);
    a.k_stride = k_stride;
    a.k_out_stride = k_out_stride;
  }
  return gdn::launch_rope(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
