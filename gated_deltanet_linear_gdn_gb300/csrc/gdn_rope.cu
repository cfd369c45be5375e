// gdn_rope.cu -- rotary positions: pairs of a head's elements turned by position x frequency, and the tables of
// frequencies that long contexts use.
//
//   (x1, x2) -> f (x1 cos a - x2 sin a, x2 cos a + x1 sin a),  a = position * w_i
//
// An angle of a far position has to be taken modulo a turn before it is rounded to fp32 (at position 10^6 an fp32 product
// is off by 0.03). So a frequency is kept as a fraction of a turn in 64 bits, w_i / (2 pi) * 2^64: position times that,
// modulo 2^64, is one integer product without rounding, its upper half the angle to 2^-32 of a turn. The table is off by
// 2^-55 of a turn (it is made from doubles), at position 2^31 2^-24.
//
// Bound by memory: an element is read and written once. A CTA takes a few tokens: it makes their sines and cosines once, in
// shared memory, for all heads of q and k.
#include <math.h>

#include "gdn_internal.h"
#include "gdn_rope.cuh"

namespace gdn {

namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float first(float a, float b, float2 cs) { return a * cs.x - b * cs.y; }
__device__ __forceinline__ float second(float a, float b, float2 cs) { return b * cs.x + a * cs.y; }

// WIDE: rot_dim is a multiple of 16 and rows are vectors of 16 bytes: an item is two vectors (8 pairs in the half layout,
// twice 4 neighbours in the interleaved one, or two vectors of what is only copied). Otherwise an item is one pair.
template <bool WIDE, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float2 s_cs[];  // [tokens of the CTA][rot / 2]
  __shared__ int32_t s_pos[kRopeTokens];
  constexpr int kFlight = WIDE ? 2 : 4;  // items that a thread loads at a time
  const int tid = threadIdx.x, half = a.rot / 2, rows = a.Hq + a.H;
  const int t0 = blockIdx.x * a.tokens, here = min(a.tokens, a.T - t0), total = here * rows * a.items;
  struct Item {
    const uint16_t* src;
    uint16_t* dst;
    int t, at, to, item;  // token of the CTA; the two vectors (or elements) of the row
    bool turns, two;
  };
  auto find = [&](int i) {
    // (i x the divisor is below 2^32, so the product with its reciprocal is exact; 2^32 / 1 is not a 32-bit number)
    Item x;
    const int row_all = a.items == 1 ? i : __umulhi(i, a.by_items);
    x.item = i - row_all * a.items;
    x.t = rows == 1 ? row_all : __umulhi(row_all, a.by_rows);
    const int row = row_all - x.t * rows;
    const bool is_k = row >= a.Hq;
    const int h = is_k ? row - a.Hq : row;
    const int64_t tok = t0 + x.t;
    x.src = (is_k ? a.k + tok * a.k_stride : a.q + tok * a.q_stride) + h * a.d;
    x.dst = (is_k ? a.k_out + tok * a.k_out_stride : a.q_out + tok * a.q_out_stride) + h * a.d;
    if constexpr (WIDE) {
      x.turns = x.item < a.rot / 16;
      x.at = INTER || !x.turns ? x.item * 16 : x.item * 8;
      x.to = INTER || !x.turns ? x.at + 8 : x.at + half;
    } else {
      x.turns = x.item < half;
      x.at = INTER || !x.turns ? x.item * 2 : x.item;
      x.to = INTER || !x.turns ? x.at + 1 : x.at + half;
    }
    x.two = x.to < a.d;
    return x;
  };
  uint4 u[kFlight], v[kFlight];
  auto load = [&](int i0) {
#pragma unroll
    for (int y = 0; y < kFlight; ++y) {
      const int i = i0 + y * kRopeThreads;
      if (i >= total) break;
      const Item x = find(i);
      if constexpr (WIDE) {
        u[y] = *reinterpret_cast<const uint4*>(x.src + x.at);
        if (x.two) v[y] = *reinterpret_cast<const uint4*>(x.src + x.to);
      } else {
        u[y].x = x.src[x.at];
        v[y].x = x.two ? x.src[x.to] : 0u;
      }
    }
  };
  load(tid);  // (on its way under the sines)
  if (tid < here) s_pos[tid] = a.positions[t0 + tid];
  __syncthreads();
  for (int i = tid; i < here * half; i += kRopeThreads) {
    const int t = i / half;
    const uint64_t turn = a.turns[i - t * half] * static_cast<uint32_t>(s_pos[t]) + 0x80000000ull;
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
    s_cs[i] = make_float2(c * a.factor, s * a.factor);
  }
  __syncthreads();
#pragma unroll 1
  for (int i0 = tid; i0 < total; i0 += kFlight * kRopeThreads) {
    if (i0 != tid) load(i0);
#pragma unroll
    for (int y = 0; y < kFlight; ++y) {
      const int i = i0 + y * kRopeThreads;
      if (i >= total) break;
      const Item x = find(i);
      if (s_pos[x.t] < 0) continue;  // a padded step's row
      const float2* cs = s_cs + x.t * half;
      if constexpr (WIDE) {
        uint32_t p[4] = {u[y].x, u[y].y, u[y].z, u[y].w}, q[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
        if (x.turns) {
          // eight angles, two at a time
          const float4* at = reinterpret_cast<const float4*>(cs + x.item * 8);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 two = at[j];
            const float2 c0 = make_float2(two.x, two.y), c1 = make_float2(two.z, two.w);
            if constexpr (INTER) {
              uint32_t& w0 = j < 2 ? p[2 * j] : q[2 * j - 4];
              uint32_t& w1 = j < 2 ? p[2 * j + 1] : q[2 * j - 3];
              const float xa = bf_lo(w0), xb = bf_hi(w0), ya = bf_lo(w1), yb = bf_hi(w1);
              w0 = pack(first(xa, xb, c0), second(xa, xb, c0));
              w1 = pack(first(ya, yb, c1), second(ya, yb, c1));
            } else {
              const float xa = bf_lo(p[j]), xb = bf_hi(p[j]), ya = bf_lo(q[j]), yb = bf_hi(q[j]);
              p[j] = pack(first(xa, ya, c0), first(xb, yb, c1));
              q[j] = pack(second(xa, ya, c0), second(xb, yb, c1));
            }
          }
        }
        *reinterpret_cast<uint4*>(x.dst + x.at) = make_uint4(p[0], p[1], p[2], p[3]);
        if (x.two) *reinterpret_cast<uint4*>(x.dst + x.to) = make_uint4(q[0], q[1], q[2], q[3]);
      } else {
        uint32_t w = u[y].x | (v[y].x << 16);
        if (x.turns) {
          const float p = bf_lo(u[y].x), q = bf_lo(v[y].x);
          w = pack(first(p, q, cs[x.item]), second(p, q, cs[x.item]));
        }
        x.dst[x.at] = static_cast<uint16_t>(w);
        if (x.two) x.dst[x.to] = static_cast<uint16_t>(w >> 16);
      }
    }
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
  // tokens of a CTA: one while they are few
  a.tokens = a.T <= kRopeFew ? 1 : kRopeTokens;
  const int smem = a.tokens * (a.rot / 2) * static_cast<int>(sizeof(float2));
  const int grid = (a.T + a.tokens - 1) / a.tokens;
  auto go = [&](auto kern) {
    kern<<<grid, kRopeThreads, smem, s>>>(a);
    return cudaGetLastError();
  };
  if (wide) return a.interleaved ? go(rope_kernel<true, true>) : go(rope_kernel<true, false>);
  return a.interleaved ? go(rope_kernel<false, true>) : go(rope_kernel<false, false>);
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
