// gdn_attn4_decode.cu -- attention of single tokens over the 4-bit paged cache.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),  k_j, v_j = code * 2^(e - 127) by groups of 32 of the head
//
// Bound by memory on paper (17 / 32 bytes a value, read once), and next to that by instructions: the tensor cores take no
// 4-bit operand whose scale goes by groups of V's rows, so every code passes through registers once. Per 16 keys of a head
// of 256 (8,192 values, 4.35 KB) a warp has about 30 cycles of its scheduler's issue slots a KB, so the design counts
// instructions:
//   - codes become f16 pairs by one conversion of a byte (exact), straight into the operand registers of the warp-level
//     product, m16n8k16: keys (or d) on the 16-row side, query heads on the 8-column side, so that groups of up to 8 heads
//     waste nothing. A byte of K has two elements of a key, a byte of V one element of two keys: the pairs that the two
//     products' operands want.
//   - a scale is never multiplied with a value. K's enters after a group's 32 elements, on the 16 x 8 scores; V's is
//     multiplied with the probabilities, once for a group's 32 d.
//   - the tensor cores behind tcgen05 would want the same conversion and then a second trip through shared memory, which at
//     this rate is full: 3 bytes a value and 40 values a clock are 120 of its 128 bytes a clock.
// Measured on the GPU: the conversion 1.35 a clock and SM and more, the warp-level product 0.5 a clock and SM; a tile of 128
// keys needs 1,024 and 256 of them, and 1,480 clocks of memory.
//
// Queries are f16, scaled by a power of two per head so that the largest element lies in [2^14, 2^15): exact for bf16
// values down to 2^-31 of it. Probabilities x V's largest scale of the key are f16: 11 significant bits, and 2^-34 of the
// row's largest.
//
// Scales of V: with x the exponent of a score and e that of the key's largest scale of V, m is the running maximum of x + e
// and stands for 2^9; it moves when an x + e passes it by 2^5. p 2^e goes into the product, next to 2^(e_group - e), and p
// itself into the sum.
//
// Split: units of a request's own length (gdn_attn_units.cuh). A CTA's warps take a unit's steps of 16 keys in turn, each
// with a running maximum, a sum and an output of its own, without a barrier between; at the unit's end the four are joined in
// order, in shared memory. Copies run ahead in a ring of each warp's own (cp.async: a step of a page is contiguous; rows are
// padded so that the operand loads have no bank twice).
#include "gdn_attn.cuh"
#include "gdn_attn_units.cuh"
#include "gdn_cache4.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 16;              // keys of a step
constexpr float kRise = 5.0f;          // log2 of what a score may pass the running maximum by
constexpr float kTop = 9.0f;           // log2 of what the running maximum stands for

using Units = UnitRule<8, 10, 24>;
using Walk = WalkOf<Units>;
static_assert((1 << 10) / kStep / kWarps <= 32, "a lane for each of a warp's steps of a unit");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(at));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at));
  return r;
}
// c += a b, 16 x 16 by 16 x 8, f16 in, fp32 sums
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// NT: query heads of a unit by eights, 1 or 2.
template <int D, int NT>
struct Cfg {
  static constexpr int kG = D / kGroup4;                  // groups of a head
  static constexpr int kRowK = D / 2 + 16, kRowV = D + 32;  // bytes of a key's, of a key pair's row in a stage
  static constexpr int kAtV = kStep * kRowK, kAtScale = kAtV + kStep / 2 * kRowV;
  static constexpr int kStage = kAtScale + 2 * kStep * kG;
  static constexpr int kStages = 3;
  static constexpr int kScaleK = kStep * kG * 4, kScaleV = kStep * kG * 2;  // the step's scales as the products want them
  static constexpr int kWarp = kStages * kStage + kScaleK + kScaleV;        // of each warp
  static constexpr int kQ = NT * kG * 512;
  static constexpr int kRowO = D + 4;                     // floats of a head's row in the join
  static constexpr int kAtFactor = kWarps * kWarp + kQ, kAtMl = kAtFactor + 64, kAtLens = kAtMl + kWarps * 16 * 8;
  static constexpr int smem_of(int nb) { return kAtLens + 4 * (nb + nb / kCoarse + 2); }
  static_assert(kStage % 16 == 0 && kWarp % 16 == 0 && kWarp >= 8 * kRowO * 4, "alignment; the join's rows are in the rings");
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 2 && D == 256 ? 2 : 3) attn4_decode_kernel(const __grid_constant__ DecodeParams p) {
  using C = Cfg<D, NT>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int32_t s_scan[kWarps];
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int g = lane >> 2, c = lane & 3;
  const uint32_t base = smem_addr(smem), ring = base + warp * C::kWarp, s_k = ring + C::kStages * C::kStage, s_v = s_k + C::kScaleK;
  const uint32_t s_q = base + kWarps * C::kWarp;
  float* s_factor = reinterpret_cast<float*>(smem + C::kAtFactor);
  float2* s_ml = reinterpret_cast<float2*>(smem + C::kAtMl);  // [warp][16]
  int32_t* lens = reinterpret_cast<int32_t*>(smem + C::kAtLens);
  int32_t* tsum = lens + p.nb;
  const int cap = a.max_blocks * a.bs, shift = 31 - __clz(a.bs), G = a.Hq / a.H;

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
  w.start(blockIdx.x, gridDim.x);
  for (; w.more(); w.next()) {
    const int head0 = w.h * G + w.chunk * 16, heads = min(p.heads, G - w.chunk * 16), keys = w.keys();
    const int steps = (keys + kStep - 1) / kStep, mine = steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0;
    // the row of the cache that each of the warp's steps starts at, one to a lane
    int row = -1;
    if (lane < mine) {
      const int pos = w.first() + (warp + kWarps * lane) * kStep;
      const int page = a.block_table[static_cast<int64_t>(p.b0 + w.b) * a.max_blocks + (pos >> shift)];
      if (page >= 0 && page < a.num_blocks) row = ((page * a.H + w.h) << shift) + (pos & (a.bs - 1));
      else if (a.err) atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);
    }
    auto fetch = [&](int i) {  // the warp's i-th step into its ring
      const int from = __shfl_sync(0xFFFFFFFFu, row, i & 31);
      if (i < mine && from >= 0) {
        const uint32_t to = ring + (i % C::kStages) * C::kStage;
        const uint8_t* k = a.k_cache + static_cast<int64_t>(from) * (D / 2);
        const uint8_t* v = a.v_cache + static_cast<int64_t>(from) * (D / 2);
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          const int at = (lane + 32 * x) * 16;
          cp_async16(to + at / (D / 2) * C::kRowK + at % (D / 2), k + at);
          cp_async16(to + C::kAtV + at / D * C::kRowV + at % D, v + at);
        }
        if (lane < 2 * C::kG) {  // 16 bytes each: K's scales, V's
          const uint8_t* sc = reinterpret_cast<const uint8_t*>(lane < C::kG ? a.k_scale : a.v_scale);
          cp_async16(to + C::kAtScale + lane * 16, sc + static_cast<int64_t>(from) * C::kG + (lane % C::kG) * 16);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) fetch(i);

    // queries as the second operand of K's product: for each eight heads and group, a lane's four registers
    {
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
        const uint32_t to = s_q + ((h / 8) * C::kG + e / 4) * 512 + ((h % 8) * 4 + e % 4) * 16;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
        // a query that is not finite makes its head NaN through its factor
        if (e == 0)
          s_factor[h] = top < 0x7F80u ? fabsf(a.scale) * kLog2e * __uint_as_float(static_cast<uint32_t>(field - 14) << 23) : __int_as_float(0x7FC00000);
      }
    }
    __syncthreads();

    float o[D / 16][NT][4], m[NT][2], l[NT][2], fac[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[n][j] = -INFINITY;
        l[n][j] = 0.0f;
        fac[n][j] = s_factor[n * 8 + 2 * c + j];
      }
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[t][n][j] = 0.0f;

#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      __syncwarp();  // the stage that is filled next, and the scales, have been read
      fetch(i + C::kStages - 1);
      cp_async_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t st = ring + (i % C::kStages) * C::kStage;
      const bool there = __shfl_sync(0xFFFFFFFFu, row, i) >= 0;
      const int live = there ? keys - (warp + kWarps * i) * kStep : 0;  // keys of the step that are seen
      // the step's scales: lane = (key, half of its groups)
      int e_own;
      {
        constexpr int kN = C::kG / 2;
        const int key = lane >> 1, g0 = (lane & 1) * kN;
        uint32_t kb[kN], vb[kN];
        const uint32_t at = st + C::kAtScale + key * C::kG + g0;
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(kb[j]) : "r"(at + j));
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(vb[j]) : "r"(at + kStep * C::kG + j));
        }
        int top = kBias4 + kLeastScale;
#pragma unroll
        for (int j = 0; j < kN; ++j) top = max(top, vb[j] == kNaN4 ? 0 : static_cast<int>(vb[j]));
        top = min(max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1)), 253);
        e_own = top - kBias4;
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          const uint32_t f = kb[j] == kNaN4 ? 0x7FC00000u : kb[j] << 23;
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(s_k + (key * C::kG + g0 + j) * 4), "r"(f) : "memory");
          // 2^(e_group - e) in f16, subnormals too
          const int d = 15 + static_cast<int>(vb[j]) - top;
          uint32_t v = d > 0 ? static_cast<uint32_t>(d) << 10 : 0x200u >> min(-d, 31);
          if (vb[j] == kNaN4) v = 0x7E00u;
          if (key >= live) v = 0;
          // [lane's c][group][pair c or c + 4][key of the pair]
          asm volatile("st.shared.b16 [%0], %1;" ::"r"(s_v + (((key & 7) >> 1) * C::kG + g0 + j) * 8 + (key >> 3) * 4 + (key & 1) * 2),
                       "h"(static_cast<uint16_t>(v))
                       : "memory");
        }
      }
      __syncwarp();
      // scores of keys g and g + 8, heads 2 c and 2 c + 1
      float2 s[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int gr = 0; gr < C::kG; ++gr) {
        uint32_t x[4], y[4];
        e2m1x8(lds32(st + g * C::kRowK + gr * 16 + c * 4), x);
        e2m1x8(lds32(st + (g + 8) * C::kRowK + gr * 16 + c * 4), y);
        const float k0 = __uint_as_float(lds32(s_k + (g * C::kG + gr) * 4)), k1 = __uint_as_float(lds32(s_k + ((g + 8) * C::kG + gr) * 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 q = lds128(s_q + (n * C::kG + gr) * 512 + lane * 16);
          float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma(t, x[0], y[0], x[1], y[1], q.x, q.y);
          mma(t, x[2], y[2], x[3], y[3], q.z, q.w);
          s[n][0] = fma2(make_float2(t[0], t[1]), make_float2(k0, k0), s[n][0]);
          s[n][1] = fma2(make_float2(t[2], t[3]), make_float2(k1, k1), s[n][1]);
        }
      }
      const float e0 = static_cast<float>(__shfl_sync(0xFFFFFFFFu, e_own, 2 * g)), e1 = static_cast<float>(__shfl_sync(0xFFFFFFFFu, e_own, 2 * g + 16));
      const bool hidden0 = g >= live, hidden1 = g + 8 >= live;
      bool above = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        s[n][0].x = hidden0 ? -INFINITY : s[n][0].x * fac[n][0] + e0;
        s[n][0].y = hidden0 ? -INFINITY : s[n][0].y * fac[n][1] + e0;
        s[n][1].x = hidden1 ? -INFINITY : s[n][1].x * fac[n][0] + e1;
        s[n][1].y = hidden1 ? -INFINITY : s[n][1].y * fac[n][1] + e1;
        above |= fmaxf(s[n][0].x, s[n][1].x) > m[n][0] + kRise || fmaxf(s[n][0].y, s[n][1].y) > m[n][1] + kRise;
      }
      if (__any_sync(0xFFFFFFFFu, above)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float corr[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = j ? fmaxf(s[n][0].y, s[n][1].y) : fmaxf(s[n][0].x, s[n][1].x);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
            const float to = top > m[n][j] + kRise ? top : m[n][j];  // by the head alone, whatever the others do
            const float root = to == -INFINITY ? 1.0f : ex2_root(m[n][j] - to);
            m[n][j] = to;
            l[n][j] = l[n][j] * root * root;
            corr[j] = root * root;
          }
#pragma unroll
          for (int t = 0; t < D / 16; ++t) {
            o[t][n][0] *= corr[0];
            o[t][n][1] *= corr[1];
            o[t][n][2] *= corr[0];
            o[t][n][3] *= corr[1];
          }
        }
      }
      // p 2^e, and p into the sum; both keys' rows turned into columns
      const float d0 = __int_as_float((kBias4 - static_cast<int>(e0)) << 23), d1 = __int_as_float((kBias4 - static_cast<int>(e1)) << 23);
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float mx = m[n][0] == -INFINITY ? 0.0f : m[n][0] - kTop, my = m[n][1] == -INFINITY ? 0.0f : m[n][1] - kTop;
        const float px0 = ex2(s[n][0].x - mx), py0 = ex2(s[n][0].y - my), px1 = ex2(s[n][1].x - mx), py1 = ex2(s[n][1].y - my);
        l[n][0] += px0 * d0 + px1 * d1;
        l[n][1] += py0 * d0 + py1 * d1;
        pb[n][0] = transpose8(pack_f16(px0, py0));
        pb[n][1] = transpose8(pack_f16(px1, py1));
      }
#pragma unroll
      for (int gr = 0; gr < C::kG; ++gr) {
        uint32_t x[4], y[4];
        e2m1x8(lds32(st + C::kAtV + c * C::kRowV + gr * 32 + g * 4), x);
        e2m1x8(lds32(st + C::kAtV + (c + 4) * C::kRowV + gr * 32 + g * 4), y);
        const uint32_t v0 = lds32(s_v + (c * C::kG + gr) * 8), v1 = lds32(s_v + (c * C::kG + gr) * 8 + 4);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t b0 = mul_f16x2(pb[n][0], v0), b1 = mul_f16x2(pb[n][1], v1);
          mma(o[2 * gr][n], x[0], x[1], y[0], y[1], b0, b1);
          mma(o[2 * gr + 1][n], x[2], x[3], y[2], y[3], b0, b1);
        }
      }
    }
    cp_async_wait<0>();
    // the unit's sums: over the warp's lanes, then over the warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][j] += __shfl_xor_sync(0xFFFFFFFFu, l[n][j], x);
        if (g == 0) s_ml[warp * 16 + n * 8 + 2 * c + j] = make_float2(m[n][j], l[n][j]);
      }
    __syncthreads();
    // a warp's weight (its root: a sum is multiplied with it twice)
    auto weight = [&](float2 e, float top) { return e.x == -INFINITY ? (e.y == 0.0f ? 0.0f : 1.0f) : ex2_root(e.x - top); };
    auto largest = [&](int h) { return fmaxf(fmaxf(s_ml[h].x, s_ml[16 + h].x), fmaxf(s_ml[32 + h].x, s_ml[48 + h].x)); };
    const int64_t f = ((static_cast<int64_t>(w.b) * a.H + w.h) * p.chunks + w.chunk) * p.each + w.index;
    const bool alone = w.count == 1;
    float* rows = reinterpret_cast<float*>(smem);  // [warp]'s part of the rings: [8][kRowO]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float corr[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float root = weight(make_float2(m[n][j], l[n][j]), largest(n * 8 + 2 * c + j));
        corr[j] = root * root;
      }
      // a lane has d 32 gr + 4 g .. + 3 of heads 2 c and 2 c + 1 (a warp without a key: zeros, not 0 * what is there)
#pragma unroll
      for (int gr = 0; gr < C::kG; ++gr)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 v = make_float4(o[2 * gr][n][j] * corr[j], o[2 * gr][n][2 + j] * corr[j], o[2 * gr + 1][n][j] * corr[j], o[2 * gr + 1][n][2 + j] * corr[j]);
          *reinterpret_cast<float4*>(rows + warp * (C::kWarp / 4) + (2 * c + j) * C::kRowO + gr * 32 + g * 4) = v;
        }
      __syncthreads();
      for (int i = tid; i < 8 * (D / 4); i += kThreads) {
        const int h = n * 8 + i / (D / 4), d = i % (D / 4) * 4;
        if (h >= heads) break;
        const float top = largest(h);
        float sum = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
          const float root = weight(s_ml[x * 16 + h], top);
          sum += s_ml[x * 16 + h].y * root * root;
          const float4 y = *reinterpret_cast<const float4*>(rows + x * (C::kWarp / 4) + (h - n * 8) * C::kRowO + d);
          v.x += y.x;
          v.y += y.y;
          v.z += y.z;
          v.w += y.w;
        }
        if (alone) {
          const float inv = sum > 0.0f || sum != sum ? __fdividef(1.0f, sum) : 0.0f;
          uint2 st;
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.x) : "f"(v.y * inv), "f"(v.x * inv));
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.y) : "f"(v.w * inv), "f"(v.z * inv));
          *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(p.b0 + w.b) * a.Hq + head0 + h) * D + d) = st;
        } else {
          if (d == 0) p.ml[f * p.heads + h] = make_float2(top, sum);
          *reinterpret_cast<float4*>(p.part + (f * p.heads + h) * D + d) = v;
        }
      }
      __syncthreads();  // the rings are filled anew
    }
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
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  int per_sm = kSmemPerSm / (smem + static_cast<int>(fa.sharedSizeBytes) + 1024);
  const int by_regs = 65536 / (((fa.numRegs + 7) & ~7) * kThreads);
  if (per_sm > by_regs) per_sm = by_regs;
  if (per_sm < 1) per_sm = 1;
  const int64_t most = static_cast<int64_t>(p.nb) * p.a.H * p.chunks * p.each;
  const int grid = static_cast<int>(most < static_cast<int64_t>(per_sm) * sm_count() ? most : per_sm * sm_count());
  kern<<<grid, kThreads, smem, s>>>(p);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join<D, Units>(p, s);
}

template <int D>
cudaError_t launch_h(DecodeParams& p, cudaStream_t s) {
  return p.heads <= 8 ? launch_d<D, 1>(p, s) : launch_d<D, 2>(p, s);
}

}  // namespace

size_t attn4_decode_workspace(int B, int max_blocks, int Hq, int H, int d, int bs) {
  const int most = attn_decode_batch(max_blocks, Hq, H, bs);
  return decode_layout<Units>(B < most ? B : most, max_blocks, Hq, H, d, bs).total;
}

cudaError_t launch_attn4_decode(const AttnArgs& a, cudaStream_t s) {
  const int G = a.Hq / a.H;
  DecodeParams p;
  p.a = a;
  p.fault = 0;
  p.heads = G < 16 ? G : 16;
  p.chunks = (G + 15) / 16;
  p.each = static_cast<int>(Units::most(static_cast<int64_t>(a.max_blocks) * a.bs));
  const int most = attn_decode_batch(a.max_blocks, a.Hq, a.H, a.bs);  // (not 0: the caller has checked)
  const int launches = (a.B + most - 1) / most, per = (a.B + launches - 1) / launches;
  for (int b0 = 0; b0 < a.B; b0 += per) {
    p.b0 = b0;
    p.nb = a.B - b0 < per ? a.B - b0 : per;
    const DecodeLayout L = decode_layout<Units>(p.nb, a.max_blocks, a.Hq, a.H, a.d, a.bs);
    char* ws = static_cast<char*>(a.workspace);
    p.ml = reinterpret_cast<float2*>(ws);
    p.part = reinterpret_cast<float*>(ws + L.part);
    const cudaError_t e = a.d == 64 ? launch_h<64>(p, s) : a.d == 128 ? launch_h<128>(p, s) : launch_h<256>(p, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace gdn
