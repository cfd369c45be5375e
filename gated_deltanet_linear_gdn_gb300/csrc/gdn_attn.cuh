// gdn_attn.cuh -- device helpers that the two attention kernels over the 8-bit cache share: key tiles
// and their TMA boxes, 8-bit tcgen05 products, splitting fp32 values into e4m3 parts.
#pragma once

#include "gdn_cache.cuh"
#include "gdn_ptx.cuh"
#include "gdn_tc.cuh"

namespace gdn {

constexpr int kTile = 128;                // keys of a tile
constexpr int kGroup = 16;                // keys of one TMA box: the smallest block
constexpr int kGroups = kTile / kGroup;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The root of exp2(x). A row's sum is multiplied with it twice: next to a scale of V of 2^90 the sum of a block of zeros (2^-64)
// is within what fp32 holds and exp2(x) is not.
__device__ __forceinline__ float ex2_root(float x) { return ex2(0.5f * x); }
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

// Four f16 values (none above 57,344) as sums of three e5m2 values each. An f16's upper byte is an e5m2 value: the first two
// parts are that byte rounded (half of its last place added to the magnitude, which carries as it should), and what they
// leave is exact in f16; the third is rounded to nearest. Exact from 2^-6 on, below that to 2^-17. NaN stays NaN through
// the third part.
__device__ __forceinline__ void split_e5m2(const uint32_t (&h)[2], uint32_t (&part)[3]) {
  uint32_t hi[2], mid[2], lo[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    uint32_t r;
    hi[y] = (h[y] + 0x00800080u) & 0xFF00FF00u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h[y]), "r"(hi[y]));
    mid[y] = (r + 0x00800080u) & 0xFF00FF00u;
    asm("{.reg .b16 x; sub.rn.f16x2 %0, %1, %2; cvt.rn.satfinite.e5m2x2.f16x2 x, %0; mov.b32 %0, {x, 0};}" : "=&r"(lo[y]) : "r"(r), "r"(mid[y]));
  }
  part[0] = __byte_perm(hi[0], hi[1], 0x7531);
  part[1] = __byte_perm(mid[0], mid[1], 0x7531);
  part[2] = __byte_perm(lo[0], lo[1], 0x5410);
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(dst), "l"(map), "r"(x), "r"(row), "r"(bar)
      : "memory");
}

// Before a barrier is made anew: nothing may be on its way to it.
__device__ __forceinline__ void mbar_inval(uint32_t bar) { asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar) : "memory"); }

// Waits for a barrier's phase, giving up after about a second or as soon as another role of the CTA has
// (`fail`, in shared memory). False: the caller stops.
// Kept small: a kernel holds some twenty of them, and its first pass through its code is paced by
// instruction fetches.
__device__ __forceinline__ bool wait_or_fail(uint32_t bar, uint32_t parity, volatile int* fail) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
#pragma unroll 1
  while (!mbar_try_wait_sleep(bar, parity, 20000u)) {
    if (*fail || global_ns() - t0 > 1000000000ull) {
      *fail = 1;
      return false;
    }
  }
  return true;
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
#define GDN_F8(v, i) "f"(v[i]), "f"(v[i + 1]), "f"(v[i + 2]), "f"(v[i + 3]), "f"(v[i + 4]), "f"(v[i + 5]), "f"(v[i + 6]), "f"(v[i + 7])
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      GDN_F8(v, 0), GDN_F8(v, 8), GDN_F8(v, 16), GDN_F8(v, 24)
      : "memory");
}
#undef GDN_F8

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
               "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
               : "memory");
}

// The factor of a score in the exponent. Never zero, so that a masked score (-inf) stays -inf: a
// smaller one moves no exponent (scores are below 2^26).
__device__ __forceinline__ float exponent_scale(float ks, float factor) { return fmaxf(fabsf(ks) * factor, 1e-37f); }

// log2 of the scales of V below which a key's part of the row's sum is computed by itself: from p * vs, as elsewhere, it
// would be lost where the row's largest p * vs is 2^126 times as large.
constexpr int kFarScale = -30;
// log2 of the least scale of V. Smaller ones, zero among them, count as it: a row's sum is of (p vs) / vs, and 2^15 / 2^-90 for
// each of 2^20 keys is within what fp32 holds. (The writer's least is 2^-64.)
constexpr int kLeastScale = -90;

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
// Instruction descriptor: fp32 D, e4m3 A and B, each optionally MN-major.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

constexpr uint32_t kIdescE5m2A = 1u << 7;  // A in e5m2 instead (the two types of this kind are free of each other)

// Operand tiles are rows of min(d, 128) bytes in the hardware swizzle that TMA writes (128-byte
// rows: 16-byte chunk ^ row mod 8; 64-byte rows: chunk ^ (row / 2) mod 4), 8 rows to an atom;
// d = 256 has two such tiles side by side.
//   K-major (Q, K): the stride offset is the next 8 rows; a K step of 32 is 32 bytes on.
//   MN-major (V, rows are K): the stride offset is the next 8 K rows, the leading offset the next
//   128 bytes of N; a K step of 32 is 32 rows on.
template <int D, int ROWS = kTile>
struct Tile {
  static constexpr int kRow = D < 128 ? D : 128;
  static constexpr int kHalf = ROWS * kRow;            // one tile of kRow bytes a row
  static constexpr int kBytes = ROWS * D;
  static __device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lbo) {
    uint64_t d = tc::smem_desc(addr, lbo, 8 * kRow);
    d |= static_cast<uint64_t>(D < 128 ? 4 : 2) << 61;  // 64-byte / 128-byte swizzle
    return d;
  }
  static __device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
    if (D < 128) return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
    return (chunk >> 3) * kHalf + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
  }
};

}  // namespace gdn
