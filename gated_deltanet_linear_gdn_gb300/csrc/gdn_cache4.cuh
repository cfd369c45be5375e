// gdn_cache4.cuh -- what the kernels of the 4-bit paged cache share: argument blocks, e2m1 conversions and the launch
// declarations.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_cache.cuh"

namespace gdn {

constexpr int kGroup4 = 32;        // elements of a head that share a scale
constexpr int kBias4 = 127;        // a scale's byte stands for 2^(byte - 127)
constexpr int kNaN4 = 255;         // ... and this one for NaN
constexpr int kLeastByte4 = 63;    // 2^-64, the least the writer stores

struct Cache4 {
  uint8_t* k;        // [num_blocks, H, bs, d / 2]: elements 2 i (low) and 2 i + 1 of a token in a byte
  uint8_t* v;        // [num_blocks, H, bs / 2, d]: an element of tokens 2 j (low) and 2 j + 1 in a byte
  uint8_t* k_scale;  // [num_blocks, H, bs, d / 32]
  uint8_t* v_scale;
  int num_blocks, H, d, bs;
};

struct Append4Args {
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_stride, v_stride;  // elements from one token to the next
  const int32_t* slot_map;
  int T;
  Cache4 c;
  int32_t* err;
};

struct Read4Args {
  Cache4 c;
  const int32_t* slot_map;
  int T;
  uint16_t* k;
  uint16_t* v;
  int64_t k_stride, v_stride;
  int32_t* err;
};

// The pages that a prompt call's requests hold, as an 8-bit cache of their own.
struct Expand4Args {
  Cache4 c;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* lens;
  const int32_t* cu_tokens;
  int B, T;
  int held;               // pages that there is room for
  int32_t* table;         // [B, max_blocks]
  uint8_t* k;             // [held, H, bs, d] e4m3
  uint8_t* v;
  float* k_scale;         // [held, H]
  float* v_scale;
  int32_t* err;
};
constexpr int kExpandBatch = 4096;  // requests of one call: their pages are counted in shared memory

cudaError_t launch_cache4_append(const Append4Args& a, cudaStream_t s);
cudaError_t launch_cache4_read(const Read4Args& a, cudaStream_t s);
// (a programmatic dependent of the prompts' plan: launch_attn_prefill launches it)
cudaError_t launch_cache4_expand(const Expand4Args& a, cudaStream_t s);

// AttnArgs over the 4-bit cache: k_cache, v_cache as bytes, k_scale and v_scale the scales' bytes.
size_t attn4_decode_workspace(int B, int max_blocks, int Hq, int H, int d, int bs);
cudaError_t launch_attn4_decode(const AttnArgs& a, cudaStream_t s);

#ifdef __CUDACC__

// Eight codes (a 32-bit word, element 0 in its lowest four bits) as four pairs of f16 values. Exact.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&o)[4]) {
  asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b; cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d;}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
// Eight values rounded to codes (nearest, ties to even, +-6 beyond), element 0 in the lowest four bits.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

#endif

}  // namespace gdn
