// gdn_rope.cuh -- argument block and launch declaration of the rotary positions.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

constexpr int kRopeMaxDim = 1024;  // of a head: its items fit in 64 threads, sines and cosines of kRopeTokens tokens in 16 KB
constexpr int kRopeTokens = 4;     // tokens of a CTA of narrow items
constexpr int kRopeFew = 256, kRopeMany = 1024;  // tokens up to which each has 256 threads, and 128

struct RopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* q_out;
  uint16_t* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;  // elements from one token to the next
  const int32_t* positions;
  const uint64_t* turns;  // [rot / 2]: frequencies in turns a position, times 2^64
  int T, Hq, H, d, rot, interleaved;
  float factor;
  // set by the launch: items of a (token, head) row, and 2^32 / items and / rows, rounded up
  int items;
  uint32_t by_items, by_rows;
};

cudaError_t launch_rope(RopeArgs a, cudaStream_t s);

}  // namespace gdn
