// gdn_cache.cu -- the tables of a step over a paged cache, built on the GPU from request
// lengths, and the writer of the 8-bit cache.
//
// cache_tables_kernel. With n(l) = ceil(l / block_size), a row that grows from `old` to `new`
// tokens takes n(new) - n(old) blocks from the head of the free ring, in row order, and a row
// that shrinks puts its blocks back at the tail:
//   need = max(0, n(new) - n(old)), give = max(0, n(old) - n(new)),
//   table[b, n(old) + j]             = ring[(head + sum_{b'<b} need + j) mod N]
//   ring[(head + count + sum give + j) mod N] = table[b, n(new) + j]
// Everything a token needs (its row, its block) follows from three prefix sums over the rows.
// Bound by latency, not bytes: a step of 64 rows moves 2 KB, one of 1,024 rows and 50,000 new tokens
// 1 MB. So it is ONE launch: every CTA computes the prefix sums for itself (warp scans over the
// lengths, which stay in shared memory) and takes its share of rows and tokens. A token of a block
// that is being handed out reads the ring, not the table, so rows and tokens need no ordering. The only
// values that could be read by all and rewritten by one are the pool's head and count and the lengths,
// when the caller updates them in place: then the CTAs form one thread-block cluster and write after its
// barrier. With outputs of their own there is no barrier and as many CTAs as the tokens fill (1,024 rows,
// 400 new tokens for one in 20: 6.2 us, and 8.6 in place; 64 rows of one token 4.0 and 4.2).
//
// cache_append_kernel. Per touched (block, head), with a = max |x| over the finite values of
// the block's new tokens:
//   s = max(s_old if the block held tokens before, a / 448, 2^-64),  byte = e4m3(x * (1 / s))
// and tokens that were there are rewritten as e4m3((byte * s_old) * (1 / s)) if s grew. All in
// IEEE fp32 with one rounding to 8 bits (nearest even, saturating): the bytes are reproducible
// bit for bit. Bound by memory (2 bytes read and 1 written per value): the new values are
// read once, into registers, between the maximum and the rounding. 202 MB of prompts take 37.0 us (5.5 TB/s), 256
// single tokens 4.0 us.
#include "gdn_cache.cuh"
#include "gdn_ptx.cuh"

namespace gdn {

namespace {

constexpr int kTabThreads = 512;
constexpr int kTabCluster = 8;   // CTAs when outputs overwrite inputs
constexpr int kTabMost = 64;     // CTAs otherwise
constexpr long long kSaturated = 0x7fffffffLL;

struct Sum3 {
  long long need, give, tok;
};

__device__ __forceinline__ Sum3 warp_scan(Sum3 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xFFFFFFFFu, v.need, o);
    const long long b = __shfl_up_sync(0xFFFFFFFFu, v.give, o);
    const long long c = __shfl_up_sync(0xFFFFFFFFu, v.tok, o);
    if (lane >= o) {
      v.need += a;
      v.give += b;
      v.tok += c;
    }
  }
  return v;
}

__device__ __forceinline__ int blocks_of(int len, int shift) { return (len + (1 << shift) - 1) >> shift; }
// x mod n for 0 <= x < 2 n (n <= 2^27)
__device__ __forceinline__ int wrap(int x, int n) { return x >= n ? x - n : x; }

// A row's lengths; one outside [0, max_blocks * block_size] makes the row empty.
__device__ __forceinline__ bool row_lens(const TablesArgs& a, int b, int& o, int& n) {
  o = a.lens_old[b];
  n = a.lens_new[b];
  const long long cap = static_cast<long long>(a.max_blocks) * a.block_size;
  if (o < 0 || n < 0 || o > cap || n > cap) {
    o = n = 0;
    return false;
  }
  return true;
}

__global__ void __launch_bounds__(kTabThreads) cache_tables_kernel(TablesArgs a, int in_place, int wide) {
  extern __shared__ int32_t sm[];
  int32_t* s_cu = sm;               // [B + 1] tokens before row b (saturated at INT32_MAX)
  int32_t* s_need = sm + a.B + 1;   // [B] blocks asked for by rows 0 .. b (saturated)
  int32_t* s_give = s_need + a.B;   // [B] blocks given back by rows 0 .. b (saturated)
  int32_t* s_old = s_give + a.B;    // [B]
  int32_t* s_new = s_old + a.B;     // [B]
  __shared__ Sum3 s_warp[kTabThreads / 32];
  __shared__ unsigned long long s_taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, nrank = gridDim.x;
  int head = a.pool[0], count = a.pool[1];
  const int bs = a.block_size, shift = 31 - __clz(a.block_size);
  const int N = a.num_blocks;
  if (tid == 0) s_taken = 0;
  int flags = 0;
  if (head < 0 || head >= N || count < 0 || count > N) {  // no such pool: nothing to hand out
    head = count = 0;
    flags = GDN_DEVERR_BLOCKS;
  }
  Sum3 carry{0, 0, 0};
#pragma unroll 1
  for (int base = 0; base < a.B; base += kTabThreads) {
    const int b = base + tid;
    int o = 0, n = 0;
    if (b < a.B && !row_lens(a, b, o, n)) flags |= GDN_DEVERR_SEQLENS;
    const int no = blocks_of(o, shift), nn = blocks_of(n, shift);
    const int need = max(nn - no, 0), give = max(no - nn, 0);
    const Sum3 inc = warp_scan(Sum3{need, give, max(n - o, 0)}, lane);
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
      const Sum3 wi = warp_scan(lane < kTabThreads / 32 ? s_warp[lane] : Sum3{0, 0, 0}, lane);
      if (lane < kTabThreads / 32) s_warp[lane] = wi;
    }
    __syncthreads();
    Sum3 before = carry;
    if (warp > 0) {
      before.need += s_warp[warp - 1].need;
      before.give += s_warp[warp - 1].give;
      before.tok += s_warp[warp - 1].tok;
    }
    if (b < a.B) {
      const long long upto = before.need + inc.need;
      const bool refused = need > 0 && upto > count;
      if (refused) flags |= GDN_DEVERR_BLOCKS;
      // the last row that is served has the largest sum: rows are served in order
      if (need > 0 && !refused) atomicMax(&s_taken, static_cast<unsigned long long>(upto));
      s_need[b] = static_cast<int32_t>(min(upto, kSaturated));
      s_give[b] = static_cast<int32_t>(min(before.give + inc.give, kSaturated));
      s_cu[b + 1] = static_cast<int32_t>(min(before.tok + inc.tok, kSaturated));
      s_old[b] = o;
      s_new[b] = n;
    }
    carry.need += s_warp[kTabThreads / 32 - 1].need;
    carry.give += s_warp[kTabThreads / 32 - 1].give;
    carry.tok += s_warp[kTabThreads / 32 - 1].tok;
    __syncthreads();
  }
  if (tid == 0) s_cu[0] = 0;
  __syncthreads();
  // every CTA has read the lengths and the pool: they may be rewritten from here on
  if (in_place && nrank > 1) {
    cluster_arrive();
    cluster_wait();
  }
  if (carry.tok > a.total_tokens) flags |= GDN_DEVERR_SEQLENS;
  if (rank == 0 && tid == 0) {
    const long long taken = static_cast<long long>(s_taken);
    a.pool_out[0] = static_cast<int32_t>((head + taken) % N);
    a.pool_out[1] = static_cast<int32_t>(count - taken + carry.give);
    a.cu_tokens[0] = 0;
  }
  if (flags != 0 && a.err && rank == 0) atomicOr(a.err, flags);

  // rows: the sums and the lengths
  const int me = rank * kTabThreads + tid, all = nrank * kTabThreads;
  auto need_of = [&](int b) { return max(blocks_of(s_new[b], shift) - blocks_of(s_old[b], shift), 0); };
  auto refused_row = [&](int b) { return need_of(b) > 0 && s_need[b] > count; };
#pragma unroll 1
  for (int b = me; b < a.B; b += all) {
    a.cu_tokens[b + 1] = s_cu[b + 1];
    a.lens[b] = refused_row(b) ? s_old[b] : s_new[b];
  }
  // blocks that change hands: the e-th taken is the ring's e-th from its head, the e-th given back goes e
  // past its tail; the row is the first whose sum exceeds e
  auto row_of = [&](const int32_t* sums, int e) {
    int lo = 0, hi = a.B - 1;
#pragma unroll 1
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sums[mid] > e) hi = mid; else lo = mid + 1;
    }
    return lo;
  };
  const int taken = static_cast<int>(s_taken), given = s_give[a.B - 1];
  const int tail = wrap(head + count, N);
#pragma unroll 1
  for (int e = me; e < taken; e += all) {
    const int b = row_of(s_need, e);
    a.block_table[static_cast<int64_t>(b) * a.max_blocks + blocks_of(s_old[b], shift) + e - (s_need[b] - need_of(b))] =
        a.ring[wrap(head + e, N)];
  }
#pragma unroll 1
  for (int e = me; e < given; e += all) {
    const int b = row_of(s_give, e), no = blocks_of(s_old[b], shift);
    a.ring[static_cast<int>((static_cast<uint32_t>(tail) + static_cast<uint32_t>(e)) % static_cast<uint32_t>(N))] =
        a.block_table[static_cast<int64_t>(b) * a.max_blocks + no + e - s_give[b]];
  }
  // tokens: four in a row for a thread
  const int real = min(s_cu[a.B], a.total_tokens);
#pragma unroll 1
  for (int t = (rank * kTabThreads + tid) * 4; t < a.total_tokens; t += nrank * kTabThreads * 4) {
    int lo = 0, hi = a.B - 1;  // the last row that starts at or before t
    if (t < real) {
#pragma unroll 1
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_cu[mid] <= t) lo = mid; else hi = mid - 1;
      }
    }
    int slot[4], pos[4], blk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      slot[i] = pos[i] = -1;
      blk[i] = 0;
      if (t + i < real) {
        while (s_cu[lo + 1] <= t + i) ++lo;
        pos[i] = s_old[lo] + t + i - s_cu[lo];
        if (!refused_row(lo)) {
          const int first = s_need[lo] - need_of(lo), no = blocks_of(s_old[lo], shift), at = pos[i] >> shift;
          blk[i] = at < no ? a.block_table[static_cast<int64_t>(lo) * a.max_blocks + at]
                           : a.ring[wrap(head + first + at - no, N)];
          slot[i] = 0;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (slot[i] == 0) slot[i] = blk[i] * bs + (pos[i] & (bs - 1));
    if (wide && t + 3 < a.total_tokens) {
      *reinterpret_cast<int4*>(a.slot_map + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t + i < a.total_tokens) {
          a.slot_map[t + i] = slot[i];
          a.positions[t + i] = pos[i];
        }
    }
  }
}

// ------------------------------------------------------------------------------- cache writer

constexpr int kAppThreads = 256;
constexpr int kAppWarps = kAppThreads / 32;
// Tokens up to which a call gets windows of 8 tokens, for decode rows, and not of a block, for prompts (4 heads of 128,
// blocks of 64). 2,048 tokens: single rows 17.2 us and 79.2, one prompt 6.2 and 3.4. 4,096: rows 31.3 and 93.4, a prompt
// 9.7 and 3.8. Rows come by the hundred and prompts by the thousand.
constexpr int kShortAppend = 2048;
constexpr int kShortHold = 4;

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void from_e4m3x2(uint32_t h, float& lo, float& hi) {
  uint32_t p;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(p) : "h"(static_cast<uint16_t>(h)));
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
      : "=f"(lo), "=f"(hi) : "r"(p));
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// max |x| of 8 bf16 values, two at a time; NaN does not count, infinity does
__device__ __forceinline__ uint32_t amax8(const uint4& u, uint32_t m) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7FFF7FFFu));
  return m;
}
// the same over the finite values alone: as integers, |x| orders like its bits, from 0x7F80 on not finite
__device__ __forceinline__ uint32_t amax8_finite(const uint4& u, uint32_t m) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    m = max(m, lo < 0x7F80u ? lo : 0u);
    m = max(m, hi < 0x7F80u ? hi : 0u);
  }
  return m;
}
__device__ __forceinline__ uint2 quant8(const uint4& u, float r) {
  uint2 o;
  o.x = to_e4m3x2(__fmul_rn(bf_lo(u.x), r), __fmul_rn(bf_hi(u.x), r)) |
        (to_e4m3x2(__fmul_rn(bf_lo(u.y), r), __fmul_rn(bf_hi(u.y), r)) << 16);
  o.y = to_e4m3x2(__fmul_rn(bf_lo(u.z), r), __fmul_rn(bf_hi(u.z), r)) |
        (to_e4m3x2(__fmul_rn(bf_lo(u.w), r), __fmul_rn(bf_hi(u.w), r)) << 16);
  return o;
}
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float s_old, float r) {
  float f[4];
  from_e4m3x2(w & 0xFFFFu, f[0], f[1]);
  from_e4m3x2(w >> 16, f[2], f[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __fmul_rn(__fmul_rn(f[i], s_old), r);
  return to_e4m3x2(f[0], f[1]) | (to_e4m3x2(f[2], f[3]) << 16);
}

// One run (consecutive tokens [t, t + n) that fill offsets [off, off + n) of one block) of one head's keys or
// values, by a team of TS warps. Its values stay in registers between the maximum and the rounding as far as
// HOLD 16-byte vectors a lane go, and are read again (from L2) beyond that.
template <int TS, int HOLD>
__device__ __forceinline__ void write_run(const AppendArgs& a, const uint16_t* x, int64_t stride, uint8_t* cache,
                                          float* scales, int t, int n, int slot, int h, int team, uint32_t* s_red) {
  constexpr int NT = TS * 32;
  const int lane = threadIdx.x % NT;
  const int lv = 28 - __clz(a.d);  // log2 of a token's 16-byte vectors
  const int total = n << lv;
  const int blk = slot / a.bs, off = slot - blk * a.bs;
  const uint16_t* src = x + static_cast<int64_t>(t) * stride + h * a.d;
  const int64_t of_head = static_cast<int64_t>(blk) * a.H + h;
  const float s_was = off > 0 ? scales[of_head] : 0.0f;  // a block that held no token has no scale yet
  auto vector = [&](int e) { return *reinterpret_cast<const uint4*>(src + (e >> lv) * stride + ((e & ((1 << lv) - 1)) << 3)); };
  uint4 held[HOLD];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < HOLD; ++i) {
    held[i] = make_uint4(0, 0, 0, 0);
    if (lane + i * NT < total) held[i] = vector(lane + i * NT);
  }
#pragma unroll
  for (int i = 0; i < HOLD; ++i) m = amax8(held[i], m);
#pragma unroll 1
  for (int e = lane + HOLD * NT; e < total; e += NT) m = amax8(vector(e), m);
  m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
  if (m >= 0x7F80u) {  // an infinity: once more without it
    m = 0;
#pragma unroll 1
    for (int e = lane; e < total; e += NT) m = amax8_finite(vector(e), m);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
  }
  if constexpr (TS > 1) {
    if (lane % 32 == 0) s_red[threadIdx.x / 32] = m;
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + team), "n"(NT) : "memory");
#pragma unroll
    for (int i = 0; i < TS; ++i) m = max(m, s_red[team * TS + i]);
  }
  const float amax = __uint_as_float(m << 16);
  const float s = fmaxf(fmaxf(__fmul_rn(amax, 1.0f / kE4m3Max), s_was), kCacheMinScale);
  const float r = __fdiv_rn(1.0f, s);
  uint8_t* dst = cache + of_head * a.bs * a.d;
  uint2* put = reinterpret_cast<uint2*>(dst + static_cast<int64_t>(off) * a.d);
#pragma unroll
  for (int i = 0; i < HOLD; ++i)
    if (lane + i * NT < total) put[lane + i * NT] = quant8(held[i], r);
#pragma unroll 1
  for (int e = lane + HOLD * NT; e < total; e += NT) put[e] = quant8(vector(e), r);
  if (off > 0 && s != s_was) {  // the tokens before: same values under the larger scale
    const int words = off * a.d / 16;
#pragma unroll 1
    for (int e = lane; e < words; e += NT) {
      uint4* p = reinterpret_cast<uint4*>(dst) + e;
      const uint4 w = *p;
      *p = make_uint4(rescale4(w.x, s_was, r), rescale4(w.y, s_was, r), rescale4(w.z, s_was, r),
                      rescale4(w.w, s_was, r));
    }
  }
  // the old scale has been read by all of the team
  if constexpr (TS > 1) asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + team), "n"(NT) : "memory");
  else __syncwarp();
  if (lane == 0) scales[of_head] = s;
}

// Four CTAs an SM: three, without the 8 bytes of spills, wrote 202 MB in 41.0 us and not in 37.0.
// grid: (windows of W tokens, groups of `pairs` (head, keys or values) pairs). The CTA's work are the runs that
// start in its window, times its pairs; its teams take them in turn. A run starts where a token does not
// continue the one before it in the same block.
constexpr int kMaxWindow = 128;

template <int TS, int HOLD>
__global__ void __launch_bounds__(kAppThreads, 4) cache_append_kernel(AppendArgs a, int W, int pairs) {
  __shared__ int32_t s_slot[2 * kMaxWindow + 32];  // slots of tokens t0 - 1 ..
  __shared__ uint32_t s_break[2 * kMaxWindow / 32];  // bit i: token t0 + i does not continue t0 + i - 1
  __shared__ uint32_t s_red[kAppWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, team = warp / TS;
  const int t0 = blockIdx.x * W, look = W + a.bs;  // a run that starts in the window ends within `look` tokens
  const int64_t cap = static_cast<int64_t>(a.num_blocks) * a.bs;
  for (int i = tid; i <= look; i += kAppThreads) {
    const int t = t0 + i - 1;
    s_slot[i] = t >= 0 && t < a.T ? a.slot_map[t] : -1;
  }
  __syncthreads();
  bool bad = false;
#pragma unroll
  for (int i = tid; i < 2 * kMaxWindow; i += kAppThreads) {  // token t0 + i (look <= 256)
    const int slot = i < look ? s_slot[i + 1] : -1, prev = i < look ? s_slot[i] : -1;
    const bool goes_on = slot >= 0 && prev >= 0 && slot == prev + 1 && (slot & (a.bs - 1)) != 0;
    bad |= i < W && slot >= cap;
    const uint32_t w = __ballot_sync(0xFFFFFFFFu, !goes_on);
    if (lane == 0) s_break[i / 32] = w;
  }
  if (bad && a.err && blockIdx.y == 0) atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);
  __syncthreads();
  const int pair0 = blockIdx.y * pairs;
  int turn = 0;
#pragma unroll 1
  for (int w = 0; w * 32 < W; ++w) {
    uint32_t starts = s_break[w];
    if (W - w * 32 < 32) starts &= (1u << (W - w * 32)) - 1u;
    const bool only = (starts & (starts - 1)) == 0;  // (a short call's window is within a word)
#pragma unroll 1
    for (; starts; starts &= starts - 1) {
      const int i = w * 32 + __ffs(starts) - 1, slot = s_slot[i + 1];
      if (slot < 0 || slot >= cap) continue;
      // the next break after i
      int e = i + 1, word = e >> 5;  // (within `look`: e <= 128)
      uint32_t bits = s_break[word] & (0xFFFFFFFFu << (e & 31));
      while (!bits) bits = ++word < 2 * kMaxWindow / 32 ? s_break[word] : 1u;
      e = word * 32 + __ffs(bits) - 1;
      const int n = e - i;
      // a run that has its window to itself and is more than a warp holds: all warps (a prompt among short calls)
      const bool alone = HOLD == kShortHold && only && n * a.d > kShortHold * 256;
#pragma unroll 1
      for (int k = 0; k < pairs; ++k, ++turn) {
        if ((!alone && turn % (kAppWarps / TS) != team) || pair0 + k >= 2 * a.H) continue;
        const bool is_v = pair0 + k >= a.H;
        if (alone) {
          write_run<kAppWarps, HOLD>(a, is_v ? a.v : a.k, is_v ? a.v_stride : a.k_stride, is_v ? a.v_cache : a.k_cache,
                                     is_v ? a.v_scale : a.k_scale, t0 + i, n, slot, is_v ? pair0 + k - a.H : pair0 + k, 0, s_red);
          continue;
        }
        write_run<TS, HOLD>(a, is_v ? a.v : a.k, is_v ? a.v_stride : a.k_stride, is_v ? a.v_cache : a.k_cache,
                            is_v ? a.v_scale : a.k_scale, t0 + i, n, slot, is_v ? pair0 + k - a.H : pair0 + k, team, s_red);
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache_tables(const TablesArgs& a, cudaStream_t s) {
  auto smem_of = [](int B) { return (static_cast<size_t>(B) * 5 + 1) * sizeof(int32_t); };
  const size_t smem = smem_of(a.B);
  if (smem > 48 * 1024) {  // the same for every such call: the limit is the kernel's, whichever thread sets it last
    cudaError_t e = cudaFuncSetAttribute(cache_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem_of(kMaxTableBatch)));
    if (e != cudaSuccess) return e;
  }
  const bool in_place = a.pool_out == a.pool || a.lens == a.lens_old || a.lens == a.lens_new;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.slot_map) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0;
  // CTAs by the tokens (each takes 4 a thread at a time) and the rows; at most one cluster in place
  int grid = (a.total_tokens + 4 * kTabThreads - 1) / (4 * kTabThreads);
  const int by_rows = (a.B + 63) / 64;  // (a row may move hundreds of blocks)
  if (grid < by_rows) grid = by_rows;
  const int most = in_place ? kTabCluster : kTabMost;
  if (grid > most) grid = most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kTabThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = grid;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = in_place ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, cache_tables_kernel, a, static_cast<int>(in_place), static_cast<int>(wide));
}

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  const int all = 2 * a.H;
  if (a.T <= kShortAppend) {
    // a decode step: 8-token windows and one pair a CTA give each row's token a warp of its own
    cache_append_kernel<1, kShortHold><<<dim3((a.T + 7) / 8, all), kAppThreads, 0, s>>>(a, 8, 1);
    return cudaGetLastError();
  }
  // prompts: a window is a block, mostly one run; a team holds a block of a head (8 vectors a lane; of 128 x 256
  // values it reads half again)
  const int size = a.bs * a.d, ts = size >= 16384 ? 8 : size >= 8192 ? 4 : size >= 4096 ? 2 : 1;
  const int pairs = all < kAppWarps / ts ? all : kAppWarps / ts;
  const dim3 grid((a.T + a.bs - 1) / a.bs, (all + pairs - 1) / pairs);
  if (ts == 1) cache_append_kernel<1, 8><<<grid, kAppThreads, 0, s>>>(a, a.bs, pairs);
  else if (ts == 2) cache_append_kernel<2, 8><<<grid, kAppThreads, 0, s>>>(a, a.bs, pairs);
  else if (ts == 4) cache_append_kernel<4, 8><<<grid, kAppThreads, 0, s>>>(a, a.bs, pairs);
  else cache_append_kernel<8, 8><<<grid, kAppThreads, 0, s>>>(a, a.bs, pairs);
  return cudaGetLastError();
}

}  // namespace gdn
