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
// Bound by latency, not bytes: a step of 64 rows moves 2 KB. So it is ONE launch: every CTA
// computes the prefix sums for itself (three warp scans over the lengths, which stay in
// shared memory) and takes its share of rows and tokens. The only value that is read by all
// and rewritten by one is the pool's head and count (and `lens`, when it is one of the inputs):
// the CTAs form one thread-block cluster and write after its barrier. A token of a block that is
// being handed out reads the ring, not the table, so rows and tokens need no ordering.
//
// cache_append_kernel. Per touched (block, head), with a = max |x| over the finite values of
// the block's new tokens:
//   s = max(s_old if the block held tokens before, a / 448, 2^-64),  byte = e4m3(x * (1 / s))
// and tokens that were there are rewritten as e4m3((byte * s_old) * (1 / s)) if s grew. All in
// IEEE fp32 with one rounding to 8 bits (nearest even, saturating): the bytes are reproducible
// bit for bit. Bound by memory (2 bytes read and 1 written per value): the new values are
// read once, into registers, between the maximum and the rounding.
#include "gdn_cache.cuh"
#include "gdn_ptx.cuh"

namespace gdn {

namespace {

constexpr int kTabThreads = 512;
constexpr int kTabCluster = 8;

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

__device__ __forceinline__ int blocks_of(int len, int bs) { return (len + bs - 1) / bs; }

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

__global__ void __launch_bounds__(kTabThreads) cache_tables_kernel(TablesArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* s_cu = sm;               // [B + 1] tokens before row b (saturated at INT32_MAX)
  int32_t* s_need = sm + a.B + 1;   // [B] blocks taken before row b, or -1: the row is refused
  int32_t* s_give = s_need + a.B;   // [B] blocks given back before row b
  int32_t* s_old = s_give + a.B;    // [B]
  int32_t* s_new = s_old + a.B;     // [B]
  __shared__ Sum3 s_warp[kTabThreads / 32];
  __shared__ long long s_taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, nrank = gridDim.x;
  int head = a.pool[0], count = a.pool[1];
  const int bs = a.block_size;
  const int N = a.num_blocks;
  if (tid == 0) s_taken = 0;
  int flags = 0;
  if (head < 0 || head >= N || count < 0 || count > N) {  // no such pool: nothing to hand out
    head = count = 0;
    flags = GDN_DEVERR_BLOCKS;
  }
  Sum3 carry{0, 0, 0};
  for (int base = 0; base < a.B; base += kTabThreads) {
    const int b = base + tid;
    int o = 0, n = 0;
    if (b < a.B && !row_lens(a, b, o, n)) flags |= GDN_DEVERR_SEQLENS;
    const int no = blocks_of(o, bs), nn = blocks_of(n, bs);
    const int need = max(nn - no, 0), give = max(no - nn, 0);
    Sum3 v{need, give, max(n - o, 0)};
    const Sum3 inc = warp_scan(v, lane);
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
      Sum3 w = lane < kTabThreads / 32 ? s_warp[lane] : Sum3{0, 0, 0};
      const Sum3 wi = warp_scan(w, lane);
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
      if (need > 0 && !refused) atomicMax(reinterpret_cast<unsigned long long*>(&s_taken),
                                          static_cast<unsigned long long>(upto));
      s_need[b] = refused ? -1 : static_cast<int32_t>(upto - need);
      s_give[b] = static_cast<int32_t>(before.give + inc.give - give);
      const long long cu = before.tok + inc.tok;
      s_cu[b + 1] = static_cast<int32_t>(min(cu, 0x7fffffffLL));
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
  if (nrank > 1) {
    cluster_arrive();
    cluster_wait();
  }
  if (carry.tok > a.total_tokens) flags |= GDN_DEVERR_SEQLENS;
  if (rank == 0 && tid == 0) {
    const long long taken = s_taken;
    a.pool_out[0] = static_cast<int32_t>((head + taken) % N);
    a.pool_out[1] = static_cast<int32_t>(count - taken + carry.give);
    a.cu_tokens[0] = 0;
  }
  if (flags != 0 && a.err) atomicOr(a.err, flags);

  // rows: the sums, the lengths, and the blocks that change hands
  const int gw = rank * (kTabThreads / 32) + warp, ngw = nrank * (kTabThreads / 32);
  for (int b = rank * kTabThreads + tid; b < a.B; b += nrank * kTabThreads) {
    a.cu_tokens[b + 1] = s_cu[b + 1];
    a.lens[b] = s_need[b] < 0 ? s_old[b] : s_new[b];
  }
  for (int b = gw; b < a.B; b += ngw) {
    const int no = blocks_of(s_old[b], bs), nn = blocks_of(s_new[b], bs);
    int32_t* row = a.block_table + static_cast<int64_t>(b) * a.max_blocks;
    const int64_t first = s_need[b];
    if (nn > no && first >= 0)
      for (int j = lane; j < nn - no; j += 32) row[no + j] = a.ring[(head + first + j) % N];
    const int64_t tail = static_cast<int64_t>(head) + count + s_give[b];
    for (int j = lane; j < no - nn; j += 32) a.ring[(tail + j) % N] = row[nn + j];
  }
  // tokens
  const int real = min(s_cu[a.B], a.total_tokens);
  for (int t = rank * kTabThreads + tid; t < a.total_tokens; t += nrank * kTabThreads) {
    int slot = -1, pos = -1;
    if (t < real) {
      int lo = 0, hi = a.B - 1;  // the last row that starts at or before t and is not empty
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_cu[mid] <= t) lo = mid; else hi = mid - 1;
      }
      pos = s_old[lo] + t - s_cu[lo];
      const int first = s_need[lo];
      if (first >= 0) {
        const int no = blocks_of(s_old[lo], bs), i = pos / bs;
        const int blk = i < no ? a.block_table[static_cast<int64_t>(lo) * a.max_blocks + i]
                               : a.ring[(static_cast<int64_t>(head) + first + i - no) % N];
        slot = blk * bs + pos % bs;
      }
    }
    a.slot_map[t] = slot;
    a.positions[t] = pos;
  }
}

// ------------------------------------------------------------------------------- cache writer

constexpr int kAppThreads = 256;
constexpr int kAppWarps = kAppThreads / 32;

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

// max |x| over the finite values of 8 bf16: as integers, |x| orders like its bits and every
// non-finite value lies at or above 0x7F80
__device__ __forceinline__ uint32_t amax8(const uint4& u, uint32_t m) {
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

// A run: consecutive tokens [t, t + n) that fill offsets [off, off + n) of one block. The warp's
// lanes look at the slots after t, 32 at a time.
__device__ __forceinline__ int run_length(const int32_t* slot_map, int T, int t, int slot, int bs, int lane) {
  const int most = bs - slot % bs;
  int n = 0;
  while (n < most) {
    const int i = n + lane;
    const bool in = i < most && t + i < T && slot_map[t + i] == slot + i;
    const uint32_t miss = ~__ballot_sync(0xFFFFFFFFu, in);
    if (miss) return n + __ffs(miss) - 1;
    n += 32;
  }
  return n;
}

// One run of one head's keys or values. NT threads (a warp or the CTA) work on it; each value is
// held in registers between the maximum and the rounding when the run fits kHold 16-byte
// vectors per thread, and read again (from L1 / L2) beyond that.
constexpr int kHold = 4;

template <bool kCta>
__device__ __forceinline__ void write_run(const AppendArgs& a, const uint16_t* x, int64_t stride,
                                          uint8_t* cache, float* scales, int t, int n, int slot,
                                          int h, int lane_id, uint32_t* s_red) {
  constexpr int NT = kCta ? kAppThreads : 32;
  const int vec = a.d >> 3;  // 16-byte vectors per token
  const int total = n * vec;
  const int blk = slot / a.bs, off = slot % a.bs;
  const uint16_t* src = x + static_cast<int64_t>(t) * stride + static_cast<int64_t>(h) * a.d;
  float* sp = scales + static_cast<int64_t>(blk) * a.H + h;
  const float s_was = off > 0 ? *sp : 0.0f;  // a block that held no token has no scale yet
  uint4 held[kHold];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int e = lane_id + i * NT;
    if (e < total) held[i] = *reinterpret_cast<const uint4*>(src + (e / vec) * stride + (e % vec) * 8);
  }
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (lane_id + i * NT < total) m = amax8(held[i], m);
  for (int e = lane_id + kHold * NT; e < total; e += NT)
    m = amax8(*reinterpret_cast<const uint4*>(src + (e / vec) * stride + (e % vec) * 8), m);
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (kCta) {
    if ((lane_id & 31) == 0) s_red[lane_id >> 5] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int i = 0; i < kAppWarps; ++i) m = max(m, s_red[i]);
  }
  const float amax = __uint_as_float(m << 16);
  const float s = fmaxf(fmaxf(__fmul_rn(amax, 1.0f / kE4m3Max), s_was), kCacheMinScale);
  const float r = __fdiv_rn(1.0f, s);
  uint8_t* dst = cache + (static_cast<int64_t>(blk) * a.H + h) * a.bs * a.d;
  uint8_t* put = dst + static_cast<int64_t>(off) * a.d;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int e = lane_id + i * NT;
    if (e < total) *reinterpret_cast<uint2*>(put + static_cast<int64_t>(e) * 8) = quant8(held[i], r);
  }
  for (int e = lane_id + kHold * NT; e < total; e += NT)
    *reinterpret_cast<uint2*>(put + static_cast<int64_t>(e) * 8) =
        quant8(*reinterpret_cast<const uint4*>(src + (e / vec) * stride + (e % vec) * 8), r);
  if (off > 0 && s != s_was) {  // the tokens before: same values under the larger scale
    const int words = off * a.d / 16;
    for (int e = lane_id; e < words; e += NT) {
      uint4* p = reinterpret_cast<uint4*>(dst) + e;
      const uint4 w = *p;
      *p = make_uint4(rescale4(w.x, s_was, r), rescale4(w.y, s_was, r), rescale4(w.z, s_was, r),
                      rescale4(w.w, s_was, r));
    }
  }
  if (kCta) __syncthreads();  // the old scale has been read by all
  else __syncwarp();
  if (lane_id == 0) *sp = s;
}

// grid: (windows of W tokens, heads, keys / values). The runs that start in the CTA's window
// are its work: with one or two (a prompt) the whole CTA takes each, with more (decode rows:
// a run per token) each warp takes its own.
template <int W>
__global__ void __launch_bounds__(kAppThreads) cache_append_kernel(AppendArgs a) {
  __shared__ uint32_t s_red[kAppWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * W, h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  // every warp finds the window's run starts for itself: bit i for token t0 + i
  const int t = t0 + lane;
  const bool mine = lane < W && t < a.T;
  const int slot = mine ? a.slot_map[t] : -1;
  const int64_t cap = static_cast<int64_t>(a.num_blocks) * a.bs;
  const bool bad = mine && slot >= cap;
  int prev = __shfl_up_sync(0xFFFFFFFFu, slot, 1);
  if (lane == 0) prev = t0 > 0 && t0 < a.T ? a.slot_map[t0 - 1] : -1;
  const bool starts = mine && slot >= 0 && !bad && (slot % a.bs == 0 || prev < 0 || slot != prev + 1);
  if (bad && a.err && warp == 0) atomicOr(a.err, GDN_DEVERR_BLOCK_RANGE);
  uint32_t runs = __ballot_sync(0xFFFFFFFFu, starts);
  const uint16_t* x = is_v ? a.v : a.k;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  uint8_t* cache = is_v ? a.v_cache : a.k_cache;
  float* scales = is_v ? a.v_scale : a.k_scale;
  const bool by_cta = __popc(runs) <= 2;
  for (int i = 0; runs; ++i, runs &= runs - 1) {
    if (!by_cta && i % kAppWarps != warp) continue;
    const int at = __ffs(runs) - 1;
    const int s0 = __shfl_sync(0xFFFFFFFFu, slot, at);
    const int n = run_length(a.slot_map, a.T, t0 + at, s0, a.bs, lane);
    if (by_cta) write_run<true>(a, x, stride, cache, scales, t0 + at, n, s0, h, threadIdx.x, s_red);
    else write_run<false>(a, x, stride, cache, scales, t0 + at, n, s0, h, lane, s_red);
  }
}

}  // namespace

cudaError_t launch_cache_tables(const TablesArgs& a, cudaStream_t s) {
  const size_t smem = (static_cast<size_t>(a.B) * 5 + 1) * sizeof(int32_t);
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(cache_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  // One CTA while a pass of its threads covers the step; a cluster beyond that.
  const int grid = a.B <= kTabThreads && a.total_tokens <= 4 * kTabThreads ? 1 : kTabCluster;
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
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_tables_kernel, a);
}

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  // 8-token windows give a decode step a warp per row; long batches are prompts, whose runs
  // are at least a block of 16 tokens long
  if (a.T <= 4096) {
    cache_append_kernel<8><<<dim3((a.T + 7) / 8, a.H, 2), kAppThreads, 0, s>>>(a);
  } else {
    cache_append_kernel<16><<<dim3((a.T + 15) / 16, a.H, 2), kAppThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace gdn
