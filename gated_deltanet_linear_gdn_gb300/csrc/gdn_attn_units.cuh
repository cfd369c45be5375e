// gdn_attn_units.cuh -- how the attention of single tokens is cut into units, walked by a persistent grid and joined: what
// the kernels over the 8-bit and the 4-bit cache share. (Everything is local to the file that includes it.)
#pragma once

#include "gdn_attn.cuh"

namespace gdn {

namespace {

// Requests of one launch. Their lengths stay in shared memory, next to what two CTAs an SM of the 8-bit kernel leave of it
// (static_assert there): with 384, batches of 330 to 384 ran one CTA an SM (384 requests of 2,000 tokens, 16 / 2 heads of
// 256: 205 us, and 167 in two launches).
constexpr int kBatchPerLaunch = 320;
constexpr int kCoarse = 16;             // requests between two kept tile sums
constexpr int kSmemPerSm = 228 * 1024;  // 1 KB of it taken by each resident CTA

// The units of a request by its own length: 2^MIN keys each up to FEW units, then 2^(MIN + 1) up to FEW, and so on up to
// 2^MAX, by the length alone and never by the batch.
template <int MIN, int MAX, int FEW>
struct UnitRule {
  __host__ __device__ __forceinline__ static int shift(int len) {  // log2 of the keys of a unit
    int s = MIN;
#pragma unroll
    for (int i = MIN; i < MAX; ++i) s += len > FEW << i;
    return s;
  }
  __host__ __device__ __forceinline__ static int count(int len) {
    const int s = shift(len);
    return (len + (1 << s) - 1) >> s;
  }
  // The most units that any length up to `cap` has.
  static int64_t most(int64_t cap) {
    if (cap <= FEW << MIN) return (cap + (1 << MIN) - 1) >> MIN;
    return cap <= FEW << MAX ? FEW : (cap + (1 << MAX) - 1) >> MAX;
  }
};

struct DecodeParams {
  AttnArgs a;
  int heads;      // query heads of one unit: min(G, 16)
  int chunks;     // units' head chunks per kv head: ceil(G / 16)
  int b0, nb;     // the launch's requests
  int fault;      // test hook: CTA 0 looks up one batch of tiles and no more
  int each;       // the most units of a request's (kv head, chunk): unit u of it has slot (b * HC + hc) * each + u
  float2* ml;     // workspace: [slots][heads] (maximum, sum) of a unit that is one of several
  float* part;    // [slots][heads][D]
};

// The units of one CTA, in order: those whose first tile lies in its equal share of the launch's tiles (all
// requests, kv heads and head chunks end to end). A share holds whole units, so CTAs differ by a unit's
// tiles at most, and neighbours in a CTA are neighbours in memory.
template <class U>
struct WalkOf {
  const int32_t* lens;
  const int32_t* tsum;  // tiles before request kCoarse * i
  int nb, end;
  int H, chunks;
  int b, h, chunk, index;  // request, kv head, head chunk, the unit's place in its (request, head, chunk)
  int len, shift, count;   // the request's keys, log2 of the keys of a unit, units
  int pos;              // the unit's first tile

  __device__ __forceinline__ static int tiles_of(int len) { return (len + kTile - 1) / kTile; }
  __device__ __forceinline__ void request() {
    len = lens[b];
    shift = U::shift(len);
    count = U::count(len);
  }
  __device__ __forceinline__ void next_head() {
    index = 0;
    if (++chunk == chunks) {
      chunk = 0;
      ++h;
    }
    if (h == H) {
      h = 0;
      do ++b;
      while (b < nb && lens[b] == 0);
      if (b == nb) {
        pos = end;
        return;
      }
      request();
    }
  }
  __device__ __forceinline__ void start(int share, int shares) {
    const int HC = H * chunks;
    const int all = tsum[(nb + kCoarse - 1) / kCoarse] * HC, each = all / shares, more = all - each * shares;
    const int from = each * share + min(share, more);
    end = from + each + (share < more);
    pos = from;
    if (from == end) return;
    // the last request whose tiles start at or before `from`: not an empty one
    int lo = 0;
#pragma unroll 1
    while ((lo + 1) * kCoarse < nb && tsum[lo + 1] * HC <= from) ++lo;
    int before = tsum[lo];
    b = lo * kCoarse;
#pragma unroll 1
    while ((before + tiles_of(lens[b])) * HC <= from) before += tiles_of(lens[b++]);
    request();
    const int tiles = tiles_of(len), rem = from - before * HC, ut = shift - 7;  // (a tile is 2^7 keys)
    const int hc = rem / tiles, in = rem - hc * tiles;
    h = hc / chunks;
    chunk = hc - h * chunks;
    index = (in + (1 << ut) - 1) >> ut;
    pos += min(index << ut, tiles) - in;
    if (index == count) next_head();
  }
  __device__ __forceinline__ bool more() const { return pos < end; }
  __device__ __forceinline__ void next() {
    pos += tiles();
    if (++index == count) next_head();
  }
  __device__ __forceinline__ int first() const { return index << shift; }
  __device__ __forceinline__ int keys() const { return min(1 << shift, len - first()); }
  __device__ __forceinline__ int tiles() const { return (keys() + kTile - 1) / kTile; }
};

// Joins the units of one request, kv head and head chunk; an empty request gets zeros. A thread has four d
// of one head. Up to kJoinRows units it takes in order; more are taken by kJoinRows threads, unit u by
// u mod kJoinRows, whose sums are then taken in order (for few units that is the same). Either way the order
// goes by the request's own units.
constexpr int kJoinRows = 16;

struct JoinSum {
  float m = -INFINITY, l = 0.0f;
  float4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  // the root of a unit's weight
  __device__ __forceinline__ static float weight(float m, float l, float top) {
    // a unit without keys has m = -inf, l = 0; with only NaN scores m = -inf, l = NaN
    return m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : ex2_root(m - top);
  }
  __device__ __forceinline__ void add(float2 e, const float4& v) {
    const float top = fmaxf(m, e.x), ra = weight(m, l, top), rb = weight(e.x, e.y, top), wa = ra * ra, wb = rb * rb;
    m = top;
    l = l * ra * ra + e.y * rb * rb;
    o.x = o.x * wa + v.x * wb;
    o.y = o.y * wa + v.y * wb;
    o.z = o.z * wa + v.z * wb;
    o.w = o.w * wa + v.w * wb;
  }
  // units u, u + step, ..
  __device__ __forceinline__ void add_units(const float2* ml, const float4* part, int u, int n, int step, int heads, int d4s) {
    constexpr int kAhead = 4;
#pragma unroll 1
    for (; u < n; u += kAhead * step) {
      float2 e[kAhead];
      float4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (u + i * step < n) {
          const int64_t at = static_cast<int64_t>(u + i * step) * heads;
          e[i] = ml[at];
          v[i] = part[at * d4s];
        }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (u + i * step < n) add(e[i], v[i]);
    }
  }
  __device__ __forceinline__ void store(uint16_t* out) const {
    const float inv = l > 0.0f || l != l ? __fdividef(1.0f, l) : 0.0f;
    uint2 st;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.x) : "f"(o.y * inv), "f"(o.x * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(st.y) : "f"(o.w * inv), "f"(o.z * inv));
    *reinterpret_cast<uint2*>(out) = st;
  }
};

template <int D, class U>
__global__ void __launch_bounds__(256) attn_decode_join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kLanes = D / 4;
  __shared__ float4 s_o[kJoinRows][16];
  __shared__ float2 s_ml[kJoinRows];
  const AttnArgs& a = p.a;
  const int HC = a.H * p.chunks, G = a.Hq / a.H, tid = threadIdx.x;
  const int b = blockIdx.x / HC, hc = blockIdx.x - b * HC, h = hc / p.chunks, chunk = hc - h * p.chunks;
  const int heads = min(p.heads, G - chunk * 16);
  const int n = U::count(min(max(a.lens[p.b0 + b], 0), a.max_blocks * a.bs));
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (by every CTA: this kernel's end stands for the call's)
  if (n == 1 || (n <= kJoinRows && blockIdx.y > 0)) return;
  const int64_t f = static_cast<int64_t>(blockIdx.x) * p.each * p.heads;
  const float2* ml = p.ml + f;
  const float4* part = reinterpret_cast<const float4*>(p.part + f * D);
  uint16_t* out = a.out + (static_cast<int64_t>(p.b0 + b) * a.Hq + h * G + chunk * 16) * D;
  if (n <= kJoinRows) {
#pragma unroll 1
    for (int i = tid; i < heads * kLanes; i += 256) {
      JoinSum sum;
      const int head = i / kLanes;
      sum.add_units(ml + head, part + i, 0, n, 1, p.heads, kLanes);
      sum.store(out + i * 4);
    }
    return;
  }
  const int row = tid / 16, lane = tid % 16;
#pragma unroll 1
  for (int i0 = blockIdx.y * 16; i0 < heads * kLanes; i0 += gridDim.y * 16) {  // 16 lanes of one head
    JoinSum sum;
    const int head = i0 / kLanes;
    sum.add_units(ml + head, part + i0 + lane, row, n, kJoinRows, p.heads, kLanes);
    s_o[row][lane] = sum.o;
    if (lane == 0) s_ml[row] = make_float2(sum.m, sum.l);
    __syncthreads();
    if (row == 0) {
#pragma unroll 1
      for (int i = 1; i < kJoinRows; ++i) sum.add(s_ml[i], s_o[i][lane]);
      sum.store(out + (i0 + lane) * 4);
    }
    __syncthreads();
  }
}

struct DecodeLayout {
  size_t part, total;
};
template <class U>
DecodeLayout decode_layout(int nb, int max_blocks, int Hq, int H, int d, int bs) {
  const int G = Hq / H, heads = G < 16 ? G : 16, chunks = (G + 15) / 16;
  const size_t units = static_cast<size_t>(nb) * H * chunks * U::most(static_cast<int64_t>(max_blocks) * bs);
  DecodeLayout L;
  L.part = (units * heads * 8 + 255) & ~static_cast<size_t>(255);
  L.total = L.part + units * heads * d * 4;
  return L;
}

// The join, a programmatic dependent of the kernel that left the partial sums.
template <int D, class U>
cudaError_t launch_join(const DecodeParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  // where requests may have many units, CTAs enough for all their heads and d
  cfg.gridDim = dim3(p.nb * p.a.H * p.chunks, p.each > kJoinRows ? p.heads * D / 64 : 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_join_kernel<D, U>, p);
}

}  // namespace

}  // namespace gdn
