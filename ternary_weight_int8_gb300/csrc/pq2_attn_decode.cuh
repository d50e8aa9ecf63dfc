// pq2_attn_decode.cuh — attention of the newest tokens over a paged cache.
//
// Per row (a token's query head), with scores s_j = c q . k_j (c = scale /
// ln 2) over the positions that it sees, out = sum 2^(s_j - m) v_j / sum
// 2^(s_j - m), m a running maximum of the scores seen so far, or at most 8
// below it.
//
// Bound: HBM, the cache is read once.  The T * G rows of the query heads that
// share a key head are taken together, so every key and value is used for all
// of them: the products are m16n8k16 MMAs with the keys, and the values
// transposed, as their 16 rows and 8 query rows as their columns (scores^T = K
// Q^T, out^T = V^T W^T), so that few rows leave little of them empty.
//
// Work is cut evenly whatever the lengths: the tiles of 64 to 384 tokens of
// all (sequence, key head, row tile) are numbered, and a CTA takes a
// contiguous share of them, which may end inside a sequence and span several.
// Inside a tile each warp has 16 or 32 tokens of its own, which it copies itself
// (tensor-map boxes of 16 slots into a ring that no other warp touches, so
// nothing waits for another warp before the join; many rows of 256 columns: two
// or three warps with rows of their own share them) and folds into sums of its
// own.  At the end of a CTA's part of a sequence the warps join; parts that
// are not whole go to the workspace, and a second kernel joins them.  Short tables
// with few items: a CTA or a cluster an item, joined in distributed shared memory.
//
// 8-bit caches: codes become fp16 by byte permutes (0x6400 | code + 128 is
// 1024 + 128 + code) and one exact subtraction.  A key's scale multiplies its
// score; a value's goes into its weight, w_j = 2^(s_j - m - u) scale_j with a
// unit 2^u of its own beside 2^m, so that weights are at most 2^8 and keep their
// bits whatever the scales are.  u is held relative to m, as large maxima have no
// bits for it.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "pq2_internal.h"
#include "pq2_tensor.cuh"

namespace pq2 {

// What a launch of the kernels is about.
struct AttnDecode {
  DecodeParams a;
  pq2_kv_cache cache;
  int group, rows, row_groups, items;  // G, T * G, groups of Geo::rows, heads * row_groups
  float c;
  float* parts;   // [2 * CTAs][slot]
  int4* places;   // [CTAs]: sequence, item, first CTA, number of parts (0: nothing to join)
  int cluster;    // CTAs that share an item and join it themselves; 0: even shares
};

int launch_attn_decode8(AttnDecode& p, int sm_count, cudaStream_t stream);

namespace {

constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;   // how far m may stay behind, in powers of two
// How far below 2^m the unit of an 8-bit cache's sums may lie: 2^(s_j - m - u) stays
// finite, and what the sums lose when the unit moves up to there is below
// 2^-149 of 2^(m - kLead).
constexpr float kLead = 118.f;
constexpr int kBlock = 8;       // query rows of an MMA
constexpr int kMaxCtas = 160;   // the SMs of the largest sm_103 device
constexpr int kCluster = 8;     // CTAs that share an item at most, without a workspace
constexpr int kScaleBytes = 128;  // of 16 scales: a copy's target is 128-byte aligned

// A warp has NB blocks of 8 rows.  RT warps share a slice of tokens, each with
// rows of its own.
template <typename CT, int D, int RT, int NB>
struct Geo {
  static constexpr bool eight = sizeof(CT) == 1;
  static constexpr int warps = RT == 3 || (eight && D <= 128 && NB <= 2) ? 12 : 8, slices = warps / RT;
  static constexpr int threads = warps * 32;
  // Tokens of a slice: 32 share the steps between the MMAs where a thread's
  // registers and the ring have room for them.
  static constexpr int boxes16 = NB < 4 && (eight || D <= 128) ? 2 : 1, tokens = 16 * boxes16;
  static constexpr int tile = slices * tokens;      // tokens that a CTA takes at a time
  static constexpr int rowBytes = D * (int)sizeof(CT);
  static constexpr int boxBytes = rowBytes < 128 ? rowBytes : 128;
  static constexpr int boxes = rowBytes / boxBytes;  // of 16 tokens
  static constexpr int sixteen = 16 * rowBytes;      // bytes of 16 tokens
  static constexpr int unit = boxes16 * sixteen;     // a slice's K, or its V
  static constexpr int warpRows = NB * kBlock, rows = RT * warpRows;
  // The warps' join takes joinCols columns at a time; the stride puts the four
  // pairs of rows that a store touches on other banks.
  static constexpr int joinCols = NB == 1 ? 64 : 32, joinStride = joinCols + 4;
  static constexpr int joinBytes = warps * warpRows * joinStride * 4;
  static constexpr int qBytes = RT * NB * (D / 32) * 512;
  static constexpr int statBytes = 3 * warps * warpRows * 4;
  // What beginning an item costs (its queries, the join), in tiles: about the
  // time of 96 KB.  Without it shares of many short sequences took longer than the
  // rest: 32 ragged ones of up to 8192 over 8 bits 102 us, the same number of
  // tokens in equal ones 73 us.
  static constexpr int begin = (98304 + tile * rowBytes * 2 - 1) / (tile * rowBytes * 2);
  static constexpr int scale = eight ? boxes16 * kScaleBytes : 0;  // of a unit
  static constexpr int depth =
      std::min(8, (227 * 1024 - 1024 - 1024 - joinBytes - qBytes - statBytes) /
                      ((unit + scale) * slices));
  static constexpr int offScale = slices * depth * unit;
  static constexpr int offJoin = offScale + slices * depth * scale;
  static constexpr int offQ = offJoin + joinBytes;
  static constexpr int offStat = offQ + qBytes;       // [3][warps][warpRows]
  static constexpr int offBar = offStat + statBytes;
  static constexpr int smem = offBar + 2 * slices * depth * 8 + 1024;
  static_assert(smem <= 227 * 1024 && depth >= 2, "shared memory");
  static_assert(offJoin % 128 == 0 && offQ % 16 == 0 && offBar % 8 == 0, "alignment");
  static_assert(rows * joinCols / 4 <= threads, "the join's threads");
  static constexpr int slot = rows * D + 3 * rows;  // floats of a part in the workspace
};

using Params = AttnDecode;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 2^(m - top), 0 for the maximum of nothing.
__device__ __forceinline__ float weight(float m, float top) {
  return m == -INFINITY ? 0.f : ex2(m - top);
}
// The exponent of the unit of sums beside a maximum m, counted from M >= m: u over
// an 8-bit cache, 0 over others; -infinity where nothing has been summed.
template <typename CT>
__device__ __forceinline__ float unit_from(float m, float u, float M) {
  if (sizeof(CT) == 1) return u == -INFINITY ? u : m - M + u;
  return m == -INFINITY ? m : m - M;
}

template <typename T> __device__ __forceinline__ uint32_t pack(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <> __device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(int8_t x) { return (float)x; }

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float (&d)[4], const uint4& a, uint32_t b0,
                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&d)[4], const uint4& a, uint32_t b0,
                                                   uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 ldsm(uint32_t addr) {
  uint4 r;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}
__device__ __forceinline__ uint4 ldsm_t(uint32_t addr) {
  uint4 r;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}
// Eight elements with zeros in the place of infinities and NaN.
template <typename T>
__device__ __forceinline__ uint4 finite(uint4 x) {
  constexpr uint32_t kTop = std::is_same<T, __half>::value ? 0x7C007C00u : 0x7F807F80u;
  const auto pair = [](uint32_t y) { return y & ~__vcmpeq2(y & kTop, kTop); };
  return make_uint4(pair(x.x), pair(x.y), pair(x.z), pair(x.w));
}
// The transpose of an 8 x 8 matrix of 16-bit elements, a pair of a row a lane.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// The larger one, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Codes x and y (bytes X and Y of u, already 128 above) as fp16 pairs.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes(uint32_t u) {
  const uint32_t h = __byte_perm(u, 0x64646464u, SEL);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h),
                            __half2half2(__ushort_as_half(0x6480)));  // 1152
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                       int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                       uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// An address of this CTA's shared memory in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float remote(uint32_t addr) {
  float r;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ float4 remote4(uint32_t addr) {
  float4 r;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
               : "r"(addr));
  return r;
}

__device__ __forceinline__ int length(const Params& p, int b) {
  return b < p.a.batch.B ? min(max(__ldg(p.a.batch.lens + b), 0), 1 << 30) : 0;
}
__device__ __forceinline__ int tiles_of(int len, int tile) {
  return max(1, len / tile + (len % tile != 0));
}

// Where a CTA, or one of its warps' copies, is in the CTA's share.
struct Cursor {
  int b, head, group, tile, tiles, len, next_len, left;
};
template <int TILE, int BEGIN>
__device__ __forceinline__ void next_tile(Cursor& c, const Params& p) {
  --c.left;
  if (++c.tile < c.tiles) return;
  c.tile = 0, c.left -= BEGIN;
  if (++c.group < p.row_groups) return;
  c.group = 0;
  if (++c.head < (int)p.cache.heads) return;
  c.head = 0, ++c.b;
  c.len = c.next_len;
  c.tiles = tiles_of(c.len, TILE);
  c.next_len = length(p, c.b + 1);
}

// Four columns of a joined row to out, and its lse: o in units of 2^(m + u), the
// weights' sum l in units of 2^m.
template <typename QT, typename CT, int D>
__device__ __forceinline__ void finish(const Params& p, int b, int kh, int R, int d, int len,
                                       float4 o, float m, float l, float u) {
  if (R >= p.rows) return;
  const int t = R / p.group, most = len - p.a.T + t + 1;
  const int64_t row =
      ((int64_t)b * p.a.T + t) * p.a.q_heads + kh * p.group + R % p.group;
  if (most <= 0) {
    o = make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    const float f = (sizeof(CT) == 1 ? ex2(u) : 1.f) / l;
    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
  }
  *reinterpret_cast<uint2*>(static_cast<QT*>(p.a.out) + row * D + d) =
      make_uint2(pack<QT>(o.x, o.y), pack<QT>(o.z, o.w));
  if (d == 0 && p.a.lse) p.a.lse[row] = most > 0 ? m * kLn2 + logf(l) : -INFINITY;
}

template <typename QT, typename CT, int D, int RT, int NB>
__global__ void __launch_bounds__(Geo<CT, D, RT, NB>::threads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ CUtensorMap map_ks,
                  const __grid_constant__ CUtensorMap map_vs, const Params p) {
  using G = Geo<CT, D, RT, NB>;
  constexpr int W = G::warps, kTile = G::tile, kTokens = G::tokens, MT16 = kTokens / 16;
  constexpr bool kEight = G::eight;
  using MT = typename std::conditional<kEight, __half, QT>::type;  // the MMAs' type
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_s + 1023u) & ~1023u) - raw_s);
  float* join = reinterpret_cast<float*>(smem + G::offJoin);
  uint4* q_frag = reinterpret_cast<uint4*>(smem + G::offQ);
  float* stat = reinterpret_cast<float*>(smem + G::offStat);  // m, l, u of [warp][row]
  constexpr int kWarpRows = G::warpRows;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + G::offBar);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, i4 = lane & 3;  // fragment row and column pair
  const int slice = warp % G::slices, rt = warp / G::slices;
  uint64_t* bar = bars + slice * G::depth;           // a unit has arrived
  uint64_t* freed = bar + G::slices * G::depth;      // all row tiles have read it
  if (rt == 0 && lane == 0) {
    for (int i = 0; i < G::depth; ++i) mbar_init(&bar[i], 1), mbar_init(&freed[i], RT);
    fence_barrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // The CTA's share: the tiles of all items are counted, with G::begin more in
  // front of each item's, then the sequence that holds the first of the share
  // is found.
  Cursor here;
  int parts = 1, rank = 0;  // of a cluster's item
  if (p.cluster) {
    const int of = blockIdx.x / p.cluster;
    rank = blockIdx.x % p.cluster;
    here.b = of / p.items;
    here.head = of % p.items / p.row_groups, here.group = of % p.items % p.row_groups;
    here.len = length(p, here.b), here.next_len = 0;
    here.tiles = tiles_of(here.len, kTile);
    parts = min(here.tiles, p.cluster);
    here.tile = rank < parts ? (int)((int64_t)rank * here.tiles / parts) : 0;
    here.left = rank < parts ? (int)((int64_t)(rank + 1) * here.tiles / parts) - here.tile : 0;
    __syncthreads();
  } else {
    uint64_t* sums = reinterpret_cast<uint64_t*>(join);   // [W], then the place
    int* place = reinterpret_cast<int*>(sums + W);
    uint64_t total = 0;
    for (int b = tid; b < p.a.batch.B; b += G::threads) total += tiles_of(length(p, b), kTile) + G::begin;
#pragma unroll
    for (int o = 16; o; o /= 2) total += __shfl_xor_sync(~0u, total, o);
    if (lane == 0) sums[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) total += sums[w];
    total *= p.items;
    const uint64_t ctas = min((uint64_t)gridDim.x, total), c = blockIdx.x;
    if (c >= ctas) {
      if (tid == 0) p.places[c] = make_int4(0, 0, 0, 0);
      return;
    }
    const uint64_t t0 = c * total / ctas, t1 = (c + 1) * total / ctas;
    uint64_t before = 0;
    for (int b0 = 0; b0 < p.a.batch.B; b0 += G::threads) {
      const int b = b0 + tid;
      const uint64_t n =
          b < p.a.batch.B ? (uint64_t)(tiles_of(length(p, b), kTile) + G::begin) * p.items : 0;
      uint64_t upto = n;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const uint64_t x = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += x;
      }
      __syncthreads();
      if (lane == 31) sums[warp] = upto;
      __syncthreads();
      uint64_t sum = before;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (w < warp) upto += sums[w];
        sum += sums[w];
      }
      upto += before;
      if (t0 >= upto - n && t0 < upto) {
        const uint64_t in = t0 - (upto - n);
        const int tiles = (int)(n / p.items);
        place[0] = b, place[1] = (int)(in / tiles), place[2] = (int)(in % tiles);
      }
      before = sum;
      if (t0 < sum) break;
    }
    __syncthreads();
    const int in = place[2];  // place in the item
    here.b = place[0], here.tile = max(in - G::begin, 0);
    here.head = place[1] / p.row_groups, here.group = place[1] % p.row_groups;
    here.len = length(p, here.b), here.next_len = length(p, here.b + 1);
    here.tiles = tiles_of(here.len, kTile);
    here.left = (int)(t1 - t0) - max(G::begin - in, 0);
    // If the share begins inside an item, and no share before it does, the
    // second kernel's CTA of this number joins that item.
    if (tid == 0) {
      int4 to = make_int4(0, 0, 0, 0);
      if (here.tile > 0) {
        const uint64_t a = t0 - here.tile, z = a + here.tiles - 1;
        const uint64_t c0 = ((a + 1) * ctas - 1) / total, c1 = ((z + 1) * ctas - 1) / total;
        if (c0 + 1 == c) to = make_int4(here.b, place[1], (int)c0, (int)(c1 - c0 + 1));
      }
      p.places[c] = to;
    }
    __syncthreads();
  }

  // ------------------------------------------------------------- the copies
  bool ok = true;
  uint8_t* ring_p = smem + slice * (G::depth * G::unit);
  const uint32_t ring = smem_u32(ring_p);
  uint8_t* scale_p = smem + G::offScale + slice * (G::depth * G::scale);
  Cursor copy = here;
  uint32_t issued = 0, used = 0;  // units: K and V of a slice in turn
  // Lane i: page and slot of 16 tokens, those of the slice in the tiles from
  // pages_tile on, in order.
  constexpr int kAhead = 32 / G::boxes16;
  int pages = 0, slots = 0, pages_b = -1, pages_tile = 0;
  // To the slice's next tile that holds a token.
  const auto seek = [&]() {
    while (copy.left > 0 && copy.tile * kTile + slice * kTokens >= copy.len)
      next_tile<kTile, G::begin>(copy, p);
    if (copy.left > 0 && (copy.b != pages_b || copy.tile < pages_tile ||
                          copy.tile >= pages_tile + kAhead)) {
      pages_b = copy.b, pages_tile = copy.tile;
      const int page_size = (int)p.cache.page_size, tile = copy.tile + lane / G::boxes16;
      pages = -1, slots = 0;
      if (tile < copy.tiles) {
        const int token = tile * kTile + slice * kTokens + lane % G::boxes16 * 16;
        const int at = token / page_size;
        slots = token - at * page_size;
        if (at < p.a.batch.table_width)
          pages = __ldg(p.a.batch.table + copy.b * p.a.batch.table_stride + at);
      }
    }
  };
  // The next unit's copies; where RT warps share the slice, the first of them
  // makes them when all have read what the ring holds there.
  const auto issue = [&]() {
    if (copy.left <= 0) return;
    const uint32_t st = issued % G::depth;
    if (RT > 1 && rt == 0 && issued >= G::depth)
      ok = ok && mbar_wait(&freed[st], (issued / G::depth - 1) & 1);
    const int from = (copy.tile - pages_tile) * G::boxes16;
    int page[G::boxes16], slot[G::boxes16];
#pragma unroll
    for (int k = 0; k < G::boxes16; ++k) {
      page[k] = __shfl_sync(~0u, pages, from + k);
      slot[k] = __shfl_sync(~0u, slots, from + k);
    }
    if (rt == 0 && lane == 0 && ok) {  // no more copies once a wait has given up
      const bool values = issued & 1;
      const uint32_t mb = smem_u32(&bar[st]);
      mbar_arrive_expect_tx(&bar[st], G::unit + (kEight ? kTokens * 4 : 0));
#pragma unroll
      for (int k = 0; k < G::boxes16; ++k) {
#pragma unroll
        for (int x = 0; x < G::boxes; ++x)
          tma_4d(ring + st * G::unit + k * G::sixteen + x * (16 * G::boxBytes),
                 values ? &map_v : &map_k, x * (G::boxBytes / (int)sizeof(CT)), slot[k], copy.head,
                 page[k], mb);
        if (kEight)
          tma_3d(smem_u32(scale_p) + st * G::scale + k * kScaleBytes, values ? &map_vs : &map_ks,
                 slot[k], copy.head, page[k], mb);
      }
    }
    if (issued & 1) {
      next_tile<kTile, G::begin>(copy, p);
      seek();
    }
    ++issued;
  };
  // The warp has read the unit in use.
  const auto release = [&]() {
    __syncwarp();
    if (RT > 1) warp_arrive(&freed[used % G::depth]);
    issue();
    ++used;
  };
  seek();
  // Where warps share a slice, one less: a unit's place is then filled again when
  // the next one has been read, which the others have mostly done too.
#pragma unroll 1
  for (int i = 0; i < G::depth - (RT > 1); ++i) issue();

  // Lane addresses inside 16 tokens of a unit.  An A fragment's matrices are
  // (rows 0-7 and 8-15) x (columns 0-7 and 8-15), the second half of the rows
  // after the first.  16 bits: K's rows are tokens; V is read transposed, its
  // rows are columns.  8 bits: 16 codes of a token are one row of a matrix, so
  // that one read gives both halves of two steps.  Pieces of 16 bytes are
  // swizzled as the copies left them.
  const int low = (lane & 7) + (lane >> 3 & 1) * 8, high = lane >> 4;
  const auto lane_base = [&](int token, int piece) {
    const int turn = G::boxBytes == 128 ? token & 7 : token >> 1 & 3;
    return (uint32_t)(token * G::boxBytes + ((piece ^ turn) << 4));
  };
  const uint32_t at_k = lane_base(low, high);
  const uint32_t at_v = kEight ? at_k : lane_base((lane & 7) + high * 8, lane >> 3 & 1);
  // The lane's piece pair i of 16 tokens.
  const auto piece = [&](uint32_t base, uint32_t at, int i) {
    constexpr int kPairs = G::boxBytes / 32;
    return base + i / kPairs * (16 * G::boxBytes) + (at ^ (i % kPairs << 5));
  };

  // ------------------------------------------------------- the rows' queries
  // B fragments of two steps: row g of a block, columns of step i: 16 bits 16 i
  // + 2 i4 + {0, 1, 8, 9}; 8 bits 16 i + 4 i4 + {0 .. 3}, the order of a code
  // word.
  const auto fetch_q = [&](const Cursor& at) {
    constexpr int kFrags = D / 32 * 32;  // of a block
    for (int f = tid; f < RT * NB * kFrags; f += G::threads) {
      const int fl = f & 31, pair = f % kFrags >> 5;
      const int R = at.group * G::rows + f / kFrags * kBlock + (fl >> 2);
      const QT* q = static_cast<const QT*>(p.a.q);
      if (R < p.rows)
        q += at.b * p.a.batch_stride + R / p.group * p.a.token_stride +
             (at.head * p.group + R % p.group) * p.a.head_stride;
      const uint32_t to = smem_u32(q_frag + f), bytes = R < p.rows ? 4 : 0;  // else zeros
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int d = R < p.rows ? pair * 32 + (fl & 3) * (kEight ? 4 : 2) + x / 2 * 16 +
                                       x % 2 * (kEight ? 2 : 8)
                                 : 0;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 4 * x), "l"(q + d),
                     "r"(bytes)
                     : "memory");
      }
    }
  };
  if (here.left > 0) fetch_q(here);

  while (here.left > 0) {
    const int first = here.tile, last = min(here.tiles, here.tile + here.left);
    const int b = here.b, head = here.head, len = here.len, R0 = here.group * G::rows;
    const bool whole = first == 0 && last == here.tiles;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // The thread's query rows, columns of the MMAs: 8 nb + 2 i4 + {0, 1}.
    const int row0 = rt * kWarpRows + 2 * i4;
    const uint4* mine_q = q_frag + rt * (NB * D) + lane;  // [nb][D / 32][32]
    float c[NB][2];
    int most[NB][2];  // how many positions they see
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        c[nb][e] = p.c;
        most[nb][e] = len - p.a.T + (R0 + row0 + nb * kBlock + e) / p.group + 1;
      }
    if constexpr (kEight && !std::is_same<QT, __half>::value) {
      // bf16 queries as fp16: scaled by a power of two so that the row's
      // largest lies in [2^14, 2^15); what fp16 loses lies 2^-39 below that.
      float up[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        uint32_t top = 0;  // a pair of magnitudes of row g
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 a = mine_q[(nb * (D / 32) + i) * 32];
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu),
                                       __vmaxu2(a.z & 0x7FFF7FFFu, a.w & 0x7FFF7FFFu)));
        }
        top = __vmaxu2(top, __shfl_xor_sync(~0u, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(~0u, top, 2));
        // The scale's exponent; that of 1 for rows of zeros or infinities.
        int e = (int)(max(top & 0xFFFFu, top >> 16) >> 7);
        e = e == 0 || e == 255 ? 127 : min(max(268 - e, 1), 253);
        up[nb] = __uint_as_float((uint32_t)e << 23);
        const float down = __uint_as_float((uint32_t)(254 - e) << 23);
        c[nb][0] *= __shfl_sync(~0u, down, 8 * i4), c[nb][1] *= __shfl_sync(~0u, down, 8 * i4 + 4);
      }
      const auto scaled = [](uint32_t x, float by) {
        return pack<__half>(__uint_as_float(x << 16) * by, __uint_as_float(x & 0xFFFF0000u) * by);
      };
      __syncthreads();
      uint4* out_q = q_frag + rt * (NB * D) + lane;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        for (int i = slice; i < D / 32; i += G::slices) {
          uint4& a = out_q[(nb * (D / 32) + i) * 32];
          a = make_uint4(scaled(a.x, up[nb]), scaled(a.y, up[nb]), scaled(a.z, up[nb]),
                         scaled(a.w, up[nb]));
        }
      __syncthreads();
    }

    // out^T: columns of out 16 i + g (+ 8) (8 bits: 16 i + 2 g (+ 1)) in o[i],
    // for the rows above.
    float o[D / 16][NB][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][nb][e] = 0.f;
    float m[NB][2], l[NB][2];
    float u[NB][2], ratio[NB][2];  // 8-bit caches: u, and 2^-u
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        m[nb][e] = u[nb][e] = -INFINITY, l[nb][e] = 0.f, ratio[nb][e] = 1.f;
    const auto rescale = [&](const float (&f)[NB][2]) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][nb][e] *= f[nb][e & 1];
    };
    // The largest of a row over the lanes that hold its tokens.
    const auto over_tokens = [](float x) {
      x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
      x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
      return fmaxf(x, __shfl_xor_sync(~0u, x, 16));
    };
#pragma unroll 1
    for (int tile = first; tile < last; ++tile) {
      const int token = tile * kTile + slice * kTokens;
      if (token >= len) continue;
      // ------------------------------------------------------------- scores
      uint32_t st = used % G::depth;
      ok = ok && mbar_wait(&bar[st], used / G::depth & 1);
      uint32_t from = ring + st * G::unit;
      const float* scales = reinterpret_cast<const float*>(scale_p + st * G::scale) + g;
      // Tokens 16 t + g (elements 0, 1) and + 8 (2, 3).  Where they are few, two
      // sums of each, for chains of MMAs half as long.
      constexpr bool kTwo = MT16 * NB <= 2;
      float s[MT16][NB][4] = {}, s2[kTwo ? MT16 : 1][kTwo ? NB : 1][4] = {};
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint4 q[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) q[nb] = mine_q[(nb * (D / 32) + i) * 32];
#pragma unroll
        for (int t = 0; t < MT16; ++t) {
          uint4 a, a2;
          if constexpr (kEight) {
            uint4 k = ldsm(piece(from + t * G::sixteen, at_k, i));
            k.x ^= 0x80808080u, k.y ^= 0x80808080u, k.z ^= 0x80808080u, k.w ^= 0x80808080u;
            a = make_uint4(codes<0x4140>(k.x), codes<0x4140>(k.y), codes<0x4342>(k.x),
                           codes<0x4342>(k.y));
            a2 = make_uint4(codes<0x4140>(k.z), codes<0x4140>(k.w), codes<0x4342>(k.z),
                            codes<0x4342>(k.w));
          } else {
            a = ldsm(piece(from + t * G::sixteen, at_k, 2 * i));
            a2 = ldsm(piece(from + t * G::sixteen, at_k, 2 * i + 1));
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma<MT>(s[t][nb], a, q[nb].x, q[nb].y);
            mma<MT>(kTwo ? s2[t % (kTwo ? MT16 : 1)][nb % (kTwo ? NB : 1)] : s[t][nb], a2, q[nb].z,
                    q[nb].w);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < MT16; ++t) {
        float ka = 1.f, kb = 1.f;
        if constexpr (kEight) ka = scales[t * (kScaleBytes / 4)], kb = scales[t * (kScaleBytes / 4) + 8];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (kTwo) s[t][nb][e] += s2[t][nb][e];
            s[t][nb][e] *= kEight ? (e < 2 ? ka : kb) * c[nb][e & 1] : c[nb][e & 1];
          }
      }
      release();
      const bool edge = token + kTokens > len - p.a.T + 1;  // some row does not see all
      if (edge) {
#pragma unroll
        for (int t = 0; t < MT16; ++t)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (token + 16 * t + g + e / 2 * 8 >= most[nb][e & 1]) s[t][nb][e] = -INFINITY;
      }
      // ------------------------------------------------------------ weights
      // The rows' maximum is only put together when a lane's is over the slack.
      float h[NB][2];
      bool rise = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(s[0][nb][e], s[0][nb][e + 2]);
#pragma unroll
          for (int t = 1; t < MT16; ++t) x = fmaxf(x, fmaxf(s[t][nb][e], s[t][nb][e + 2]));
          h[nb][e] = x;
          rise = rise || x - m[nb][e] > kSlack;
        }
      if (__any_sync(~0u, rise)) {
        float f[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float top = fmaxf(over_tokens(h[nb][e]), m[nb][e]);
            f[nb][e] = weight(m[nb][e], top);
            l[nb][e] *= f[nb][e];
            if (kEight && u[nb][e] != -INFINITY) {
              // The sums keep their unit; where it lies too far below now, the
              // weights are made for the lowest one and the sums scaled after them.
              u[nb][e] -= top - m[nb][e];
              ratio[nb][e] = ex2(fminf(-u[nb][e], kLead));
            }
            m[nb][e] = top;
          }
        if constexpr (!kEight) rescale(f);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float z = m[nb][e] == -INFINITY ? 0.f : m[nb][e];
#pragma unroll
          for (int t = 0; t < MT16; ++t) {
            s[t][nb][e] = ex2(s[t][nb][e] - z), s[t][nb][e + 2] = ex2(s[t][nb][e + 2] - z);
            l[nb][e] += s[t][nb][e] + s[t][nb][e + 2];
          }
        }
      st = used % G::depth;
      ok = ok && mbar_wait(&bar[st], used / G::depth & 1);
      from = ring + st * G::unit;
      uint2 w[MT16][NB];  // the weights, two tokens' a word
      if constexpr (kEight) {
        // The same with the values' scales in the weights: 2^(s - m) scale 2^-u, first in
        // the units as they are.
        scales = reinterpret_cast<const float*>(scale_p + st * G::scale) + g;
        constexpr float kMost = 256.f;  // 2^kSlack
        // What a row does not see may have any scale.
        const auto unseen = [&](int t, int nb, int e) {
          return edge && token + 16 * t + g + e / 2 * 8 >= most[nb][e & 1];
        };
        const auto scaled = [&](int t, int nb, int e, float by) {
          return unseen(t, nb, e) ? 0.f : s[t][nb][e] * ratio[nb][e & 1] * by;
        };
        bool up = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) h[nb][0] = h[nb][1] = 0.f;
#pragma unroll
        for (int t = 0; t < MT16; ++t) {
          const float va = scales[t * (kScaleBytes / 4)], vb = scales[t * (kScaleBytes / 4) + 8];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e] = s[t][nb][e] * ((e < 2 ? va : vb) * ratio[nb][e & 1]);
              if (unseen(t, nb, e)) x[e] = 0.f;
              h[nb][e & 1] = max_nan(h[nb][e & 1], x[e]);
            }
            w[t][nb] = make_uint2(pack<MT>(x[0], x[1]), pack<MT>(x[2], x[3]));
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) up = up || !(h[nb][e] <= kMost) || u[nb][e] < -kLead;
        if (__any_sync(~0u, up)) {
          // Once more, in other units: those of the rows' largest 2^(s - m) scale, whose
          // exponents go to h.
          float f[NB][2];
          bool out_of_range = false, moved = false;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              out_of_range = out_of_range || !(h[nb][e] < 0x1p126f);
              h[nb][e] = lg2(h[nb][e]) + (u[nb][e] == -INFINITY ? 0.f : fmaxf(u[nb][e], -kLead));
            }
          if (__any_sync(~0u, out_of_range)) {
            // Taken without the unit; 2^-9 of it, as s - m <= 8.
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x = 0.f;
#pragma unroll
                for (int t = 0; t < MT16; ++t) {
                  const float* by = scales + t * (kScaleBytes / 4);
                  if (!unseen(t, nb, e)) x = fmaxf(x, s[t][nb][e] * (by[0] * 0x1p-9f));
                  if (!unseen(t, nb, e + 2)) x = fmaxf(x, s[t][nb][e + 2] * (by[8] * 0x1p-9f));
                }
                h[nb][e] = lg2(x) + 9.f;
              }
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // At most 125, where 2^-u and the weights are in range.  -infinity: nothing
              // but zeros so far, no unit.
              const float to = fminf(over_tokens(h[nb][e]), 125.f), was = u[nb][e];
              if (was == -INFINITY || to > was + kSlack) u[nb][e] = to;
              if (u[nb][e] != -INFINITY) u[nb][e] = fmaxf(u[nb][e], -kLead);
              f[nb][e] = was == -INFINITY ? 1.f : ex2(was - u[nb][e]);
              moved = moved || f[nb][e] != 1.f;
              ratio[nb][e] = u[nb][e] == -INFINITY ? 1.f : ex2(-u[nb][e]);
            }
          if (__any_sync(~0u, moved)) rescale(f);
#pragma unroll
          for (int t = 0; t < MT16; ++t) {
            const float va = scales[t * (kScaleBytes / 4)], vb = scales[t * (kScaleBytes / 4) + 8];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              w[t][nb] = make_uint2(pack<MT>(scaled(t, nb, 0, va), scaled(t, nb, 1, va)),
                                    pack<MT>(scaled(t, nb, 2, vb), scaled(t, nb, 3, vb)));
          }
        }
      } else if (edge) {
        // The MMA multiplies every value of the slice by its weight, and 0 * NaN is
        // not 0.  Slots behind the last position hold anything: zeros.  What is not
        // finite among the newest positions, which only some rows see, is added to the
        // sums of those, and then zero too.
        const int newest = max(len - p.a.T + 1 - token, 0), end = min(len - token, kTokens);
        constexpr int kPieces = G::rowBytes / 16;
        uint8_t* unit = ring_p + st * G::unit;
        const auto at = [&](int j, int piece) {  // 16 bytes of the slice's position j
          return unit + j / 16 * G::sixteen + piece / 8 * (16 * G::boxBytes) + j % 16 * G::boxBytes +
                 (piece % 8 ^ j % 8) * 16;
        };
        bool odd = false;
        for (int x = newest * kPieces + lane; x < end * kPieces; x += 32) {
          const uint4 y = *reinterpret_cast<const uint4*>(at(x / kPieces, x % kPieces)), z = finite<QT>(y);
          odd = odd || y.x != z.x || y.y != z.y || y.z != z.z || y.w != z.w;
        }
        odd = __any_sync(~0u, odd);
        if (odd) {
#pragma unroll 1
          for (int j = newest; j < end; ++j)
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              const float y = widen(reinterpret_cast<const QT*>(at(j, i))[g]);
              if (fabsf(y) < INFINITY) continue;
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (token + j < most[nb][e]) o[i / 2][nb][i % 2 * 2 + e] += y;
            }
          if (RT > 1) named_bar_sync(1 + slice, RT * 32);
        }
        if (odd || token + kTokens > len) {
          if (rt == 0) {
            for (int x = (odd ? newest : end) * kPieces + lane; x < kTokens * kPieces; x += 32) {
              uint4& y = *reinterpret_cast<uint4*>(at(x / kPieces, x % kPieces));
              y = x < end * kPieces ? finite<QT>(y) : make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          if (RT > 1) named_bar_sync(1 + slice, RT * 32);
          __syncwarp();
        }
      }
      // ------------------------------------------------------------ products
#pragma unroll
      for (int t = 0; t < MT16; ++t) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (!kEight)
            w[t][nb] = make_uint2(pack<MT>(s[t][nb][0], s[t][nb][1]),
                                  pack<MT>(s[t][nb][2], s[t][nb][3]));
          w[t][nb] = make_uint2(transposed(w[t][nb].x), transposed(w[t][nb].y));
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint4 a, a2;
          if constexpr (kEight) {
            uint4 v = ldsm_t(piece(from + t * G::sixteen, at_v, i));
            v.x ^= 0x80808080u, v.y ^= 0x80808080u, v.z ^= 0x80808080u, v.w ^= 0x80808080u;
            a = make_uint4(codes<0x4240>(v.x), codes<0x4341>(v.x), codes<0x4240>(v.y),
                           codes<0x4341>(v.y));
            a2 = make_uint4(codes<0x4240>(v.z), codes<0x4341>(v.z), codes<0x4240>(v.w),
                            codes<0x4341>(v.w));
          } else {
            a = ldsm_t(piece(from + t * G::sixteen, at_v, 2 * i));
            a2 = ldsm_t(piece(from + t * G::sixteen, at_v, 2 * i + 1));
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma<MT>(o[2 * i][nb], a, w[t][nb].x, w[t][nb].y);
            mma<MT>(o[2 * i + 1][nb], a2, w[t][nb].x, w[t][nb].y);
          }
        }
      }
      release();
    }

    // ----------------------------------------------------- the warps' join
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nb][e];
        sum += __shfl_xor_sync(~0u, sum, 4);
        sum += __shfl_xor_sync(~0u, sum, 8);
        sum += __shfl_xor_sync(~0u, sum, 16);
        if (g == 0) {
          float* to = stat + warp * kWarpRows + nb * kBlock + 2 * i4 + e;
          to[0] = m[nb][e];
          to[W * kWarpRows] = sum;
          if (kEight) to[2 * W * kWarpRows] = u[nb][e];
        }
      }
    // On to the next item: its queries come in while this one is joined.
    here.left -= last - first - 1;
    here.tile = last - 1;
    next_tile<kTile, G::begin>(here, p);
    // In a cluster the ring, which is empty now, takes the part.
    float* part = p.cluster ? reinterpret_cast<float*>(smem)
                            : p.parts + (size_t)(2 * blockIdx.x + (first == 0)) * G::slot;
    // Thread (r, x): row r, columns 4 x of every round; the warps that have it.
    constexpr int S = G::slices, kCols = G::joinCols, kQuads = kCols / 4;
    const int r = tid / kQuads, x4 = tid % kQuads * 4, w0 = r / kWarpRows * S;
    float M = -INFINITY, U = -INFINITY, L = 0.f, f[S];
#pragma unroll
    for (int round = 0; round < D / kCols; ++round) {
      if (round) __syncthreads();
      float* mine = join + warp * (kWarpRows * G::joinStride) + 2 * i4 * G::joinStride;
#pragma unroll
      for (int i = 0; i < kCols / 16; ++i)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mine[(nb * kBlock + (e & 1)) * G::joinStride + i * 16 +
                 (kEight ? 2 * g + e / 2 : g + e / 2 * 8)] = o[round * (kCols / 16) + i][nb][e];
      __syncthreads();
      if (round == 0 && here.left > 0) fetch_q(here);
      if (r < G::rows && R0 + r < p.rows) {
        const float* st = stat + w0 * kWarpRows + r % kWarpRows;
        if (round == 0) {
#pragma unroll
          for (int w = 0; w < S; ++w) M = fmaxf(M, st[w * kWarpRows]);
#pragma unroll
          for (int w = 0; w < S; ++w) {
            L += st[(W + w) * kWarpRows] * weight(st[w * kWarpRows], M);
            f[w] = unit_from<CT>(st[w * kWarpRows], kEight ? st[(2 * W + w) * kWarpRows] : 0.f, M);
            U = fmaxf(U, f[w]);
          }
#pragma unroll
          for (int w = 0; w < S; ++w) f[w] = weight(f[w], U);
        }
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < S; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(
              join + ((w0 + w) * kWarpRows + r % kWarpRows) * G::joinStride + x4);
          sum.x = fmaf(y.x, f[w], sum.x), sum.y = fmaf(y.y, f[w], sum.y);
          sum.z = fmaf(y.z, f[w], sum.z), sum.w = fmaf(y.w, f[w], sum.w);
        }
        const int d = round * kCols + x4;
        if (whole) {
          finish<QT, CT, D>(p, b, head, R0 + r, d, len, sum, M, L, U);
        } else {
          *reinterpret_cast<float4*>(part + r * D + d) = sum;
          if (d == 0) {
            part[G::rows * D + r] = M;
            part[G::rows * D + G::rows + r] = L;
            part[G::rows * D + 2 * G::rows + r] = U;
          }
        }
      }
    }
  }
  if (p.cluster > 1) {
    cluster_sync();
    if (parts > 1) {
      const int of = blockIdx.x / p.cluster, b = of / p.items;
      const int head = of % p.items / p.row_groups, R0 = of % p.items % p.row_groups * G::rows;
      const int valid = min(G::rows, p.rows - R0), len = length(p, b);
      const float* part = reinterpret_cast<const float*>(smem);
      for (int i = tid * p.cluster + rank; i < valid * (D / 4); i += G::threads * p.cluster) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float m[kCluster], l[kCluster], u[kCluster];
        float4 y[kCluster];
        float M = -INFINITY, U = -INFINITY, L = 0.f;
#pragma unroll
        for (int k = 0; k < kCluster; ++k) {
          m[k] = u[k] = -INFINITY, l[k] = 0.f, y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < parts) {
            const uint32_t at = map_rank(part, k), st = at + (G::rows * D + r) * 4;
            m[k] = remote(st), l[k] = remote(st + G::rows * 4), u[k] = remote(st + G::rows * 8);
            y[k] = remote4(at + (r * D + d) * 4);
          }
          M = fmaxf(M, m[k]);
        }
#pragma unroll
        for (int k = 0; k < kCluster; ++k) {
          u[k] = unit_from<CT>(m[k], u[k], M);
          U = fmaxf(U, u[k]);
        }
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kCluster; ++k) {
          L += l[k] * weight(m[k], M);
          const float f = weight(u[k], U);
          sum.x = fmaf(y[k].x, f, sum.x), sum.y = fmaf(y[k].y, f, sum.y);
          sum.z = fmaf(y[k].z, f, sum.z), sum.w = fmaf(y[k].w, f, sum.w);
        }
        finish<QT, CT, D>(p, b, head, R0 + r, d, len, sum, M, L, U);
      }
    }
    cluster_sync();  // until all have read this CTA's part
  }
  if (!ok) report(p.a.status, PQ2_ERR_TIMEOUT);
}

// Joins the parts of one row: the CTA that began the item wrote its part into
// its second slot, the ones after it into their first.
template <typename QT, typename CT, int D, int RT, int NB>
__global__ void __launch_bounds__(256) join_kernel(const Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using G = Geo<CT, D, RT, NB>;
  constexpr int kCols = D / 4, kSplit = 256 / kCols;  // threads of a row, shares of the parts
  __shared__ float4 sums[kSplit][kCols];
  __shared__ float stats[kSplit][3];
  const int4 to = p.places[blockIdx.x];
  if (!to.w) return;
  const int r = blockIdx.y, col = threadIdx.x % kCols, share = threadIdx.x / kCols;
  const auto part = [&](int i) {
    return p.parts + (size_t)(2 * (to.z + i) + (i == 0)) * G::slot;
  };
  float M = -INFINITY, U = -INFINITY, L = 0.f;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto add = [&](float4 y, float m, float l, float u) {
    const float top = fmaxf(M, m), now = unit_from<CT>(M, U, top), more = unit_from<CT>(m, u, top);
    L = L * weight(M, top) + l * weight(m, top);
    M = top, U = fmaxf(now, more);
    const float a = weight(now, U), e = weight(more, U);
    sum.x = sum.x * a + y.x * e, sum.y = sum.y * a + y.y * e;
    sum.z = sum.z * a + y.z * e, sum.w = sum.w * a + y.w * e;
  };
  for (int i = share; i < to.w; i += kSplit) {
    const float* from = part(i);
    const float m = from[G::rows * D + r], l = from[G::rows * D + G::rows + r],
                u = from[G::rows * D + 2 * G::rows + r];
    add(*reinterpret_cast<const float4*>(from + r * D + col * 4), m, l, u);
  }
  sums[share][col] = sum;
  if (col == 0) stats[share][0] = M, stats[share][1] = L, stats[share][2] = U;
  __syncthreads();
  if (share) return;
  for (int i = 1; i < kSplit; ++i) add(sums[i][col], stats[i][0], stats[i][1], stats[i][2]);
  finish<QT, CT, D>(p, to.x, to.y / p.row_groups, to.y % p.row_groups * G::rows + r, col * 4,
                    length(p, to.x), sum, M, L, U);
}

// ------------------------------------------------------------------- host
// Pages as [pages][heads][slots][dim], boxes of 16 slots x 128 bytes at most.
bool page_map(CUtensorMap* map, const void* pages, const pq2_kv_cache& c) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int e = c.dtype == PQ2_I8 ? 1 : 2;
  const int row = (int)c.dim * e, box_bytes = row < 128 ? row : 128;
  // Strides of dimensions with one element are never walked, but must be valid.
  const auto stride = [&](int64_t n, int64_t s) { return (cuuint64_t)(n > 1 ? s * e : row); };
  const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.page_size, (cuuint64_t)c.heads,
                              (cuuint64_t)c.pages};
  const cuuint64_t strides[3] = {stride(c.page_size, c.token_stride),
                                 stride(c.heads, c.head_stride), stride(c.pages, c.page_stride)};
  const cuuint32_t box[4] = {(cuuint32_t)(box_bytes / e), 16, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type = c.dtype == PQ2_I8    ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : c.dtype == PQ2_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return enc(map, type, 4, const_cast<void*>(pages), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool scale_map(CUtensorMap* map, const float* scales, const pq2_kv_cache& c) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)c.page_size, (cuuint64_t)c.heads, (cuuint64_t)c.pages};
  const cuuint64_t strides[2] = {(cuuint64_t)c.page_size * 4, (cuuint64_t)(c.page_size * c.heads) * 4};
  const cuuint32_t box[3] = {16, 1, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(scales), dims, strides,
             box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename QT, typename CT, int D, int RT, int NB>
int launch(Params& p, int sm_count, cudaStream_t stream) {
  using G = Geo<CT, D, RT, NB>;
  auto kern = decode_kernel<QT, CT, D, RT, NB>;
  static std::atomic<uint64_t> allowed{0};
  if (!allow_shared(kern, G::smem, allowed)) return PQ2_ERR_LAUNCH;
  CUtensorMap mk{}, mv{}, mks{}, mvs{};
  if (!page_map(&mk, p.cache.k, p.cache) || !page_map(&mv, p.cache.v, p.cache) ||
      (G::eight && (!scale_map(&mks, p.cache.k_scales, p.cache) ||
                    !scale_map(&mvs, p.cache.v_scales, p.cache))))
    return PQ2_ERR_LAUNCH;
  p.row_groups = (p.rows + G::rows - 1) / G::rows;
  p.items = (int)p.cache.heads * p.row_groups;
  const int ctas = p.cluster ? p.a.batch.B * p.items * p.cluster : std::min(sm_count, kMaxCtas);
  p.places = reinterpret_cast<int4*>(p.a.workspace);
  p.parts = reinterpret_cast<float*>(p.a.workspace + kMaxCtas * sizeof(int4));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(G::threads);
  cfg.dynamicSmemBytes = G::smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)p.cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, mk, mv, mks, mvs, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  if (p.cluster) return PQ2_OK;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(ctas, std::min(p.rows, G::rows));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, join_kernel<QT, CT, D, RT, NB>, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  return PQ2_OK;
}

template <typename QT, typename CT, int D>
int launch_rows(Params& p, int sm_count, cudaStream_t stream) {
  if (p.rows <= 8) return launch<QT, CT, D, 1, 1>(p, sm_count, stream);
  if (p.rows <= 16) return launch<QT, CT, D, 1, 2>(p, sm_count, stream);
  // 32 rows of 256 columns are more than a thread's registers.  24 are three warps'
  // of 8, with twelve warps an SM instead of eight of 16: 12 ragged sequences of up
  // to 6000, 24 rows, 39.5 -> 36.3 us (equal ones 62.2 -> 60.6).  20 rows of 128
  // columns: 92 us with eight warps of 32 rows, 97 so.
  if constexpr (D == 256) {
    if (p.rows <= 24) return launch<QT, CT, D, 3, 1>(p, sm_count, stream);
  }
  return launch<QT, CT, D, D <= 128 ? 1 : 2, D <= 128 ? 4 : 2>(p, sm_count, stream);
}

template <typename QT, typename CT>
int launch_dim(Params& p, int sm_count, cudaStream_t stream) {
  if (p.cache.dim == 64) return launch_rows<QT, CT, 64>(p, sm_count, stream);
  if (p.cache.dim == 128) return launch_rows<QT, CT, 128>(p, sm_count, stream);
  return launch_rows<QT, CT, 256>(p, sm_count, stream);
}

}  // namespace

}  // namespace pq2
