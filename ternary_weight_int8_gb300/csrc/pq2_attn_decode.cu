// pq2_attn_decode.cu — attention of the newest tokens over a paged cache.
//
// Per row (a token's query head), with scores s_j = c q . k_j (c = scale /
// ln 2) over the positions that it sees, out = sum 2^(s_j - m) v_j / sum
// 2^(s_j - m), m a running maximum of the scores seen so far, or at most 8
// below it.
//
// Bound: HBM, the cache is read once.  The T * G rows of the query heads that
// share a key head make one tile of 16 (more rows: several tiles, which read
// the cache through L2), so every key and value is used for all of them: the
// products are m16n8k16 MMAs, which at 16 rows need a third of the time that
// the bytes take.
//
// Work is cut evenly whatever the lengths: the tiles of 16 * warps tokens of
// all (sequence, key head, row tile) are numbered, and a CTA takes a
// contiguous share of them, which may end inside a sequence and span several.
// Inside a tile each warp has 16 tokens of its own, which it copies itself
// (tensor-map boxes of 16 slots into a ring that no other warp touches, so
// nothing waits for another warp before the join) and folds into sums of its
// own.  At the end of a CTA's part of a sequence the warps join; parts that
// are not whole go to the workspace, and a second kernel joins them.
//
// 8-bit caches: codes become fp16 by byte permutes (0x6400 | code + 128 is
// 1024 + 128 + code) and one exact subtraction.  A key's scale multiplies its
// score; a value's goes into its weight, w_j = 2^(s_j + log2 scale_j - m2)
// with a maximum m2 of its own, so that weights are at most 2^8 and keep their
// bits whatever the scales are.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "pq2_internal.h"
#include "pq2_tensor.cuh"

namespace pq2 {
namespace {

constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;   // how far m may stay behind, in powers of two
constexpr int kRows = 16;       // rows of a tile
constexpr int kTokens = 16;     // tokens of a warp's slice
constexpr int kJoinCols = 32;   // columns that the warps join at a time
constexpr int kJoinStride = kJoinCols + 8;  // floats: rows land on other banks
constexpr int kMaxCtas = 512;
constexpr int kScaleBytes = 128;  // of a slice's 16 scales: a copy's target is 128-byte aligned

template <typename CT, int D>
struct Geo {
  static constexpr bool eight = sizeof(CT) == 1;
  static constexpr int warps = 8;
  static constexpr int threads = warps * 32;
  static constexpr int rowBytes = D * (int)sizeof(CT);
  static constexpr int boxBytes = rowBytes < 128 ? rowBytes : 128;
  static constexpr int boxes = rowBytes / boxBytes;
  static constexpr int unit = kTokens * rowBytes;  // a slice's K, or its V
  static constexpr int depth = std::min(8, (eight ? 184320 : 196608) / (unit * warps));
  static constexpr int offScale = warps * depth * unit;
  static constexpr int offJoin = offScale + (eight ? warps * depth * kScaleBytes : 0);
  static constexpr int offQ = offJoin + warps * kRows * kJoinStride * 4;
  static constexpr int offStat = offQ + D / 16 * 32 * 16;       // [3][warps][16]
  static constexpr int offBar = offStat + 3 * warps * kRows * 4 + 2 * kRows * 4;
  static constexpr int smem = offBar + warps * depth * 8 + 64 + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
  static constexpr int slot = kRows * D + 3 * kRows;  // floats of a part in the workspace
};

struct Params {
  DecodeParams a;
  pq2_kv_cache cache;
  int group, rows, row_tiles, items;  // G, T * G, tiles of 16 of them, heads * row_tiles
  float c;
  float* parts;   // [2 * CTAs][slot]
  int4* places;   // [CTAs]: sequence, item, first CTA, number of parts (0: nothing to join)
};

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

__device__ __forceinline__ int length(const Params& p, int b) {
  return b < p.a.batch.B ? max(__ldg(p.a.batch.lens + b), 0) : 0;
}
__device__ __forceinline__ int tiles_of(int len, int tile) {
  return max(1, len / tile + (len % tile != 0));
}

// Where a CTA, or one of its warps' copies, is in the CTA's share.
struct Cursor {
  int b, x, tile, tiles, len, next_len;
  int64_t left;
};
template <int TILE>
__device__ __forceinline__ void next_tile(Cursor& c, const Params& p) {
  --c.left;
  if (++c.tile < c.tiles) return;
  c.tile = 0;
  if (++c.x < p.items) return;
  c.x = 0, ++c.b;
  c.len = c.next_len;
  c.tiles = tiles_of(c.len, TILE);
  c.next_len = length(p, c.b + 1);
}

// Four columns of one row by the formula itself, for rows whose sums met an
// infinity or NaN although they do not see the newest positions: an MMA
// multiplies every value of a slice by its weight, and 0 * NaN would stay.
template <typename QT, typename CT, int D>
__device__ __noinline__ float4 plain_columns(const Params& p, int b, int item, int r, int d,
                                             int most, float m, float l) {
  const int R = item % p.row_tiles * kRows + r, kh = item / p.row_tiles;
  const QT* q = static_cast<const QT*>(p.a.q) + b * p.a.batch_stride +
                R / p.group * p.a.token_stride + (kh * p.group + R % p.group) * p.a.head_stride;
  float o[4] = {};
#pragma unroll 1
  for (int j = 0; j < most; ++j) {
    const int64_t at = j / p.cache.page_size, slot = j - at * p.cache.page_size;
    const int64_t page =
        at < p.a.batch.table_width ? __ldg(p.a.batch.table + b * p.a.batch.table_stride + at) : -1;
    const bool there = page >= 0 && page < p.cache.pages;
    const int64_t from =
        page * p.cache.page_stride + kh * p.cache.head_stride + slot * p.cache.token_stride;
    const int64_t side = (page * p.cache.heads + kh) * p.cache.page_size + slot;
    float s = 0.f;
    if (there) {
      const CT* k = static_cast<const CT*>(p.cache.k) + from;
#pragma unroll 4
      for (int i = 0; i < D; ++i) s = fmaf(widen(q[i]), widen(k[i]), s);
      if (sizeof(CT) == 1) s *= p.cache.k_scales[side];
    }
    const float w = ex2(fmaf(s, p.c, -m));
    if (there) {
      const CT* v = static_cast<const CT*>(p.cache.v) + from + d;
      const float vs = sizeof(CT) == 1 ? p.cache.v_scales[side] : 1.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(w, widen(v[i]) * vs, o[i]);
    }
  }
  return make_float4(o[0] / l, o[1] / l, o[2] / l, o[3] / l);
}

// Four columns of a joined row to out, and its lse: o in units of 2^m2, the
// weights' sum l in units of 2^m.
template <typename QT, typename CT, int D>
__device__ __forceinline__ void finish(const Params& p, int b, int item, int r, int d, int len,
                                       float4 o, float m, float l, float m2) {
  const int R = item % p.row_tiles * kRows + r;
  if (R >= p.rows) return;
  const int t = R / p.group, most = len - p.a.T + t + 1;
  const int64_t row =
      ((int64_t)b * p.a.T + t) * p.a.q_heads + item / p.row_tiles * p.group + R % p.group;
  if (most <= 0) {
    o = make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    const float f = (sizeof(CT) == 1 ? weight(m2, m) : 1.f) / l;
    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
    const float zero = (o.x + o.y) * 0.f + (o.z + o.w) * 0.f;
    if (zero != 0.f && l - l == 0.f && most < len)
      o = plain_columns<QT, CT, D>(p, b, item, r, d, most, m, l);
  }
  *reinterpret_cast<uint2*>(static_cast<QT*>(p.a.out) + row * D + d) =
      make_uint2(pack<QT>(o.x, o.y), pack<QT>(o.z, o.w));
  if (d == 0 && p.a.lse) p.a.lse[row] = most > 0 ? m * kLn2 + logf(l) : -INFINITY;
}

template <typename QT, typename CT, int D>
__global__ void __launch_bounds__(Geo<CT, D>::threads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ CUtensorMap map_ks,
                  const __grid_constant__ CUtensorMap map_vs, const Params p) {
  using G = Geo<CT, D>;
  constexpr int W = G::warps, kTile = W * kTokens;
  constexpr bool kEight = G::eight;
  using MT = typename std::conditional<kEight, __half, QT>::type;  // the MMAs' type
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_s + 1023u) & ~1023u) - raw_s);
  float* join = reinterpret_cast<float*>(smem + G::offJoin);
  uint4* q_frag = reinterpret_cast<uint4*>(smem + G::offQ);
  float* stat = reinterpret_cast<float*>(smem + G::offStat);  // m, l, m2 of [warp][row]
  float* row_scale = stat + 3 * W * kRows;                    // of q, 8-bit caches
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + G::offBar);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, i4 = lane & 3;  // fragment row and column pair
  uint64_t* bar = bars + warp * G::depth;
  if (lane == 0) {
    for (int i = 0; i < G::depth; ++i) mbar_init(&bar[i], 1);
    fence_barrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // The CTA's share of the tiles: all of them are counted, then the sequence
  // that holds the first of the share is found.
  Cursor here;
  {
    uint64_t* sums = reinterpret_cast<uint64_t*>(join);   // [W], then the place
    int* place = reinterpret_cast<int*>(sums + W);
    uint64_t total = 0;
    for (int b = tid; b < p.a.batch.B; b += G::threads) total += tiles_of(length(p, b), kTile);
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
          b < p.a.batch.B ? (uint64_t)tiles_of(length(p, b), kTile) * p.items : 0;
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
    here.b = place[0], here.x = place[1], here.tile = place[2];
    here.len = length(p, here.b), here.next_len = length(p, here.b + 1);
    here.tiles = tiles_of(here.len, kTile);
    here.left = (int64_t)(t1 - t0);
    // If the share begins inside an item, and no share before it does, the
    // second kernel's CTA of this number joins that item.
    if (tid == 0) {
      int4 to = make_int4(0, 0, 0, 0);
      if (here.tile > 0) {
        const uint64_t a = t0 - here.tile, z = a + here.tiles - 1;
        const uint64_t c0 = ((a + 1) * ctas - 1) / total, c1 = ((z + 1) * ctas - 1) / total;
        if (c0 + 1 == c) to = make_int4(here.b, here.x, (int)c0, (int)(c1 - c0 + 1));
      }
      p.places[c] = to;
    }
    __syncthreads();
  }

  // ------------------------------------------------------------- the copies
  bool ok = true;
  const uint32_t ring = smem_u32(smem) + warp * (G::depth * G::unit);
  const uint32_t ring_scale = smem_u32(smem + G::offScale) + warp * (G::depth * kScaleBytes);
  const float* scale_of = reinterpret_cast<const float*>(smem + G::offScale) +
                          warp * (G::depth * kScaleBytes / 4);
  const int page_size = (int)p.cache.page_size;
  Cursor copy = here;
  uint32_t issued = 0, used = 0;  // units: K and V of a slice in turn
  int pages = 0, pages_b = -1, pages_tile = 0;  // lane i: the page of tile pages_tile + i
  // To the warp's next slice that holds a token.
  const auto seek = [&]() {
    while (copy.left > 0 && copy.tile * kTile + warp * kTokens >= copy.len)
      next_tile<kTile>(copy, p);
    if (copy.left > 0 && (copy.b != pages_b || copy.tile < pages_tile ||
                          copy.tile >= pages_tile + 32)) {
      pages_b = copy.b, pages_tile = copy.tile;
      const int at = ((copy.tile + lane) * kTile + warp * kTokens) / page_size;
      pages = copy.tile + lane < copy.tiles && at < p.a.batch.table_width
                  ? __ldg(p.a.batch.table + copy.b * p.a.batch.table_stride + at)
                  : -1;
    }
  };
  const auto issue = [&]() {
    if (copy.left <= 0) return;
    const int page = __shfl_sync(~0u, pages, copy.tile - pages_tile);
    if (lane == 0) {
      const uint32_t st = issued % G::depth;
      const bool values = issued & 1;
      const int token = copy.tile * kTile + warp * kTokens, slot = token % page_size;
      const int kh = copy.x / p.row_tiles;
      mbar_arrive_expect_tx(&bar[st], G::unit + (kEight ? kTokens * 4 : 0));
      const uint32_t mb = smem_u32(&bar[st]);
#pragma unroll
      for (int x = 0; x < G::boxes; ++x)
        tma_4d(ring + st * G::unit + x * (kTokens * G::boxBytes), values ? &map_v : &map_k,
               x * (G::boxBytes / (int)sizeof(CT)), slot, kh, page, mb);
      if (kEight)
        tma_3d(ring_scale + st * kScaleBytes, values ? &map_vs : &map_ks, slot, kh, page, mb);
    }
    if (issued & 1) {
      next_tile<kTile>(copy, p);
      seek();
    }
    ++issued;
  };
  seek();
#pragma unroll 1
  for (int i = 0; i < G::depth; ++i) issue();

  // Lane addresses inside a unit.  16 bits: an MMA's K fragments are tokens 0-7
  // and 8-15 x columns 0-7 and 8-15; V's are read transposed.  8 bits: 16 codes
  // of a token are one row of a matrix, for both.  Pieces of 16 bytes are
  // swizzled as the copies left them.
  const int tk = kEight ? (lane & 7) + (lane >> 3 & 1) * 8 : (lane & 7) + (lane >> 4) * 8;
  const int tv = (lane & 7) + (lane >> 3 & 1) * 8;
  const auto lane_base = [&](int token, int piece) {
    const int turn = G::boxBytes == 128 ? token & 7 : token >> 1 & 3;
    return (uint32_t)(token * G::boxBytes + ((piece ^ turn) << 4));
  };
  const uint32_t at_k = lane_base(tk, kEight ? lane >> 4 : lane >> 3 & 1);
  const uint32_t at_v = lane_base(tv, lane >> 4);
  // The lane's piece pair i of a unit.
  const auto piece = [&](uint32_t base, uint32_t at, int i) {
    constexpr int kPairs = G::boxBytes / 32;
    return base + i / kPairs * (kTokens * G::boxBytes) + (at ^ (i % kPairs << 5));
  };

  while (here.left > 0) {
    const int first = here.tile, last = (int)min((int64_t)here.tiles, here.tile + here.left);
    const int b = here.b, item = here.x, len = here.len;
    // ------------------------------------------------------ the rows' queries
    // A fragments: row g (and g + 8), columns of step i: 16 bits 16 i + 2 i4 +
    // {0, 1, 8, 9}; 8 bits 16 i + 4 i4 + {0 .. 3}, the order of a code word.
    const int R0 = item % p.row_tiles * kRows;
    const auto q_row = [&](int r) {
      const int R = R0 + r;
      return static_cast<const QT*>(p.a.q) + b * p.a.batch_stride +
             R / p.group * p.a.token_stride +
             (item / p.row_tiles * p.group + R % p.group) * p.a.head_stride;
    };
    if constexpr (kEight && !std::is_same<QT, __half>::value) {
      // bf16 queries as fp16: scaled by a power of two so that the row's
      // largest lies in [2^14, 2^15); what fp16 loses lies 2^-39 below that.
      for (int r = warp; r < kRows; r += W) {
        float top = 0.f;
        if (R0 + r < p.rows) {
          const QT* q = q_row(r);
          for (int d = lane * 2; d < D; d += 64) {
            const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(q + d);
            top = fmaxf(top, fmaxf(fabsf(widen(x.x)), fabsf(widen(x.y))));
          }
        }
#pragma unroll
        for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        const int e = (int)(__float_as_uint(top) >> 23);  // biased exponent
        // 2^(141 - e), within what fp32 has; 1 for rows of zeros or infinities
        const int up = e == 0 || e == 255 ? 127 : min(max(268 - e, 1), 253);
        if (lane == 0) {
          row_scale[r] = __uint_as_float((uint32_t)up << 23);
          row_scale[kRows + r] = __uint_as_float((uint32_t)(254 - up) << 23);
        }
      }
      __syncthreads();
    }
    for (int f = tid; f < D / 16 * 32; f += G::threads) {
      const int fl = f & 31, step = f >> 5;
      uint32_t a[4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = (fl >> 2) + 8 * half;
        uint32_t lo = 0, hi = 0;
        if (R0 + r < p.rows) {
          const QT* q = q_row(r);
          if constexpr (kEight) {
            q += step * 16 + (fl & 3) * 4;
            lo = *reinterpret_cast<const uint32_t*>(q);
            hi = *reinterpret_cast<const uint32_t*>(q + 2);
            if constexpr (!std::is_same<QT, __half>::value) {
              const float up = row_scale[r];
              lo = pack<__half>(__uint_as_float(lo << 16) * up,
                                __uint_as_float(lo & 0xFFFF0000u) * up);
              hi = pack<__half>(__uint_as_float(hi << 16) * up,
                                __uint_as_float(hi & 0xFFFF0000u) * up);
            }
          } else {
            q += step * 16 + (fl & 3) * 2;
            lo = *reinterpret_cast<const uint32_t*>(q);
            hi = *reinterpret_cast<const uint32_t*>(q + 8);
          }
        }
        a[half] = lo, a[2 + half] = hi;
      }
      q_frag[f] = make_uint4(a[0], a[1], a[2], a[3]);
    }
    __syncthreads();
    float c0 = p.c, c1 = p.c;
    if constexpr (kEight && !std::is_same<QT, __half>::value)
      c0 *= row_scale[kRows + g], c1 *= row_scale[kRows + g + 8];
    // How many positions rows g and g + 8 see.
    const int most0 = len - p.a.T + (R0 + g) / p.group + 1;
    const int most1 = len - p.a.T + (R0 + g + 8) / p.group + 1;

    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows g, g + 8
    float n0 = -INFINITY, n1 = -INFINITY;                      // m2, 8-bit caches
#pragma unroll 1
    for (int tile = first; tile < last; ++tile) {
      const int token = tile * kTile + warp * kTokens;
      if (token >= len) continue;
      // ------------------------------------------------------------- scores
      uint32_t st = used % G::depth;
      ok = ok && mbar_wait(&bar[st], used / G::depth & 1);
      uint32_t from = ring + st * G::unit;
      float s[2][4] = {};  // tokens 0-7 and 8-15
      if constexpr (kEight) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint4 k = ldsm(piece(from, at_k, i));
          k.x ^= 0x80808080u, k.y ^= 0x80808080u, k.z ^= 0x80808080u, k.w ^= 0x80808080u;
          const uint4 qa = q_frag[(2 * i) * 32 + lane], qb = q_frag[(2 * i + 1) * 32 + lane];
          mma<MT>(s[0], qa, codes<0x4140>(k.x), codes<0x4342>(k.x));
          mma<MT>(s[1], qa, codes<0x4140>(k.y), codes<0x4342>(k.y));
          mma<MT>(s[0], qb, codes<0x4140>(k.z), codes<0x4342>(k.z));
          mma<MT>(s[1], qb, codes<0x4140>(k.w), codes<0x4342>(k.w));
        }
        const float2 ka = *reinterpret_cast<const float2*>(scale_of + st * (kScaleBytes / 4) + 2 * i4);
        const float2 kb = *reinterpret_cast<const float2*>(scale_of + st * (kScaleBytes / 4) + 8 + 2 * i4);
        s[0][0] *= ka.x * c0, s[0][1] *= ka.y * c0, s[0][2] *= ka.x * c1, s[0][3] *= ka.y * c1;
        s[1][0] *= kb.x * c0, s[1][1] *= kb.y * c0, s[1][2] *= kb.x * c1, s[1][3] *= kb.y * c1;
      } else {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint4 k = ldsm(piece(from, at_k, i)), qa = q_frag[i * 32 + lane];
          mma<MT>(s[0], qa, k.x, k.y);
          mma<MT>(s[1], qa, k.z, k.w);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
          s[n][0] *= c0, s[n][1] *= c0, s[n][2] *= c1, s[n][3] *= c1;
      }
      __syncwarp();
      issue();
      ++used;
      const bool edge = token + kTokens > len - p.a.T + 1;  // some row does not see all
      if (edge) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = token + 8 * n + 2 * i4 + e;
            if (j >= most0) s[n][e] = -INFINITY;
            if (j >= most1) s[n][2 + e] = -INFINITY;
          }
      }
      // ------------------------------------------------------------ weights
      float h0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float h1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      h0 = fmaxf(h0, __shfl_xor_sync(~0u, h0, 1)), h1 = fmaxf(h1, __shfl_xor_sync(~0u, h1, 1));
      h0 = fmaxf(h0, __shfl_xor_sync(~0u, h0, 2)), h1 = fmaxf(h1, __shfl_xor_sync(~0u, h1, 2));
      const bool rise0 = h0 - m0 > kSlack, rise1 = h1 - m1 > kSlack;
      if (__any_sync(~0u, rise0 || rise1)) {
        const float f0 = rise0 ? weight(m0, h0) : 1.f, f1 = rise1 ? weight(m1, h1) : 1.f;
        if (rise0) m0 = h0;
        if (rise1) m1 = h1;
        l0 *= f0, l1 *= f1;
        if constexpr (!kEight) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n) o[n][0] *= f0, o[n][1] *= f0, o[n][2] *= f1, o[n][3] *= f1;
        }
      }
      const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
      float w[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        w[n][0] = ex2(s[n][0] - z0), w[n][1] = ex2(s[n][1] - z0);
        w[n][2] = ex2(s[n][2] - z1), w[n][3] = ex2(s[n][3] - z1);
        l0 += w[n][0] + w[n][1], l1 += w[n][2] + w[n][3];
      }
      st = used % G::depth;
      ok = ok && mbar_wait(&bar[st], used / G::depth & 1);
      from = ring + st * G::unit;
      if constexpr (kEight) {
        // The same with the values' scales in the weights.
        const float2 va = *reinterpret_cast<const float2*>(scale_of + st * (kScaleBytes / 4) + 2 * i4);
        const float2 vb = *reinterpret_cast<const float2*>(scale_of + st * (kScaleBytes / 4) + 8 + 2 * i4);
        const float v[2][2] = {{lg2(va.x), lg2(va.y)}, {lg2(vb.x), lg2(vb.y)}};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[n][e] = edge && s[n][e] == -INFINITY ? -INFINITY : s[n][e] + v[n][e & 1];
        h0 = fmaxf(fmaxf(w[0][0], w[0][1]), fmaxf(w[1][0], w[1][1]));
        h1 = fmaxf(fmaxf(w[0][2], w[0][3]), fmaxf(w[1][2], w[1][3]));
        h0 = fmaxf(h0, __shfl_xor_sync(~0u, h0, 1)), h1 = fmaxf(h1, __shfl_xor_sync(~0u, h1, 1));
        h0 = fmaxf(h0, __shfl_xor_sync(~0u, h0, 2)), h1 = fmaxf(h1, __shfl_xor_sync(~0u, h1, 2));
        const bool up0 = h0 - n0 > kSlack, up1 = h1 - n1 > kSlack;
        if (__any_sync(~0u, up0 || up1)) {
          const float f0 = up0 ? weight(n0, h0) : 1.f, f1 = up1 ? weight(n1, h1) : 1.f;
          if (up0) n0 = h0;
          if (up1) n1 = h1;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) o[n][0] *= f0, o[n][1] *= f0, o[n][2] *= f1, o[n][3] *= f1;
        }
        const float y0 = n0 == -INFINITY ? 0.f : n0, y1 = n1 == -INFINITY ? 0.f : n1;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          w[n][0] = ex2(w[n][0] - y0), w[n][1] = ex2(w[n][1] - y0);
          w[n][2] = ex2(w[n][2] - y1), w[n][3] = ex2(w[n][3] - y1);
        }
      } else if (token + kTokens > len) {
        // Slots behind the last position hold anything: zeros, so that a weight
        // of zero times them is zero.
        for (int x = lane; x < G::boxes * kTokens * 8; x += 32)
          if ((x >> 3) % kTokens >= len - token)
            *reinterpret_cast<uint4*>(smem + warp * (G::depth * G::unit) + st * G::unit + x * 16) =
                make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      const uint4 a = make_uint4(pack<MT>(w[0][0], w[0][1]), pack<MT>(w[0][2], w[0][3]),
                                 pack<MT>(w[1][0], w[1][1]), pack<MT>(w[1][2], w[1][3]));
      // ------------------------------------------------------------ products
      if constexpr (kEight) {
        // Columns 16 i + 4 i4 + {0, 2} in o[2 i], {1, 3} in o[2 i + 1].
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint4 v = ldsm_t(piece(from, at_v, i));
          v.x ^= 0x80808080u, v.y ^= 0x80808080u, v.z ^= 0x80808080u, v.w ^= 0x80808080u;
          mma<MT>(o[4 * i], a, codes<0x4240>(v.x), codes<0x4240>(v.y));
          mma<MT>(o[4 * i + 1], a, codes<0x4341>(v.x), codes<0x4341>(v.y));
          mma<MT>(o[4 * i + 2], a, codes<0x4240>(v.z), codes<0x4240>(v.w));
          mma<MT>(o[4 * i + 3], a, codes<0x4341>(v.z), codes<0x4341>(v.w));
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint4 v = ldsm_t(piece(from, at_v, i));
          mma<MT>(o[2 * i], a, v.x, v.y);
          mma<MT>(o[2 * i + 1], a, v.z, v.w);
        }
      }
      __syncwarp();
      issue();
      ++used;
    }

    // ----------------------------------------------------- the warps' join
    l0 += __shfl_xor_sync(~0u, l0, 1), l1 += __shfl_xor_sync(~0u, l1, 1);
    l0 += __shfl_xor_sync(~0u, l0, 2), l1 += __shfl_xor_sync(~0u, l1, 2);
    if (i4 == 0) {
      float* to = stat + warp * kRows;
      to[g] = m0, to[g + 8] = m1;
      to += W * kRows;
      to[g] = l0, to[g + 8] = l1;
      to += W * kRows;
      to[g] = kEight ? n0 : m0, to[g + 8] = kEight ? n1 : m1;
    }
    const bool whole = first == 0 && last == here.tiles;
    float* part = p.parts + (size_t)(2 * blockIdx.x + (first == 0)) * G::slot;
    // Thread (r, x): row r, columns 4 x of every round.
    const int r = tid >> 3, x4 = (tid & 7) * 4;
    float M = -INFINITY, M2 = -INFINITY, L = 0.f, f[W];
#pragma unroll
    for (int round = 0; round < D / kJoinCols; ++round) {
      if (round) __syncthreads();
      float* mine = join + warp * (kRows * kJoinStride);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float(&y)[4] = o[round * 4 + n];
        if constexpr (kEight) {
          const int col = n / 2 * 16 + 4 * i4 + (n & 1);
          mine[g * kJoinStride + col] = y[0], mine[g * kJoinStride + col + 2] = y[1];
          mine[(g + 8) * kJoinStride + col] = y[2], mine[(g + 8) * kJoinStride + col + 2] = y[3];
        } else {
          const int col = n * 8 + 2 * i4;
          *reinterpret_cast<float2*>(mine + g * kJoinStride + col) = make_float2(y[0], y[1]);
          *reinterpret_cast<float2*>(mine + (g + 8) * kJoinStride + col) = make_float2(y[2], y[3]);
        }
      }
      __syncthreads();
      if (tid < kRows * 8) {
        if (round == 0) {
#pragma unroll
          for (int w = 0; w < W; ++w) {
            M = fmaxf(M, stat[w * kRows + r]);
            M2 = fmaxf(M2, stat[(2 * W + w) * kRows + r]);
          }
#pragma unroll
          for (int w = 0; w < W; ++w) {
            L += stat[(W + w) * kRows + r] * weight(stat[w * kRows + r], M);
            f[w] = weight(stat[(2 * W + w) * kRows + r], M2);
          }
        }
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float4 y =
              *reinterpret_cast<const float4*>(join + (w * kRows + r) * kJoinStride + x4);
          sum.x = fmaf(y.x, f[w], sum.x), sum.y = fmaf(y.y, f[w], sum.y);
          sum.z = fmaf(y.z, f[w], sum.z), sum.w = fmaf(y.w, f[w], sum.w);
        }
        const int d = round * kJoinCols + x4;
        if (whole) {
          finish<QT, CT, D>(p, b, item, r, d, len, sum, M, L, M2);
        } else {
          *reinterpret_cast<float4*>(part + r * D + d) = sum;
          if (d == 0) {
            part[kRows * D + r] = M;
            part[kRows * D + kRows + r] = L;
            part[kRows * D + 2 * kRows + r] = M2;
          }
        }
      }
    }
    __syncthreads();
    // On to the next item.
    here.left -= last - first - 1;
    here.tile = last - 1;
    next_tile<kTile>(here, p);
  }
  if (!ok) report(p.a.status, PQ2_ERR_TIMEOUT);
}

// Joins the parts of one row: the CTA that began the item wrote its part into
// its second slot, the ones after it into their first.
template <typename QT, typename CT, int D>
__global__ void __launch_bounds__(256) join_kernel(const Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using G = Geo<CT, D>;
  constexpr int kCols = D / 4, kSplit = 256 / kCols;  // threads of a row, shares of the parts
  __shared__ float4 sums[kSplit][kCols];
  __shared__ float stats[kSplit][3];
  const int4 to = p.places[blockIdx.x];
  if (!to.w) return;
  const int r = blockIdx.y, col = threadIdx.x % kCols, share = threadIdx.x / kCols;
  const auto part = [&](int i) {
    return p.parts + (size_t)(2 * (to.z + i) + (i == 0)) * G::slot;
  };
  float M = -INFINITY, M2 = -INFINITY, L = 0.f;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = share; i < to.w; i += kSplit) {
    const float* from = part(i);
    const float m = from[kRows * D + r], l = from[kRows * D + kRows + r],
                m2 = from[kRows * D + 2 * kRows + r];
    const float4 y = *reinterpret_cast<const float4*>(from + r * D + col * 4);
    const float top = fmaxf(M, m), top2 = fmaxf(M2, m2);
    L = L * weight(M, top) + l * weight(m, top);
    const float a = weight(M2, top2), e = weight(m2, top2);
    sum.x = sum.x * a + y.x * e, sum.y = sum.y * a + y.y * e;
    sum.z = sum.z * a + y.z * e, sum.w = sum.w * a + y.w * e;
    M = top, M2 = top2;
  }
  sums[share][col] = sum;
  if (col == 0) stats[share][0] = M, stats[share][1] = L, stats[share][2] = M2;
  __syncthreads();
  if (share) return;
  for (int i = 1; i < kSplit; ++i) {
    const float m = stats[i][0], l = stats[i][1], m2 = stats[i][2];
    const float4 y = sums[i][col];
    const float top = fmaxf(M, m), top2 = fmaxf(M2, m2);
    L = L * weight(M, top) + l * weight(m, top);
    const float a = weight(M2, top2), e = weight(m2, top2);
    sum.x = sum.x * a + y.x * e, sum.y = sum.y * a + y.y * e;
    sum.z = sum.z * a + y.z * e, sum.w = sum.w * a + y.w * e;
    M = top, M2 = top2;
  }
  finish<QT, CT, D>(p, to.x, to.y, r, col * 4, length(p, to.x), sum, M, L, M2);
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
  const cuuint32_t box[4] = {(cuuint32_t)(box_bytes / e), kTokens, 1, 1};
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
  const cuuint32_t box[3] = {kTokens, 1, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(scales), dims, strides,
             box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename QT, typename CT, int D>
int launch(Params& p, int sm_count, cudaStream_t stream) {
  using G = Geo<CT, D>;
  auto kern = decode_kernel<QT, CT, D>;
  static bool configured = false;
  if (!configured) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::smem) !=
        cudaSuccess) {
      cudaGetLastError();
      return PQ2_ERR_LAUNCH;
    }
    configured = true;
  }
  CUtensorMap mk{}, mv{}, mks{}, mvs{};
  if (!page_map(&mk, p.cache.k, p.cache) || !page_map(&mv, p.cache.v, p.cache) ||
      (G::eight && (!scale_map(&mks, p.cache.k_scales, p.cache) ||
                    !scale_map(&mvs, p.cache.v_scales, p.cache))))
    return PQ2_ERR_LAUNCH;
  const int ctas = std::min(sm_count, kMaxCtas);
  p.places = reinterpret_cast<int4*>(p.a.workspace);
  p.parts = reinterpret_cast<float*>(p.a.workspace + kMaxCtas * sizeof(int4));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(G::threads);
  cfg.dynamicSmemBytes = G::smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, mk, mv, mks, mvs, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  cfg.gridDim = dim3(ctas, std::min(p.rows, kRows));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, join_kernel<QT, CT, D>, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  return PQ2_OK;
}

template <typename QT, typename CT>
int launch_dim(Params& p, int sm_count, cudaStream_t stream) {
  if (p.cache.dim == 64) return launch<QT, CT, 64>(p, sm_count, stream);
  if (p.cache.dim == 128) return launch<QT, CT, 128>(p, sm_count, stream);
  return launch<QT, CT, 256>(p, sm_count, stream);
}

}  // namespace

size_t attn_decode_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t dim) {
  return kMaxCtas * sizeof(int4) +
         (size_t)2 * kMaxCtas * (kRows * dim + 3 * kRows) * sizeof(float);
}

int launch_attn_decode(const DecodeParams& a, const pq2_kv_cache& c, int sm_count,
                       cudaStream_t stream) {
  Params p{};
  p.a = a, p.cache = c;
  p.group = a.q_heads / (int)c.heads;
  p.rows = a.T * p.group;
  p.row_tiles = (p.rows + kRows - 1) / kRows;
  p.items = (int)c.heads * p.row_tiles;
  p.c = a.scale * kLog2e;
  if (a.dtype == PQ2_BF16)
    return c.dtype == PQ2_I8 ? launch_dim<__nv_bfloat16, int8_t>(p, sm_count, stream)
                             : launch_dim<__nv_bfloat16, __nv_bfloat16>(p, sm_count, stream);
  return c.dtype == PQ2_I8 ? launch_dim<__half, int8_t>(p, sm_count, stream)
                           : launch_dim<__half, __half>(p, sm_count, stream);
}

}  // namespace pq2
