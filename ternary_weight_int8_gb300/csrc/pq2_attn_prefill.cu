// pq2_attn_prefill.cu — attention over packed sequences on the tcgen05 tensor
// cores (sm_103a).
//
// Per query row, with scores s_j = c q . k_j (c = scale / ln 2) over the keys
// that it sees, out = sum 2^(s_j - m) v_j / sum 2^(s_j - m): the keys pass by
// once in tiles of 128, m is a running maximum.  m may stay up to 8 below the
// true one (weights up to 256): only a rise beyond that scales the sums that
// are already there, which happens in the first tiles and hardly after them.
//
// A CTA takes kTiles = 2 query tiles of 128 rows (1 for dim 256) of one key
// head.  A tile's rows are tokens x the G query heads of that key head, row =
// token * G + head, so grouped heads share every key tile that is loaded and a
// short chunk still fills the tile.
//   warps 0-3 (0-7)  softmax, one row a thread and four warps a tile: scores
//            from tensor memory, maximum, weights rounded to 16 bits and stored
//            over the scores, sums in fp32; at the end the output
//   next     copies: Q once, then K and V pieces (128 keys x 128 columns at
//            most) through a ring in shared memory
//   last     allocates tensor memory and issues the MMAs: scores = Q K^T (both
//            from shared memory, K-major), out += P V (P from tensor memory, V
//            as it lies, its keys along K: MN-major)
// While the softmax works on one tile's scores the tensor cores have the other
// tile's two products (dim 256: the next key tile's scores, in a second
// buffer, and the last one's P V), so neither waits for the other for long.
//
// Few query tiles before many keys leave SMs without work: then `splits` CTAs
// take a part of a tile's keys each and write out, m and l in 32 bits, and a
// second kernel joins them.
//
// Rows that the loop cannot do (a value that is not finite in a key tile that they
// see in part, a maximum beyond kFar) are computed again by a warp each: 0.16 us a key
// with 32 of them in turn, and nothing in the loop.
//
// Bound: the MMAs, 4 * 128 * 128 * dim operations a tile pair of 128 x 128.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "pq2_internal.h"
#include "pq2_tensor.cuh"

namespace pq2 {
namespace {

constexpr int BM = 128, BN = 128;  // rows of a query tile, keys of a key tile
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;  // how far m may stay behind, in powers of two
// Weights are 2^(c s - fl(c m)), one multiply-add a score: they and their sums are in
// units of 2^fl(c m).  From this |c m| on the rounding may carry them out of range
// (fp16's at 2^27, fp32's at 2^32); such rows are computed again, c (s - m) a weight.
constexpr float kFar = 16777216.f;

template <int D>
struct Geo {
  static constexpr int tiles = D <= 128 ? 2 : 1;    // query tiles of a CTA
  static constexpr int slots = 2;                   // score buffers
  static constexpr int cols = D < 128 ? D : 128;    // columns of a ring piece
  static constexpr int pieces = D / cols;           // pieces of a key tile
  static constexpr int piece = BN * cols * 2;       // bytes
  static constexpr int stages = D < 128 ? 8 : 5;
  static constexpr int qBytes = BM * D * 2;         // of one tile
  static constexpr int offRing = tiles * qBytes;
  static constexpr int offBar = offRing + stages * piece;
  static constexpr int smem = offBar + 512 + 1024;  // + barriers, alignment
  static constexpr int threads = tiles * 128 + 64;
  static constexpr int copyWarp = tiles * 4, mmaWarp = copyWarp + 1;
  static constexpr int oCol = slots * BN;           // tensor memory columns
  static_assert(oCol + tiles * D <= 512, "tensor memory");
  static_assert(smem <= 227 * 1024, "shared memory");
};

struct Params {
  const int32_t *cu_q, *cu_k;
  const void *q, *k, *v;  // for single rows, where the copies do not serve
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  void* out;
  float* lse;
  int32_t* status;
  int B, q_rows, k_rows, q_heads, heads, group, tokens;  // tokens of a query tile
  float c;        // |scale| / ln 2
  int negative;   // scale < 0
  int causal;
  int splits;     // of a tile's keys; with more than one:
  float* parts;   // [splits][q_rows][q_heads][dim], sums of weights times values
  float2* stats;  // [splits][q_rows][q_heads], maximum (powers of two; infinity: far) and sum of weights
};

// Shared-memory matrix descriptor of a 128-byte swizzled operand whose M or N
// dimension is the contiguous one: 64 elements x 8 rows of K a core block,
// blocks of K 1024 bytes apart, the next 64 elements `next` bytes on.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t next) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(next >> 4) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// As mma_f16_ta, A from shared memory.
__device__ __forceinline__ void mma_f16_ss(uint32_t on, uint32_t d_tmem, uint64_t adesc,
                                           uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
        "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
        "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// (a0, a1) * b + c in both halves.
__device__ __forceinline__ void fma2(float& r0, float& r1, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\t"
      "mov.b64 c, {%5, %5};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r0), "=f"(r1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& r0, float& r1, float a0, float a1) {
  asm("{\n\t.reg .b64 a, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 d, {%0, %1};\n\t"
      "add.rn.f32x2 d, d, a;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "+f"(r0), "+f"(r1)
      : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

template <typename T>
constexpr uint32_t kFormat = std::is_same<T, __half>::value ? 0u : 1u;
template <typename T>
__device__ constexpr uint32_t instr_desc(int n, bool b_mn_major, bool negate_a) {
  return (1u << 4) | kFormat<T> << 7 | kFormat<T> << 10 | (negate_a ? 1u << 13 : 0u) |
         (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(BM >> 4) << 24;
}

// The columns of one row that are not finite once more, by the formula itself and
// by a whole warp: the MMA multiplies every value of a key tile by its weight, and
// 0 * NaN of a key that the row does not see would stay in the row.  A column with
// infinities or NaN among the values that the row does see is their sum (a weight
// that rounds to zero is not one), and needs no scores.  all: every column and the
// row's lse.
template <typename T, int D>
__device__ __noinline__ void plain_row(const T* q, const T* k, int64_t k_token, const T* v,
                                       int64_t v_token, int most, float c, bool negative, T* out,
                                       bool all, float* lse) {
  constexpr int E = D / 32;  // columns of a lane
  struct alignas(2 * E) Columns { T x[E]; };
  const int lane = threadIdx.x & 31;
  out += lane * E, v += lane * E;
  bool bad[E], none = true;
  float odd[E], sum[E];  // of what is not finite, of weights times values
#pragma unroll
  for (int e = 0; e < E; ++e) {
    bad[e] = all || !(fabsf(widen(out[e])) < INFINITY);
    none = none && !bad[e];
    odd[e] = sum[e] = 0.f;
  }
  if (__all_sync(~0u, none)) return;
#pragma unroll 1
  for (int j0 = 0; j0 < most; j0 += 16) {
    Columns y[16];  // behind the last key its values once more, which change nothing
#pragma unroll
    for (int j = 0; j < 16; ++j)
      y[j] = *reinterpret_cast<const Columns*>(v + (int64_t)min(j0 + j, most - 1) * v_token);
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (!(fabsf(widen(y[j].x[e])) < INFINITY)) odd[e] += widen(y[j].x[e]);
    bool settled = true;
#pragma unroll
    for (int e = 0; e < E; ++e) settled = settled && (!bad[e] || odd[e] != odd[e]);
    if (__all_sync(~0u, settled)) break;
  }
  bool settled = !all;
#pragma unroll
  for (int e = 0; e < E; ++e) settled = settled && (!bad[e] || odd[e] != 0.f);
  float m = -INFINITY, l = 0.f;
  if (!__all_sync(~0u, settled)) {
    // A key a lane for the scores, then a key at a time for the values.
#pragma unroll 1
    for (int j0 = 0; j0 < most; j0 += 32) {
      float s = -INFINITY;
      if (j0 + lane < most) {
        const T* key = k + (int64_t)(j0 + lane) * k_token;
        s = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 8) {
          const uint4 a = *reinterpret_cast<const uint4*>(q + d);
          const uint4 b = *reinterpret_cast<const uint4*>(key + d);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            s = fmaf(widen(reinterpret_cast<const T*>(&a)[e]),
                     widen(reinterpret_cast<const T*>(&b)[e]), s);
        }
        if (negative) s = -s;
      }
      float top = s;
#pragma unroll
      for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      top = fmaxf(top, m);
      const float f = m == -INFINITY ? 0.f : ex2((m - top) * c);
      const float w = s == -INFINITY ? 0.f : ex2((s - top) * c);
      float more = w;
#pragma unroll
      for (int o = 16; o; o /= 2) more += __shfl_xor_sync(~0u, more, o);
      l = fmaf(l, f, more), m = top;
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] *= f;
#pragma unroll 8
      for (int j = 0; j < 32; ++j) {
        const float by = __shfl_sync(~0u, w, j);
        if (j0 + j >= most) continue;
        const Columns y = *reinterpret_cast<const Columns*>(v + (int64_t)(j0 + j) * v_token);
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] = fmaf(by, widen(y.x[e]), sum[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (bad[e]) {
      // l - l: NaN where a score is, whatever the values are.
      const uint32_t y = pack<T>((odd[e] != 0.f ? odd[e] : sum[e] / l) + (l - l), 0.f);
      out[e] = *reinterpret_cast<const T*>(&y);
    }
  if (all && lse && lane == 0) *lse = m * c * kLn2 + logf(l);
}

template <typename T, int D>
__global__ void __launch_bounds__(Geo<D>::threads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const Params p) {
  using G = Geo<D>;
  constexpr int kTiles = G::tiles, kStages = G::stages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_s + 1023u) & ~1023u) - raw_s);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::offBar);
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;   // per query tile
  uint64_t* s_full = q_full + kTiles;   // per score buffer
  uint64_t* p_half = s_full + G::slots; // the first half of the weights, all of them
  uint64_t* p_full = p_half + G::slots;
  uint64_t* o_full = p_full + G::slots; // per query tile
  uint32_t* tmem_addr_s = reinterpret_cast<uint32_t*>(o_full + kTiles);
  int* sums = reinterpret_cast<int*>(tmem_addr_s + 1);  // per warp, then the CTA's place

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = G::threads / 32;
  // What does not wait for the kernel before.
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < kTiles; ++i) mbar_init(&q_full[i], 1), mbar_init(&o_full[i], 1);
    for (int i = 0; i < G::slots; ++i)
      mbar_init(&s_full[i], 1), mbar_init(&p_half[i], 4), mbar_init(&p_full[i], 4);
    fence_barrier_init();
  }
  if (warp == G::copyWarp && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_q) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v) : "memory");
  }
  int* place = sums + kWarps;  // sequence, tile, its rows and keys; tiles so far
  if (tid == 0) place[0] = -1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Which sequence and which of its query tiles.  A sequence of n rows has
  // ceil(n / (kTiles * tokens)); the CTAs count them from a sequence's last one
  // back, so that the tiles with the most keys come first, and up to 32 sequences
  // by their keys: the longest CTAs first, the short ones fill the gaps.
  const int per = kTiles * p.tokens;
  const int head = blockIdx.x % p.heads, nth = blockIdx.x / p.heads;
  const auto row_of = [&](const int32_t* cu, int i, int rows) {
    return min(max(__ldg(cu + i), 0), rows);
  };
  const auto sequence = [&](int b, int (&of)[4]) {  // first row, rows, first key, keys
    of[0] = row_of(p.cu_q, b, p.q_rows), of[2] = row_of(p.cu_k, b, p.k_rows);
    of[1] = max(row_of(p.cu_q, b + 1, p.q_rows) - of[0], 0);
    of[3] = max(row_of(p.cu_k, b + 1, p.k_rows) - of[2], 0);
  };
  int of[4] = {}, tile;
  if (p.B <= 32) {
    if (lane < p.B) sequence(lane, of);
    const int tiles = (of[1] + per - 1) / per;
    int before = 0;
    for (int b = 0; b < p.B; ++b) {
      const int keys = __shfl_sync(~0u, of[3], b), n = __shfl_sync(~0u, tiles, b);
      if (keys > of[3] || (keys == of[3] && b > lane)) before += n;
    }
    const uint32_t hit = __ballot_sync(~0u, nth >= before && nth < before + tiles);
    if (!hit) return;
    const int by = __ffs(hit) - 1;
    tile = __shfl_sync(~0u, before + tiles, by) - 1 - nth;
#pragma unroll
    for (int i = 0; i < 4; ++i) of[i] = __shfl_sync(~0u, of[i], by);
  } else {
    int behind = 0;  // tiles of the sequences behind those looked at
    for (int last = p.B; last > 0 && behind <= nth; last -= G::threads) {
      const int b = last - 1 - tid;
      int mine[4] = {};
      if (b >= 0) sequence(b, mine);
      const int tiles = (mine[1] + per - 1) / per;
      int upto = tiles;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += x;
      }
      if (lane == 31) sums[warp] = upto;
      __syncthreads();
      upto += behind;
      int all = behind;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int x = sums[w];
        upto += w < warp ? x : 0, all += x;
      }
      if (nth < upto && nth >= upto - tiles) {
        place[0] = b, place[1] = upto - 1 - nth;
#pragma unroll
        for (int i = 0; i < 4; ++i) place[2 + i] = mine[i];
      }
      behind = all;
      __syncthreads();
    }
    if (place[0] < 0) return;
    tile = place[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) of[i] = place[2 + i];
  }
  const int q0 = of[0], nq = of[1], k0_all = of[2], nk_all = of[3];
  // This CTA's part of the keys begins at the tile pair's key tile `from`; keys
  // are counted from there.
  int low = 0, high = nk_all;
  if (p.splits > 1) {
    const int last = min((tile + 1) * kTiles * p.tokens, nq) - 1;
    const int all = ((p.causal ? min(max(nk_all - nq + last + 1, 0), nk_all) : nk_all) + BN - 1) / BN;
    low = (int)((int64_t)blockIdx.y * all / p.splits) * BN;
    high = min((int)((int64_t)(blockIdx.y + 1) * all / p.splits) * BN, nk_all);
  }
  const int k0 = k0_all + low, nk = nk_all - low;
  // The keys of its part that token t sees.
  const auto sees = [&](int t) {
    const int n = p.causal ? min(nk_all - nq + t + 1, nk_all) : nk_all;
    return max(min(n, high) - low, 0);
  };
  int first[kTiles], count[kTiles], most_tiles = 0;  // first token, key tiles
#pragma unroll
  for (int s = 0; s < kTiles; ++s) {
    first[s] = (tile * kTiles + s) * p.tokens;
    count[s] = first[s] < nq ? (sees(min(first[s] + p.tokens, nq) - 1) + BN - 1) / BN : 0;
    most_tiles = max(most_tiles, count[s]);
  }

  if (warp == G::mmaWarp) {
    tmem_alloc(tmem_addr_s, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_addr_s;
  bool ok = true;

  // The ring holds the pieces in the order in which the MMAs use them: a key
  // tile's K, then the V of the tile before (dim 256: one further behind).
  if (warp == G::copyWarp) {
    if (lane == 0 && most_tiles > 0) {
      int use = 0;
      const auto pieces = [&](const CUtensorMap* map, int j) {
        for (int i = 0; i < G::pieces; ++i, ++use) {
          const int st = use % kStages;
          if (use >= kStages) ok = ok && mbar_wait(&empty[st], (use / kStages - 1) & 1);
          if (!ok) return;  // no more copies once a wait has given up
          mbar_arrive_expect_tx(&full[st], G::piece);
          uint8_t* to = smem + G::offRing + st * G::piece;
          for (int x = 0; x < G::cols / 64; ++x)
            tma_3d(to + x * (BN * 128), map, i * G::cols + x * 64, head, k0 + j * BN, &full[st]);
        }
      };
#pragma unroll
      for (int s = 0; s < kTiles; ++s) {
        if (!count[s]) continue;
        mbar_arrive_expect_tx(&q_full[s], p.tokens * p.group * D * 2);
        for (int x = 0; x < D / 64; ++x)
          tma_3d(smem + s * G::qBytes + x * (BM * 128), &map_q, x * 64, head * p.group,
                 q0 + first[s], &q_full[s]);
        if (s == 0) pieces(&map_k, 0);
      }
      if (!count[0]) pieces(&map_k, 0);
      for (int j = 0; j < most_tiles; ++j) {
        if (kTiles == 2) {
          pieces(&map_v, j);
          if (j + 1 < most_tiles) pieces(&map_k, j + 1);
        } else {
          if (j + 1 < most_tiles) pieces(&map_k, j + 1);
          pieces(&map_v, j);
        }
      }
    }
    __syncwarp();
  } else if (warp == G::mmaWarp) {
    const uint32_t on = elect_one();
    constexpr uint32_t idesc_pv = instr_desc<T>(G::cols, true, false);
    const uint32_t idesc_qk = instr_desc<T>(BN, false, p.negative);
    const uint32_t ring = smem_u32(smem + G::offRing);
    int k_use = 0, v_use = 0;  // ring positions of the K and V in use
    // Scores of tile s against the K pieces at ring position `use`.
    const auto scores = [&](int s, int slot, int use, bool release) {
      const uint64_t qd = smem_desc_sw128(smem_u32(smem + s * G::qBytes));
#pragma unroll
      for (int i = 0; i < G::pieces; ++i) {
        const int st = (use + i) % kStages;
        ok = ok && mbar_wait(&full[st], ((use + i) / kStages) & 1);
        tc_fence_after();
        const uint64_t kd = smem_desc_sw128(ring + st * G::piece);
#pragma unroll
        for (int x = 0; x < G::cols / 16; ++x) {
          const int d = i * G::cols + x * 16;
          const uint64_t qo = ((d / 64) * (BM * 128) + (d % 64) * 2) >> 4;
          const uint64_t ko = ((x / 4) * (BN * 128) + (x % 4) * 32) >> 4;
          mma_f16_ss(on, tmem + slot * BN, qd + qo, kd + ko, idesc_qk, i > 0 || x > 0);
        }
        if (release) mma_commit(on, &empty[st]);
      }
      mma_commit(on, &s_full[slot]);
    };
    // out += P V of tile s, V's pieces at ring position `use`.
    const auto product = [&](int s, int slot, int use, int j, bool release, bool clean) {
      const uint32_t phase = (kTiles == 2 ? j : j / 2) & 1;
      ok = ok && mbar_wait(&p_half[slot], phase);
#pragma unroll
      for (int i = 0; i < G::pieces; ++i) {
        const int st = (use + i) % kStages;
        ok = ok && mbar_wait(&full[st], ((use + i) / kStages) & 1);
        if (clean) {
          // The keys behind the sequence's last one are another sequence's, or
          // nothing: their values may be infinite or NaN, and the MMA would
          // multiply those by a weight of zero.
          for (int x = 0; x < G::cols / 64; ++x)
            for (int r = nk - j * BN + lane / 8; r < BN; r += 4)
              *reinterpret_cast<uint4*>(smem + G::offRing + st * G::piece + x * (BN * 128) +
                                        r * 128 + (lane % 8) * 16) = make_uint4(0, 0, 0, 0);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        tc_fence_after();
        const uint64_t vd = smem_desc_mn(ring + st * G::piece, BN * 128);
#pragma unroll
        for (int x = 0; x < BN / 16; ++x) {
          if (i == 0 && x == BN / 32) {
            ok = ok && mbar_wait(&p_full[slot], phase);
            tc_fence_after();
          }
          mma_f16_ta(on, tmem + G::oCol + s * D + i * G::cols, tmem + slot * BN + x * 8,
                     vd + ((x * 2048) >> 4), idesc_pv, j > 0 || x > 0);
        }
        if (release) mma_commit(on, &empty[st]);
      }
      mma_commit(on, &o_full[s]);
    };
    const auto ragged = [&](int j) { return (j + 1) * BN > nk; };
    if (most_tiles > 0) {
      if constexpr (kTiles == 2) {
        // positions: K0 V0 K1 V1 ...; the last tile that uses a piece frees it
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!count[s]) continue;
          ok = ok && mbar_wait(&q_full[s], 0);
          scores(s, s, 0, s == 1 || count[1] == 0);
        }
        for (int j = 0; j < most_tiles; ++j) {
          k_use = (2 * j + 2) * G::pieces, v_use = (2 * j + 1) * G::pieces;
          bool cleaned = false;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (j >= count[s]) continue;
            product(s, s, v_use, j, s == 1 || j >= count[1], ragged(j) && !cleaned);
            cleaned = true;
            if (j + 1 < count[s]) scores(s, s, k_use, s == 1 || j + 1 >= count[1]);
          }
        }
      } else {
        // positions: K0 K1 V0 K2 V1 ...
        ok = ok && mbar_wait(&q_full[0], 0);
        scores(0, 0, 0, true);
        int use = G::pieces;
        for (int j = 0; j < most_tiles; ++j) {
          if (j + 1 < most_tiles) {
            scores(0, (j + 1) & 1, use, true);
            use += G::pieces;
          }
          product(0, j & 1, use, j, true, ragged(j));
          use += G::pieces;
        }
      }
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- softmax
    const int s = warp / 4, r = tid % 128, tiles = s ? count[kTiles - 1] : count[0];
    const int t0 = s ? first[kTiles - 1] : first[0], t = t0 + r / p.group;
    const bool live = r < p.tokens * p.group && t < nq;
    const int most = live ? sees(t) : 0;  // keys of this row
    // All rows of the tile see the keys before this.
    const int common = sees(t0);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t o_tmem = tmem + lanes + G::oCol + s * D;
    float m = -INFINITY, l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
    bool far = false;
    for (int j = 0; j < tiles; ++j) {
      const int slot = kTiles == 2 ? s : j & 1;
      const uint32_t s_tmem = tmem + lanes + slot * BN;
      ok = ok && mbar_wait(&s_full[slot], (kTiles == 2 ? j : j / 2) & 1);
      tc_fence_after();
      float v[BN];
#pragma unroll
      for (int i = 0; i < BN / 32; ++i) tmem_ld32(s_tmem + 32 * i, v + 32 * i);
      tmem_ld_wait();
      if ((j + 1) * BN > common) {
        const int end = most - j * BN;
#pragma unroll
        for (int i = 0; i < BN; ++i) v[i] = i < end ? v[i] : -INFINITY;
      }
      float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
      for (int i = 4; i < BN - 4; i += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e] = max3(top[e], v[i + e], v[i + 4 + e]);
#pragma unroll
      for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], v[BN - 4 + e]);
      const float high = max3(top[0], top[1], fmaxf(top[2], top[3]));
      if (j == 0) {
        m = high;
        far = fabsf(m * p.c) > kFar && m != -INFINITY;
      } else {
        const bool rise = (high - m) * p.c > kSlack;
        if (__any_sync(~0u, rise)) {
          const float to = __fmul_rn(high, p.c), f = rise ? ex2(__fmul_rn(m, p.c) - to) : 1.f;
          if (rise) m = high, far = far || fabsf(to) > kFar;
          l0 *= f, l1 *= f, l2 *= f, l3 *= f;
          ok = ok && mbar_wait(&o_full[s], (j - 1) & 1);
          tc_fence_after();
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            uint32_t o[16];
            tmem_ld16(o_tmem + d, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(o_tmem + d, o);
          }
          tmem_st_wait();
        }
      }
      // With one tile the last product but one may still be running here; a
      // phase further and the wait for the last one could not tell them apart.
      if (kTiles == 1 && j > 0 && j + 1 == tiles) ok = ok && mbar_wait(&o_full[0], (j - 1) & 1);
      const float mc = m == -INFINITY ? 0.f : m * p.c;
#pragma unroll
      for (int i = 0; i < BN; i += 32) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float a, b, c, d;
          fma2(a, b, v[i + e], v[i + e + 1], p.c, -mc);
          fma2(c, d, v[i + e + 2], v[i + e + 3], p.c, -mc);
          a = ex2(a), b = ex2(b), c = ex2(c), d = ex2(d);
          add2(l0, l1, a, b);
          add2(l2, l3, c, d);
          w[e / 2] = pack<T>(a, b), w[e / 2 + 1] = pack<T>(c, d);
        }
        tmem_st16(s_tmem + i / 2, w);
        if (i == BN / 2 - 32) {
          // The products with the first half of the keys can begin.
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          warp_arrive(&p_half[slot]);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      warp_arrive(&p_full[slot]);
    }
    const float l = (l0 + l1) + (l2 + l3);
    if (tiles) {
      ok = ok && mbar_wait(&o_full[s], (tiles - 1) & 1);
      tc_fence_after();
    }
    const int h = head * p.group + r % p.group;
    const int64_t row = live ? ((int64_t)q0 + t) * p.q_heads + h : -1;
    const float factor = most > 0 ? 1.f / l : 0.f;
    const float mc = m == -INFINITY ? 0.f : m * p.c;
    // Through the query tile's place in shared memory, which the scores have
    // read for the last time: a thread's row there, then whole rows by all lanes
    // (a thread's own row straight to global memory took 32 lines a store, 5000
    // clocks at dim 128).
    uint8_t* rows = smem + s * G::qBytes + (warp & 3) * 32 * 128;
    const auto staged = [&](int r, int d) {
      return reinterpret_cast<uint4*>(rows + d / 64 * (BM * 128) + r * 128 +
                                      ((d / 8 % 8 ^ (r & 7)) << 4));
    };
    if (p.splits > 1) {
      // Two rounds of half the columns, in 32 bits.
      const int64_t part = (int64_t)blockIdx.y * p.q_rows * p.q_heads;
      if (live) p.stats[part + row] = make_float2(far ? INFINITY : m == -INFINITY ? m : mc, l);
#pragma unroll 1
      for (int round = 0; round < 2; ++round) {
#pragma unroll 1
        for (int d = 0; d < D / 2; d += 32) {
          float o[32];
          if (tiles) {
            tmem_ld32(o_tmem + round * (D / 2) + d, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (tiles)
              w = make_uint4(__float_as_uint(o[i]), __float_as_uint(o[i + 1]),
                             __float_as_uint(o[i + 2]), __float_as_uint(o[i + 3]));
            *staged(lane, (d + i) * 2) = w;
          }
        }
        __syncwarp();
#pragma unroll 2
        for (int i = 0; i < D / 8; ++i) {
          const int piece = i * 32 + lane, of = piece / (D / 8), d = piece % (D / 8) * 4;
          const int64_t to = __shfl_sync(~0u, row, of);
          if (to >= 0)
            *reinterpret_cast<uint4*>(p.parts + (part + to) * D + round * (D / 2) + d) =
                *staged(of, d * 2);
        }
        __syncwarp();
      }
    } else {
    bool bad = false;  // something is not finite
#pragma unroll 1
    for (int d = 0; d < D; d += 32) {
      float o[32];
      if (tiles) {
        tmem_ld32(o_tmem + d, o);
        tmem_ld_wait();
      }
      float zero = 0.f;  // NaN if an element is not finite
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (most <= 0) o[i] = 0.f;
        zero = fmaf(o[i], 0.f, zero);
      }
      bad = bad || zero != 0.f;
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        uint4 w;
        w.x = pack<T>(o[i] * factor, o[i + 1] * factor);
        w.y = pack<T>(o[i + 2] * factor, o[i + 3] * factor);
        w.z = pack<T>(o[i + 4] * factor, o[i + 5] * factor);
        w.w = pack<T>(o[i + 6] * factor, o[i + 7] * factor);
        *staged(lane, d + i) = w;
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const int piece = i * 32 + lane, of = piece / (D / 8), d = piece % (D / 8) * 8;
      const int64_t to = __shfl_sync(~0u, row, of);
      if (to >= 0) *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + to * D + d) = *staged(of, d);
    }
    __syncwarp();
    if (live && p.lse) p.lse[row] = most > 0 ? mc * kLn2 + logf(l) : -INFINITY;
    uint32_t again = __ballot_sync(~0u, live && (far || (bad && factor - factor == 0.f)));
    while (again) {
      const int of = __ffs(again) - 1;
      again &= again - 1;
      const int token = __shfl_sync(~0u, t, of), qh = __shfl_sync(~0u, h, of);
      const int64_t to = __shfl_sync(~0u, row, of);
      plain_row<T, D>(
          static_cast<const T*>(p.q) + ((int64_t)q0 + token) * p.q_token + qh * p.q_head,
          static_cast<const T*>(p.k) + (int64_t)k0 * p.k_token + head * p.k_head, p.k_token,
          static_cast<const T*>(p.v) + (int64_t)k0 * p.v_token + head * p.v_head, p.v_token,
          __shfl_sync(~0u, most, of), p.c, p.negative, static_cast<T*>(p.out) + to * D,
          __shfl_sync(~0u, far, of), p.lse ? p.lse + to : nullptr);
    }
    }
  }
  if (!ok) report(p.status, PQ2_ERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == G::mmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a row: a warp for each, D / 32 neighbouring columns a lane.
template <typename T, int D>
__global__ void __launch_bounds__(256) prefill_join_kernel(const Params p) {
  constexpr int E = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, i = (int)(row / p.q_heads), h = (int)(row % p.q_heads);
  const auto bound = [&](const int32_t* cu, int b, int rows) {
    return min(max(__ldg(cu + b), 0), rows);
  };
  if (i >= p.q_rows || i < bound(p.cu_q, 0, p.q_rows) || i >= bound(p.cu_q, p.B, p.q_rows)) return;
  const int64_t step = (int64_t)p.q_rows * p.q_heads;
  const float2 ml = lane < p.splits ? p.stats[lane * step + row] : make_float2(-INFINITY, 0.f);
  float m = ml.x, l;
#pragma unroll
  for (int o = 16; o; o /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  const float weight = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
  l = ml.y * weight;
  if (ml.y == 0.f) l = 0.f;
#pragma unroll
  for (int o = 16; o; o /= 2) l += __shfl_xor_sync(~0u, l, o);
  float sum[E] = {};
  for (int s = 0; s < p.splits; ++s) {
    const float w = __shfl_sync(~0u, weight, s);
    if (w == 0.f) continue;
    const float* from = p.parts + (s * step + row) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 y = *reinterpret_cast<const float2*>(from + e);
      sum[e] = fmaf(y.x, w, sum[e]), sum[e + 1] = fmaf(y.y, w, sum[e + 1]);
    }
  }
  float zero = l - l;  // NaN if something is not finite
#pragma unroll
  for (int e = 0; e < E; ++e) zero = fmaf(sum[e], 0.f, zero);
  T* out = static_cast<T*>(p.out) + row * D;
  // Rows with sums that are not finite, or that see nothing: which keys do they
  // see?
  const bool far = __any_sync(~0u, ml.x == INFINITY);
  const bool odd = far || __any_sync(~0u, zero != 0.f) || l == 0.f;
  int most = 1, k0 = 0;
  if (odd) {
    int lo = 0, hi = p.B + 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu_q + mid) <= i) lo = mid + 1; else hi = mid;
    }
    const int b = max(min(lo - 1, p.B - 1), 0), q0 = bound(p.cu_q, b, p.q_rows);
    const int nq = bound(p.cu_q, b + 1, p.q_rows) - q0;
    k0 = bound(p.cu_k, b, p.k_rows);
    const int nk = max(bound(p.cu_k, b + 1, p.k_rows) - k0, 0);
    most = p.causal ? min(max(nk - nq + (i - q0) + 1, 0), nk) : nk;
  }
  const float factor = most > 0 ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(out + lane * E + e) =
        most > 0 ? pack<T>(sum[e] * factor, sum[e + 1] * factor) : 0u;
  if (lane == 0 && p.lse) p.lse[row] = most > 0 ? m * kLn2 + logf(l) : -INFINITY;
  __syncwarp();
  if (odd && most > 0 && (far || factor - factor == 0.f)) {
    const int kh = h / p.group;
    plain_row<T, D>(static_cast<const T*>(p.q) + i * p.q_token + h * p.q_head,
                    static_cast<const T*>(p.k) + k0 * p.k_token + kh * p.k_head, p.k_token,
                    static_cast<const T*>(p.v) + k0 * p.v_token + kh * p.v_head, p.v_token, most,
                    p.c, p.negative, out, far, p.lse ? p.lse + row : nullptr);
  }
}

// ------------------------------------------------------------------- host
// Rows of `heads` heads of D 16-bit elements, boxes of 64 elements x box_heads
// x box_rows.
bool row_map(CUtensorMap* map, const KvRows& r, int64_t rows, int heads, int dim, int dtype,
             int box_heads, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  // Strides of dimensions with one element are never walked, but must be valid.
  const cuuint64_t head = (cuuint64_t)(heads > 1 ? r.head_stride : dim) * 2;
  const cuuint64_t token = (cuuint64_t)(rows > 1 ? r.token_stride : (int64_t)heads * dim) * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {head, token};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(map,
             dtype == PQ2_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             3, r.p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// As many tile pairs (dim 256: tiles) as the sequences can have at most.
int64_t tile_pairs(int64_t B, int64_t q_rows, int64_t group, int64_t dim) {
  const int64_t per = (dim <= 128 ? 2 : 1) * (BM / group);
  return std::min(q_rows, (q_rows + per - 1) / per + B - 1);
}
// Parts of a tile's keys: as many as fill one wave of 152 SMs (the workspace's size
// is asked for without a device), of at least 8 key tiles on average, 16 at most.
// 64 rows of 40 heads after 16000 keys, 9 parts: 152 -> 32 us; but 300 tile pairs in
// two parts: 355 -> 392 us (dim 256, 16896 keys), 328 in two: 44 -> 93 us (dim 128,
// 2048 keys), for what the parts write and read.
int key_splits(int64_t B, int64_t q_rows, int64_t k_rows, int64_t q_heads, int64_t heads,
               int64_t dim) {
  const int64_t ctas = tile_pairs(B, q_rows, q_heads / heads, dim) * heads;
  return (int)std::max<int64_t>(
      1, std::min<int64_t>({16, 152 / ctas, k_rows / (B * 8 * BN)}));
}

template <typename T, int D>
int launch(const PrefillParams& a, cudaStream_t stream) {
  using G = Geo<D>;
  auto kern = prefill_kernel<T, D>;
  static std::atomic<uint64_t> allowed{0};
  if (!allow_shared(kern, G::smem, allowed)) return PQ2_ERR_LAUNCH;
  Params p{};
  p.cu_q = a.cu_q, p.cu_k = a.cu_k;
  p.q = a.q.p, p.k = a.k.p, p.v = a.v.p;
  p.q_token = a.q.token_stride, p.q_head = a.q.head_stride;
  p.k_token = a.k.token_stride, p.k_head = a.k.head_stride;
  p.v_token = a.v.token_stride, p.v_head = a.v.head_stride;
  p.out = a.out, p.lse = a.lse, p.status = a.status;
  p.B = a.B, p.q_rows = (int)a.q_rows, p.k_rows = (int)a.k_rows;
  p.q_heads = a.q_heads, p.heads = a.heads, p.group = a.q_heads / a.heads;
  p.tokens = BM / p.group;
  // A scale of zero as one that is too small to matter: a key that is not seen
  // has the score -infinity, and 0 times that is NaN.
  p.c = std::max(std::fabs(a.scale) * kLog2e, 1e-38f);
  p.negative = a.scale < 0.f;
  p.causal = a.causal;
  CUtensorMap mq, mk, mv;
  // Without keys no copy is made; the maps then describe q.
  const KvRows& k = a.k_rows ? a.k : a.q;
  const KvRows& v = a.k_rows ? a.v : a.q;
  const int64_t rows = a.k_rows ? a.k_rows : a.q_rows;
  const int heads = a.k_rows ? a.heads : a.q_heads;
  if (!row_map(&mq, a.q, a.q_rows, a.q_heads, D, a.dtype, p.group, p.tokens) ||
      !row_map(&mk, k, rows, heads, D, a.dtype, 1, BN) ||
      !row_map(&mv, v, rows, heads, D, a.dtype, 1, BN))
    return PQ2_ERR_LAUNCH;
  const int64_t tiles = tile_pairs(a.B, a.q_rows, p.group, D);
  if (tiles * a.heads > 0x7fffffff || (a.q_rows * a.q_heads + 7) / 8 > 0x7fffffff)
    return PQ2_ERR_SHAPE;
  p.splits = key_splits(a.B, a.q_rows, a.k_rows, a.q_heads, a.heads, D);
  p.parts = reinterpret_cast<float*>(a.workspace);
  p.stats = reinterpret_cast<float2*>(p.parts + (size_t)p.splits * a.q_rows * a.q_heads * D);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * a.heads), p.splits);
  cfg.blockDim = dim3(G::threads);
  cfg.dynamicSmemBytes = G::smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  if (p.splits == 1) return PQ2_OK;
  cfg.gridDim = dim3((unsigned)((a.q_rows * a.q_heads + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, prefill_join_kernel<T, D>, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  return PQ2_OK;
}

template <typename T>
int launch_dim(const PrefillParams& p, cudaStream_t stream) {
  if (p.dim == 64) return launch<T, 64>(p, stream);
  if (p.dim == 128) return launch<T, 128>(p, stream);
  return launch<T, 256>(p, stream);
}

}  // namespace

size_t attn_prefill_workspace_bytes(int64_t B, int64_t q_rows, int64_t k_rows, int64_t q_heads,
                                    int64_t heads, int64_t dim) {
  const int splits = key_splits(B, q_rows, k_rows, q_heads, heads, dim);
  return splits == 1 ? 0 : (size_t)splits * q_rows * q_heads * (dim + 2) * sizeof(float);
}

int launch_attn_prefill(const PrefillParams& p, int sm_count, cudaStream_t stream) {
  (void)sm_count;
  return p.dtype == PQ2_BF16 ? launch_dim<__nv_bfloat16>(p, stream)
                             : launch_dim<__half>(p, stream);
}

}  // namespace pq2
