// pq2_w4.cu — matrix-vector products with 4-bit weights and group scales
// (pq2_w4_prepare, pq2_w4_mmv):
//   y[m][n] = sum_g s[n][g] * sum_{k in g} (c[n][k] - z[n][g]) * x[m][k]
//
// Plane layout.  Rows go in tiles of 16 and columns in units of 128; a unit
// (tile, 128 columns) is one contiguous block in the order in which a warp's
// mma.sync.m16n8k16 takes it as the A operand:
//   512 B   lane l's 16 bytes: words of MMA steps 0..3
//   512 B   lane l's 16 bytes: words of MMA steps 4..7
//   for i = 0..7, per group: (scale of row i, scale of row i + 8), fp16
//   with zero points, for i, per group: zero of row i | zero of row i + 8 << 4
//   padding to 16 bytes
// Step 2j + h of lane 4i + t covers the columns b = 32 j + 8 t + 4 h, ..,
// b + 3 of rows i and i + 8, so that every step lies in one group of 32 and a
// lane's x values of a 32-group are 8 consecutive elements.  Its word holds
//   row i:     b at bit 0, b + 1 at bit 16, b + 2 at bit 8,  b + 3 at bit 24
//   row i + 8: the same 4 bits higher,
// so one shift and one masked OR give a register pair of the A fragment.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "pq2.h"
#include "pq2_device.cuh"
#include "pq2_internal.h"

namespace pq2 {
namespace {

constexpr int kTileRows = 16;
constexpr int kUnitK = 128;
constexpr int kUnitCodeBytes = kTileRows * kUnitK / 2;

__host__ __device__ constexpr int unit_bytes(int group, bool zeros) {
  return (kUnitCodeBytes + kUnitK / group * (zeros ? 40 : 32) + 15) / 16 * 16;
}

// ---------------------------------------------------------------------------
// Preparation: a move of nibbles, one warp per unit.

struct W4PrepParams {
  const uint8_t* codes;    // [N][ldc], two columns per byte, the even one low
  const uint16_t* scales;  // [N][K / group]
  const uint8_t* zeros;    // [N][K / group] or null
  uint8_t* plane;
  int64_t ldc, N, K;
  int64_t units;  // units per tile
  int64_t total;  // units in all
  int group;
};

__global__ void w4_prepare_kernel(W4PrepParams p) {
  const int lane = threadIdx.x & 31, i = lane >> 2, t = lane & 3;
  const int64_t unit = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (unit >= p.total) return;
  const int64_t tile = unit / p.units, u = unit % p.units;
  const int64_t row[2] = {tile * kTileRows + i, tile * kTileRows + i + 8};
  uint8_t* out = p.plane + unit * unit_bytes(p.group, p.zeros != nullptr);
  // Columns beyond K and rows beyond N hold code 0 and scale 0.
  uint32_t words[8] = {};
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if (row[r] >= p.N) continue;
    const uint8_t* src = p.codes + row[r] * p.ldc;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t k = u * kUnitK + 32 * j + 8 * t;
      if (k >= p.K) continue;  // K is a multiple of 32
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t v = src[k / 2 + b];  // columns k + 2b, k + 2b + 1
        const int at = 8 * (b & 1) + 4 * r;
        words[2 * j + (b >> 1)] |= ((v & 15u) << at) | ((v >> 4) << (at + 16));
      }
    }
  }
  reinterpret_cast<uint4*>(out)[lane] = make_uint4(words[0], words[1], words[2], words[3]);
  reinterpret_cast<uint4*>(out + 512)[lane] = make_uint4(words[4], words[5], words[6], words[7]);
  const int groups = kUnitK / p.group;
  const int64_t row_groups = p.K / p.group;
  uint16_t* scales = reinterpret_cast<uint16_t*>(out + kUnitCodeBytes);
  uint8_t* zeros = out + kUnitCodeBytes + groups * 32;
  for (int e = lane; e < groups * 16; e += 32) {  // e = pair, group, half
    const int64_t g = u * groups + e / 2 % groups;
    const int64_t n = tile * kTileRows + e / 2 / groups + 8 * (e & 1);
    scales[e] = g < row_groups && n < p.N ? p.scales[n * row_groups + g] : 0;
  }
  if (p.zeros)
    for (int e = lane; e < groups * 8; e += 32) {  // e = pair, group
      const int64_t g = u * groups + e % groups, n = tile * kTileRows + e / groups;
      uint32_t z = 0;
      if (g < row_groups && n < p.N) z = p.zeros[n * row_groups + g] & 15u;
      if (g < row_groups && n + 8 < p.N) z |= (p.zeros[(n + 8) * row_groups + g] & 15u) << 4;
      zeros[e] = (uint8_t)z;
    }
}

// ---------------------------------------------------------------------------
// Product.
//
// A CTA holds a range of tiles and a range of units (all of them, or its
// share when a cluster splits K), taken in pairs from the range's start.  It
// runs the pairs in passes of one per warp: a warp keeps its pair's x in
// registers (the B fragments) and streams that pair of tile after tile through
// a private ring of cp.async copies, so a weight byte is read once and x once
// per CTA.  The warps' scaled sums of a tile meet in shared memory, where they
// are added in the order of the pairs.
// Bound by instruction issue (133 a unit, 72 of them the decoding) just above
// its bytes: 131072 x 5120 at M = 1 in 62 us, 0.85 of the measured copy rate
// (75 us with one unit a warp; 65 us with five CTAs an SM at 96 registers).
// The order of a y's additions: MMA steps of a group, groups of a unit, the
// two units of a pair, pairs of a CTA's range in ascending order, ranges in
// cluster order.

struct W4Params {
  const void* x;
  const uint8_t* plane;
  void* y;
  int64_t ldx, N;
  int M, K, y_dtype;
  int tiles, units;     // of the matrix
  int split;            // CTAs of a cluster, each with a share of the units
  int warps;            // of the narrow kernel's CTAs
  int block_tiles;      // tiles whose sums the accumulator holds
  int batch_log;        // log2 of the tiles between two joins of the sums
  int vector_x;         // x rows may be read 16 bytes at a time
  int overlap;
};

// Operands are fp16 whatever x's type: a code OR-ed into the mantissa of 1024
// is exactly 1024 + c (or 1024 + 16 c, four bits higher), and one fp16
// operation makes it c - z, exactly (the published way to unpack small whole
// numbers through a floating-point mantissa).  (bf16 has 7 mantissa bits: the higher
// field would need a shift of its own, 7 instead of 5 integer operations per
// 8 weights, and integer operations run at half rate.)
//
// A bf16 or 32-bit x is scaled by a power of two, one per column and pair of
// units, so that the pair's largest |x| lies in [2^14, 2^15).  A bf16 value is then
// exact in fp16 down to 2^-28 of that largest one, and 2^-39 of it is the most
// that rounding below costs.  A 32-bit x is the sum of two fp16 parts, each an
// MMA column of its own: the first has 11 of its 24 bits, the second at least
// 11 of the 12 left (2^-23 of the value).  What the first leaves is at most 2^3,
// so the second has a scale 2^12 times the first's, undone with it after the
// sums: within 2^-51 of the pair's largest |x| where that is more than 2^-23 of
// the value.  (Under one scale for both, 2^-39 of the largest; the second scale
// costs 0.1 us a call.)
constexpr float kPartScale = 4096.f;
template <typename XT>
constexpr int parts() {
  return std::is_same<XT, float>::value ? 2 : 1;
}

__device__ __forceinline__ uint32_t bits(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ __half2 half2_of(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }

// d = a b + (first ? 0 : d)
template <bool FIRST>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (FIRST)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What turns the two fields of a row into c - z: 1024 + z to subtract from
// the low one, -(64 + z) to add to a sixteenth of the high one.  As fp16 their
// high bytes are 0x64 and 0xD4, their low bytes z and 16 z.
__device__ __forceinline__ __half2 offset_low(uint32_t zeros, int g) {
  return half2_of(__byte_perm(zeros, 0x64u, 0x4040u + 0x0101u * g));
}
__device__ __forceinline__ __half2 offset_high(uint32_t zeros16, int g) {
  return half2_of(__byte_perm(zeros16, 0xD4u, 0x4040u + 0x0101u * g));
}

// (v & mask) | 0x64006400 in one operation.
__device__ __forceinline__ __half2 field(uint32_t v, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(0x64006400u));
  return half2_of(r);
}

// The A fragment of one step's word: row i is in the fields at bits 0 and 8,
// row i + 8 in those at bits 4 and 12.
__device__ __forceinline__ void decode(uint32_t w, __half2 low, __half2 high, uint32_t* a) {
  const __half2 sixteenth = half2_of(0x2C002C00u);
  const uint32_t v = w >> 8;
  a[0] = bits(__hsub2(field(w, 0x000F000Fu), low));
  a[1] = bits(__hfma2(field(w, 0x00F000F0u), sixteenth, high));
  a[2] = bits(__hsub2(field(v, 0x000F000Fu), low));
  a[3] = bits(__hfma2(field(v, 0x00F000F0u), sixteenth, high));
}

// 8 consecutive elements of a 32-bit x.
__device__ __forceinline__ void load8(const float* x, bool vec, float* v) {
  if (vec) {
    const float4 lo = reinterpret_cast<const float4*>(x)[0];
    const float4 hi = reinterpret_cast<const float4*>(x)[1];
    v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
    v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = x[e];
}
// 8 consecutive elements of a 16-bit x in each 32-group of a pair of units.
__device__ __forceinline__ void load_raw(const uint16_t* x, int64_t k, int64_t K, bool vec, uint4* b) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    b[j] = make_uint4(0, 0, 0, 0);
    if (x && k + 32 * j < K) {  // K is a multiple of 32
      const uint16_t* q = x + k + 32 * j;
      if (vec)
        b[j] = *reinterpret_cast<const uint4*>(q);
      else
        b[j] = make_uint4(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16,
                          q[4] | (uint32_t)q[5] << 16, q[6] | (uint32_t)q[7] << 16);
    }
  }
}

// The B fragments of column `part` of row x (null: zeros) over one pair of
// units from column k (this lane's first), and the factor that undoes their
// scaling.  Every lane of the warp calls it; the four lanes of a column agree
// on the scaling.
template <typename XT>
__device__ __forceinline__ float load_b(const XT* x, int64_t k, int64_t K, int part, bool vec,
                                        uint4* b) {
  if constexpr (std::is_same<XT, __half>::value) {
    load_raw(reinterpret_cast<const uint16_t*>(x), k, K, vec, b);
    return 1.f;
  } else {
    // bf16 stays in its registers until it is scaled; a 32-bit x is read twice
    // (from L1 the second time), as its values would take 64 registers.
    constexpr bool kKeep = !std::is_same<XT, float>::value;
    auto get = [&](int j, float* v) {
      if constexpr (kKeep) {
        const uint32_t w[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = __uint_as_float(w[e] << 16);
          v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
        if (x && k + 32 * j < K) load8(x + k + 32 * j, vec, v);
      }
    };
    if constexpr (kKeep) load_raw(reinterpret_cast<const uint16_t*>(x), k, K, vec, b);
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v[8];
      get(j, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[e]));
    }
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
    const int e8 = (int)(__float_as_uint(most) >> 23);
    // 2^(14 - exponent), as a biased exponent.  Beside an infinity it is the
    // least of them, so that no finite value becomes another, and a second part
    // is left out: the first decides the sums.
    const int up = min(268 - min(e8, 254), 254);
    const uint32_t kept = part && e8 == 255 ? 0u : 0xFFFFFFFFu;
    const float scale = __uint_as_float((uint32_t)up << 23);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v[8];
      get(j, v);
      uint32_t r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float f0 = v[2 * e] * scale, f1 = v[2 * e + 1] * scale;
        if (part) {
          f0 = (f0 - __half2float(__float2half_rn(f0))) * kPartScale;
          f1 = (f1 - __half2float(__float2half_rn(f1))) * kPartScale;
        }
        r[e] = bits(__floats2half2_rn(f0, f1)) & kept;
      }
      b[j] = make_uint4(r[0], r[1], r[2], r[3]);
    }
    const float undo =
        up == 254 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(254 - up) << 23);
    return part ? undo * (1.f / kPartScale) : undo;
  }
}

// Shared memory by 32-bit address, and predicated without a branch: the loop
// over tiles is bound by the instructions it issues.
__device__ __forceinline__ void cp_async16_if(bool on, uint32_t dst, const void* src) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t"
      "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst),
      "l"(src), "r"((int)on)
      : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts_if(bool on, uint32_t at, float v) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.shared.f32 [%0], %1;\n\t}" ::"r"(at),
      "f"(v), "r"((int)on)
      : "memory");
}

// The scales and zero points of lane row pair i, per group of a unit.
template <int GROUP, bool ZEROS>
struct Side {
  static constexpr int kGroups = kUnitK / GROUP;
  uint32_t scale[kGroups], zero;
  __device__ __forceinline__ void load(uint32_t unit, int i) {
    const uint32_t at = unit + kUnitCodeBytes + i * 4 * kGroups;
    if constexpr (kGroups == 1) scale[0] = lds32(at);
    if constexpr (kGroups == 2)
      asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(scale[0]), "=r"(scale[1]) : "r"(at) : "memory");
    if constexpr (kGroups == 4) {
      const uint4 v = lds128(at);
      scale[0] = v.x, scale[1] = v.y, scale[2] = v.z, scale[3] = v.w;
    }
    if constexpr (ZEROS) {
      const uint32_t z = unit + kUnitCodeBytes + 32 * kGroups + i * kGroups;
      if constexpr (kGroups == 1) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(zero) : "r"(z) : "memory");
      if constexpr (kGroups == 2) asm volatile("ld.shared.u16 %0, [%1];" : "=r"(zero) : "r"(z) : "memory");
      if constexpr (kGroups == 4) zero = lds32(z);
    }
  }
  __device__ __forceinline__ float2 scales(int g) const { return __half22float2(half2_of(scale[g])); }
  __device__ __forceinline__ __half2 low(int g) const {
    return ZEROS ? offset_low(zero & 0x0F0F0F0Fu, g) : half2_of(0x64086408u);
  }
  __device__ __forceinline__ __half2 high(int g) const {
    return ZEROS ? offset_high(zero & 0xF0F0F0F0u, g) : half2_of(0xD480D480u);
  }
};

__device__ __forceinline__ uint32_t word_of(uint4 c, int i) {
  return i == 0 ? c.x : i == 1 ? c.y : i == 2 ? c.z : c.w;
}
// sum = (ADD or not the unit's first group ? sum : 0) + s d; s of rows i, i + 8.
template <bool ADD>
__device__ __forceinline__ void add_scaled(int g, float2 s, const float* d, float* sum) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float sc = e < 2 ? s.x : s.y;
    sum[e] = g == 0 && !ADD ? __fmul_rn(sc, d[e]) : __fmaf_rn(sc, d[e], sum[e]);
  }
}

// One unit's products with 8 columns (fragments b), scaled by the groups'
// scales: sum = ADD ? sum + unit : unit.
template <int GROUP, bool ZEROS, bool ADD>
__device__ __forceinline__ void unit_product(uint32_t unit, int lane, const uint4* b, float* sum) {
  constexpr int kGroups = kUnitK / GROUP, kSteps = GROUP / 16;
  Side<GROUP, ZEROS> side;
  side.load(unit, lane >> 2);
  uint4 c;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const __half2 low = side.low(g), high = side.high(g);
    float d[4];
#pragma unroll
    for (int s2 = 0; s2 < kSteps; ++s2) {
      const int step = g * kSteps + s2;
      if (step % 4 == 0) c = lds128(unit + lane * 16 + step / 4 * 512);
      uint32_t a[4];
      decode(word_of(c, step % 4), low, high, a);
      const uint4 bb = b[step / 2];
      if (s2 == 0)
        mma16816<true>(d, a, step % 2 ? bb.z : bb.x, step % 2 ? bb.w : bb.y);
      else
        mma16816<false>(d, a, step % 2 ? bb.z : bb.x, step % 2 ? bb.w : bb.y);
    }
    add_scaled<ADD>(g, side.scales(g), d, sum);
  }
}

__device__ __forceinline__ void store_y(void* y, int dtype, int64_t at, float v) {
  if (dtype == PQ2_F32) reinterpret_cast<float*>(y)[at] = v;
  else if (dtype == PQ2_BF16) reinterpret_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16(v);
  else reinterpret_cast<__half*>(y)[at] = __float2half(v);
}

constexpr int kPitch = 20;  // floats per column of 16 rows: conflict-free

// The narrow kernel's CTA: 4, 8, 12 or 16 warps (one pair of units each at a
// time; multiples of four, as an SM's four schedulers take warps in turn), 16
// of them an SM (128 registers a thread; shared memory is bounded for that),
// and ring stages.
constexpr int kMaxWarps = 16, kStages = 3;
constexpr int ctas_of(int warps) { return kMaxWarps / warps; }  // an SM
constexpr int smem_of(int warps) { return (227 / ctas_of(warps) - 1) * 1024; }

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ void dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename XT, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) w4_mmv_kernel(const W4Params p) {
  constexpr int kParts = parts<XT>();
  constexpr bool kScaled = !std::is_same<XT, __half>::value;
  constexpr int kUnitBytes = unit_bytes(GROUP, ZEROS), kChunks = kUnitBytes / 16;
  constexpr int kSlot = 2 * kUnitBytes;
  extern __shared__ __align__(16) uint8_t smem[];

  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = lane >> 2, t = lane & 3;
  const int cols = p.M * kParts;
  float* const red = reinterpret_cast<float*>(smem + warps * (kStages * kSlot));
  const int red_warp = cols * kPitch, red_tile = warps * red_warp;
  const int red_buf = red_tile << p.batch_log;
  float* const acc = red + 2 * red_buf;

  const int rank = blockIdx.x % p.split, cluster = blockIdx.x / p.split;
  const int clusters = gridDim.x / p.split;
  const int t0 = (int)((int64_t)cluster * p.tiles / clusters);
  const int t1 = (int)((int64_t)(cluster + 1) * p.tiles / clusters);
  const int u0 = (int)((int64_t)rank * p.units / p.split);
  const int u1 = (int)((int64_t)(rank + 1) * p.units / p.split);
  const int pairs = (u1 - u0 + 1) / 2;
  const int64_t tile_bytes = (int64_t)p.units * kUnitBytes;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!p.overlap) dependency_wait();

  // The copies run kStages - 1 items ahead; items are (block of tiles, pass,
  // tile), the last fastest.  `left`: tiles left of the pass being copied;
  // `chunks`: what of an item this warp has (0: nothing).
  const uint32_t ring = smem_u32(smem) + warp * (kStages * kSlot), ring_end = ring + kStages * kSlot;
  int lb = t0, left = min(p.block_tiles, t1 - t0), lp = warp;
  auto chunks_of = [&](int pair) {
    return pair >= pairs ? 0 : u0 + 2 * pair + 1 < u1 ? 2 * kChunks : kChunks;
  };
  int chunks = chunks_of(lp) - lane;
  const uint8_t* src = p.plane + lb * tile_bytes + (int64_t)(u0 + 2 * lp) * kUnitBytes + lane * 16;
  auto copy_next = [&](uint32_t slot) {
    const uint32_t at = slot + lane * 16;
#pragma unroll
    for (int j = 0; j < (2 * kChunks + 31) / 32; ++j)
      cp_async16_if(chunks > 32 * j, at + 512 * j, src + 512 * j);
    asm volatile("cp.async.commit_group;" ::: "memory");
    src += tile_bytes;
    if (--left == 0) {
      lp += warps;
      if (lp - warp >= pairs) {
        lp = warp;
        lb += p.block_tiles;
      }
      left = min(p.block_tiles, t1 - lb);
      chunks = left > 0 ? chunks_of(lp) - lane : 0;
      src = p.plane + lb * tile_bytes + (int64_t)(u0 + 2 * lp) * kUnitBytes + lane * 16;
    }
  };
  uint32_t dst = ring;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    copy_next(dst);
    dst += kSlot;
  }
  if (p.overlap == 1) dependency_wait();

  // dst: the slot that the item before the current one used; cur: its own.
  uint32_t cur = ring;
  const uint32_t out0 = smem_u32(red + warp * red_warp + 2 * t * kPitch + i);
  uint4 b[8];
  float undo[2];
  int buf = 0;
  bool waited = p.overlap != 2;
  for (int b0 = t0; b0 < t1; b0 += p.block_tiles) {
    const int b1 = min(b0 + p.block_tiles, t1);
    for (int pp = 0; pp < pairs || pp == 0; pp += warps) {
      const int pair = pp + warp, active = min(warps, pairs - pp);
      const bool last = pp + warps >= pairs, idle = pair >= pairs;
      const bool two = u0 + 2 * pair + 1 < u1;
      if (!idle && (b0 == t0 || pairs > warps)) {
        // A unit beyond the range belongs to another CTA.
        const int64_t end = min((int64_t)p.K, (int64_t)u1 * kUnitK);
        const int m = i / kParts;
        const XT* x = m < p.M ? static_cast<const XT*>(p.x) + m * p.ldx : nullptr;
        const float f = load_b(x, (int64_t)(u0 + 2 * pair) * kUnitK + 8 * t, end, i % kParts,
                               p.vector_x != 0, b);
        if (kScaled) {
          undo[0] = __shfl_sync(0xffffffffu, f, 8 * t);
          undo[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
        }
      }
      // The fragments are values of their own from here on, not to be formed
      // again from x inside the loop.
#pragma unroll
      for (int j = 0; j < 8; ++j)
        asm volatile("" : "+r"(b[j].x), "+r"(b[j].y), "+r"(b[j].z), "+r"(b[j].w));
      for (int tb = b0; tb < b1; tb += 1 << p.batch_log) {
        const int te = min(tb + (1 << p.batch_log), b1);
        uint32_t out = out0 + buf * red_buf * 4;
        if (idle) {
          for (int tile = tb; tile < te; ++tile) {
            copy_next(dst);
            dst = cur;
            cur = cur + kSlot == ring_end ? ring : cur + kSlot;
          }
        } else {
#pragma unroll 1
          for (int tile = tb; tile < te; ++tile) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncwarp();
            copy_next(dst);
            dst = cur;
            cur += kSlot;
            cur = cur == ring_end ? ring : cur;
            float sum[4];
            if (two) {
              unit_product<GROUP, ZEROS, false>(dst, lane, b, sum);
              unit_product<GROUP, ZEROS, true>(dst + kUnitBytes, lane, b + 4, sum);
            } else {
              unit_product<GROUP, ZEROS, false>(dst, lane, b, sum);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v = kScaled ? __fmul_rn(sum[e], undo[e % 2]) : sum[e];
              sts_if(2 * t + e % 2 < cols, out + (e % 2 * kPitch + e / 2 * 8) * 4, v);
            }
            out += red_tile * 4;
          }
        }
        __syncthreads();
        // Join: one thread per (column, row of the batch), in the order of the pairs.
        const bool done = last && p.split == 1 && kParts == 1;
        if (done && !waited) {
          dependency_wait();
          waited = true;
        }
        const int rows_log = p.batch_log + 4, rows = (te - tb) * kTileRows;
        for (int e = threadIdx.x; e < cols << rows_log; e += blockDim.x) {
          const int v = e >> rows_log, r = e & ((1 << rows_log) - 1);
          if (r >= rows) continue;
          float* a = acc + (v * p.block_tiles + tb - b0) * kTileRows + r;
          const float* q = red + buf * red_buf + (r >> 4) * red_tile + v * kPitch + (r & 15);
          float sum = pp == 0 ? 0.f : *a;
#pragma unroll 4
          for (int w = 0; w < active; ++w) sum += q[w * red_warp];
          if (done) {
            const int64_t n = (int64_t)tb * kTileRows + r;
            if (n < p.N) store_y(p.y, p.y_dtype, v * p.N + n, sum);
          } else {
            *a = sum;
          }
        }
        buf ^= 1;
      }
    }
    if (p.split == 1 && kParts == 1) continue;
    if (!waited) {
      dependency_wait();
      waited = true;
    }
    // Parts of a 32-bit x (the smaller first) and ranges of the cluster.
    if (p.split > 1)
      cluster_sync();
    else
      __syncthreads();
    const int rows = (b1 - b0) * kTileRows;
    for (int e = threadIdx.x + rank * blockDim.x; e < rows * p.M; e += p.split * blockDim.x) {
      const int m = e / rows, r = e % rows;
      float y = 0.f;
      for (int z = 0; z < p.split; ++z) {
        float sum = 0.f;
        for (int q = kParts - 1; q >= 0; --q) {
          const float* a = acc + (m * kParts + q) * p.block_tiles * kTileRows + r;
          float v;
          if (p.split > 1)
            asm volatile(
                "{\n\t.reg .u32 at;\n\tmapa.shared::cluster.u32 at, %1, %2;\n\t"
                "ld.shared::cluster.f32 %0, [at];\n\t}"
                : "=f"(v)
                : "r"(smem_u32(a)), "r"(z)
                : "memory");
          else
            v = *a;
          sum += v;
        }
        y += sum;
      }
      const int64_t n = (int64_t)b0 * kTileRows + r;
      if (n < p.N) store_y(p.y, p.y_dtype, m * p.N + n, y);
    }
    if (p.split > 1)
      cluster_sync();
    else
      __syncthreads();
  }
  if (!waited) dependency_wait();
}

// The wide kernel, for 9 to 32 columns.  x fragments of that many columns do
// not fit a warp's registers, so a CTA keeps those of its range of units in
// shared memory, and a warp takes a tile through the whole range: its sums need
// no join within the CTA.
// The ranges of a cluster are joined round by round by warps of their own,
// while the others are at the next round: a cluster barrier a round, two sets
// of sums.  The order of the additions is the narrow kernel's.
// 131072 x 5120 at M = 32 in 140 us (297 us with 16 columns a launch in the
// narrow form, 145 us with 8 warps of two tiles), 550 multiply-adds a clock and
// SM: the HMMA pipe at 55 %, shared memory at 70 % (every warp reads all of x's
// fragments for each unit), and clusters of five leave 12 of 152 SMs without
// work.  Which of them bounds it was not measured apart.
constexpr int kWideWarps = 16, kJoinWarps = 4, kWideStages = 4;
constexpr int kRoundTiles = kWideWarps;
constexpr int kRoundRows = kRoundTiles * kTileRows;
constexpr int kRoundPitch = kRoundRows + 4;  // floats per column: conflict-free
constexpr int kWideSmem = 227 * 1024;

template <int NT>
constexpr int wide_smem(int pairs, int unit_b) {
  return kRoundTiles * kWideStages * unit_b + pairs * 8 * NT * 512 +
         (pairs + 2 * kRoundPitch) * 8 * NT * 4;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 remote_float4(const float* p, int rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .u32 at;\n\tmapa.shared::cluster.u32 at, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [at];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(smem_u32(p)), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// unit_product for NT column tiles, with the fragments from shared memory.
template <int NT, int GROUP, bool ZEROS, bool ADD>
__device__ __forceinline__ void unit_product_wide(uint32_t unit, int lane, uint32_t b_at,
                                                  float (&sum)[NT][4]) {
  constexpr int kGroups = kUnitK / GROUP, kSteps = GROUP / 16;
  Side<GROUP, ZEROS> side;
  side.load(unit, lane >> 2);
  uint4 c, b[NT];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const __half2 low = side.low(g), high = side.high(g);
    float d[NT][4];
#pragma unroll
    for (int s2 = 0; s2 < kSteps; ++s2) {
      const int step = g * kSteps + s2;
      if (step % 4 == 0) c = lds128(unit + lane * 16 + step / 4 * 512);
      if (step % 2 == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) b[nt] = lds128(b_at + (step / 2 * NT + nt) * 512);
      }
      uint32_t a[4];
      decode(word_of(c, step % 4), low, high, a);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (s2 == 0)
          mma16816<true>(d[nt], a, step % 2 ? b[nt].z : b[nt].x, step % 2 ? b[nt].w : b[nt].y);
        else
          mma16816<false>(d[nt], a, step % 2 ? b[nt].z : b[nt].x, step % 2 ? b[nt].w : b[nt].y);
      }
    }
    const float2 s = side.scales(g);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) add_scaled<ADD>(g, s, d[nt], sum[nt]);
  }
}

template <typename XT, int NT, int GROUP, bool ZEROS>
__global__ void __launch_bounds__((kWideWarps + kJoinWarps) * 32, 1) w4_wide_kernel(const W4Params p) {
  constexpr int kParts = parts<XT>();
  constexpr bool kScaled = !std::is_same<XT, __half>::value;
  constexpr int kUnitBytes = unit_bytes(GROUP, ZEROS), kChunks = kUnitBytes / 16;
  constexpr int kCols = 8 * NT, kSlot = kUnitBytes;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = lane >> 2, t = lane & 3;

  const int rank = blockIdx.x % p.split, cluster = blockIdx.x / p.split;
  const int clusters = gridDim.x / p.split;
  const int t0 = (int)((int64_t)cluster * p.tiles / clusters);
  const int t1 = (int)((int64_t)(cluster + 1) * p.tiles / clusters);
  const int u0 = (int)((int64_t)rank * p.units / p.split);
  const int u1 = (int)((int64_t)(rank + 1) * p.units / p.split);
  const int units = u1 - u0, pairs = (units + 1) / 2;
  const int rounds = (t1 - t0 + kRoundTiles - 1) / kRoundTiles;
  const int64_t tile_bytes = (int64_t)p.units * kUnitBytes;

  uint8_t* const frag = smem + kWideWarps * kWideStages * kSlot;  // [pair][8][NT][32 lanes] 16 B
  // The same places in every CTA of the cluster, whose ranges differ by a unit.
  const int places = ((p.units + p.split - 1) / p.split + 1) / 2;
  float* const undo = reinterpret_cast<float*>(frag + places * 8 * NT * 512);  // [pair][kCols]
  float* const sums = undo + places * kCols;                                   // [2][kCols][pitch]

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!p.overlap) dependency_wait();

  // The copies: items are (round, unit) of the warp's tile.
  const uint32_t ring = smem_u32(smem) + warp * (kWideStages * kSlot);
  int ct = t0 + warp, cu = 0;  // tile and unit of the next copy
  auto copy_next = [&](uint32_t slot) {
    if (ct < t1) {
      const uint8_t* src = p.plane + ct * tile_bytes + (int64_t)(u0 + cu) * kUnitBytes + lane * 16;
      const uint32_t at = slot + lane * 16;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        cp_async16_if(lane < kChunks - 32 * j, at + 512 * j, src + 512 * j);
      }
      if (++cu == units) {
        cu = 0;
        ct += kRoundTiles;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  uint32_t dst = ring;
  if (warp < kWideWarps) {
#pragma unroll
    for (int s = 0; s < kWideStages - 1; ++s) {
      copy_next(dst);
      dst += kSlot;
    }
  }
  if (p.overlap == 1) dependency_wait();

  // x's fragments, once.
  for (int task = warp; task < pairs * NT; task += kWideWarps + kJoinWarps) {
    const int q = task / NT, nt = task % NT, v = 8 * nt + i, m = v / kParts;
    const XT* x = m < p.M ? static_cast<const XT*>(p.x) + m * p.ldx : nullptr;
    const int64_t end = min((int64_t)p.K, (int64_t)u1 * kUnitK);
    uint4 b[8];
    const float f = load_b(x, (int64_t)(u0 + 2 * q) * kUnitK + 8 * t, end, v % kParts,
                           p.vector_x != 0, b);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *reinterpret_cast<uint4*>(frag + ((q * 8 + j) * NT + nt) * 512 + lane * 16) = b[j];
    if (t == 0) undo[q * kCols + v] = f;
  }
  __syncthreads();

  if (warp < kWideWarps) {
    const uint32_t ring_end = ring + kWideStages * kSlot;
    uint32_t cur = ring;
    for (int n = 0; n < rounds; ++n) {
      float acc[NT][4] = {};
      if (t0 + n * kRoundTiles + warp < t1) {
        float sum[NT][4];
#pragma unroll 1
        for (int q = 0; q < pairs; ++q) {
          const uint32_t b_at = smem_u32(frag) + q * 8 * NT * 512 + lane * 16;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (2 * q + h >= units) break;
            asm volatile("cp.async.wait_group %0;" ::"n"(kWideStages - 2) : "memory");
            __syncwarp();
            copy_next(dst);
            dst = cur;
            cur += kSlot;
            cur = cur == ring_end ? ring : cur;
            if (h == 0)
              unit_product_wide<NT, GROUP, ZEROS, false>(dst, lane, b_at, sum);
            else
              unit_product_wide<NT, GROUP, ZEROS, true>(dst, lane, b_at + 4 * NT * 512, sum);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 f = *reinterpret_cast<const float2*>(undo + q * kCols + 8 * nt + 2 * t);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[nt][e] = __fadd_rn(
                  acc[nt][e], kScaled ? __fmul_rn(sum[nt][e], e % 2 ? f.y : f.x) : sum[nt][e]);
          }
        }
      }
      if (n) cluster_wait();  // the sums of round n - 2 have been joined
      float* s = sums + (n & 1) * kCols * kRoundPitch + 2 * t * kRoundPitch + warp * kTileRows + i;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[(8 * nt + e % 2) * kRoundPitch + e / 2 * 8] = acc[nt][e];
      cluster_arrive();
    }
    if (rounds) cluster_wait();
  } else {
    if (p.overlap == 2) dependency_wait();
    for (int n = 0; n < rounds; ++n) {
      cluster_arrive();
      cluster_wait();
      // Parts of a 32-bit x (the smaller first) and ranges of the cluster.
      const int64_t n0 = (int64_t)(t0 + n * kRoundTiles) * kTileRows;
      const int rows = min(kRoundTiles, t1 - t0 - n * kRoundTiles) * kTileRows;
      const float* s = sums + (n & 1) * kCols * kRoundPitch;
      // Four rows of a column a thread.
      const uint32_t fours = rows / 4;
      for (uint32_t e = threadIdx.x - kWideWarps * 32 + rank * kJoinWarps * 32; e < fours * p.M;
           e += p.split * kJoinWarps * 32) {
        const int m = e / fours, r = e % fours * 4;
        if (n0 + r >= p.N) continue;
        float4 v[8][kParts];
#pragma unroll
        for (int z = 0; z < 8; ++z)
          if (z < p.split) {
#pragma unroll
            for (int q = 0; q < kParts; ++q)
              v[z][q] = remote_float4(s + (m * kParts + q) * kRoundPitch + r, z);
          }
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int z = 0; z < 8; ++z)
          if (z < p.split) y = add4(y, kParts == 2 ? add4(v[z][kParts - 1], v[z][0]) : v[z][0]);
        const int64_t at = m * p.N + n0 + r;
        const float out[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (n0 + r + h < p.N) store_y(p.y, p.y_dtype, at + h, out[h]);
      }
    }
  }
  // No CTA leaves while others read its sums.
  cluster_arrive();
  cluster_wait();
  if (p.overlap == 2 && warp < kWideWarps) dependency_wait();
}

// The split of K over a cluster orders the additions, so it depends on the
// matrix and the SM count only; the warps of the narrow kernel's CTAs come with
// it.  A CTA's time is its passes times (its tiles + the start of a pass, worth
// about 6 tiles), and a cluster's join is worth about 4 more; taken where that
// is least, for a full device.  The narrow kernel's passes alone count here:
// whether the range's fragments fit the wide kernel does not, so for more than
// 8 columns K = 4096 (16 pairs, split 1) runs 8 at a time and K = 5120 (4 pairs,
// split 5) 32: 236 against 145 us at M = 32 and 131072 rows.  (Against every other choice, measured: 5120 x
// 17408 16.3 us, the best 15.1, four warps always 17.4; 1280 x 17408 6.6, 6.5,
// 8.8; 10240 x 5120 and 4096 x 14336 are the best ones; 131072 x 5120 63.8 and
// 62.8.)
struct W4Split {
  int split, warps;
};
W4Split w4_split(int tiles, int units, int sms) {
  // The last shape's choice: 32 candidates cost as much as the launch's checks.
  static thread_local struct {
    int tiles, units, sms;
    W4Split split;
  } last{0, 0, 0, {1, 4}};
  if (last.tiles == tiles && last.units == units && last.sms == sms) return last.split;
  W4Split best{1, 4};
  int64_t least = INT64_MAX;
  for (int w = 4; w <= kMaxWarps; w += 4)
    for (int c = 1; c <= 8 && c <= units; ++c) {
      const int pairs = ((units + c - 1) / c + 1) / 2, passes = (pairs + w - 1) / w;
      const int clusters = std::max(1, ctas_of(w) * sms / c);
      const int64_t cost = (int64_t)passes * ((tiles + clusters - 1) / clusters + 6) + (c > 1 ? 4 : 0);
      if (cost < least) least = cost, best = {c, w};
    }
  last = {tiles, units, sms, best};
  return best;
}

// Clusters of `kern` that fit the device at once, looked up once per device
// and cluster size.
template <typename Kernel>
int resident_clusters(Kernel kern, std::atomic<int> (&known)[64][9], int split, int threads,
                      int smem, int* most) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PQ2_ERR_CUDA;
  *most = known[dev][split].load(std::memory_order_acquire);
  if (*most) return PQ2_OK;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(most, kern, &cfg) != cudaSuccess || *most < 1) {
    cudaGetLastError();
    return PQ2_ERR_CUDA;
  }
  known[dev][split].store(*most, std::memory_order_release);
  return PQ2_OK;
}

template <typename Kernel>
int launch(Kernel kern, const W4Params& p, int clusters, int threads, int smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(clusters * p.split));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  return PQ2_OK;
}

template <typename XT, int GROUP, bool ZEROS>
int launch_narrow(W4Params p, cudaStream_t stream) {
  static std::atomic<int> known[kMaxWarps / 4][64][9];
  auto kern = w4_mmv_kernel<XT, GROUP, ZEROS>;
  const int room = smem_of(p.warps);
  int most = 0;
  if (int st = resident_clusters(kern, known[p.warps / 4 - 1], p.split, p.warps * 32, room, &most))
    return st;
  const int pairs = ((p.units + p.split - 1) / p.split + 1) / 2;
  const int warps = std::min(p.warps, pairs);
  // Equal shares: the clusters that run at once take as many tiles each.
  const int each = (p.tiles + most - 1) / most;
  const int clusters = (p.tiles + each - 1) / each;
  const int cols = p.M * parts<XT>();
  const int ring = warps * kStages * 2 * unit_bytes(GROUP, ZEROS);
  const int red_tile = warps * cols * kPitch * 4, acc_tile = cols * kTileRows * 4;
  const auto red = [&](int log) { return 2 * (red_tile << log); };
  p.batch_log = 0;
  while (p.batch_log < 3 && 1 << p.batch_log < each && red(p.batch_log + 1) <= p.warps * 4096 &&
         ring + red(p.batch_log + 1) + 4 * acc_tile <= room)
    ++p.batch_log;
  p.block_tiles = std::min(each, (room - ring - red(p.batch_log)) / acc_tile);
  if (p.block_tiles < 1) return PQ2_ERR_SHAPE;
  return launch(kern, p, clusters, warps * 32,
                ring + red(p.batch_log) + p.block_tiles * acc_tile, stream);
}

template <typename XT, int NT, int GROUP, bool ZEROS>
int launch_wide(const W4Params& p, cudaStream_t stream) {
  static std::atomic<int> known[64][9];
  auto kern = w4_wide_kernel<XT, NT, GROUP, ZEROS>;
  constexpr int kThreads = (kWideWarps + kJoinWarps) * 32;
  int most = 0;
  if (int st = resident_clusters(kern, known, p.split, kThreads, kWideSmem, &most)) return st;
  // Equal shares, which need not be whole rounds: a short last round leaves some
  // warps without a tile.
  const int each = (p.tiles + most - 1) / most;
  const int clusters = (p.tiles + each - 1) / each;
  const int pairs = ((p.units + p.split - 1) / p.split + 1) / 2;
  return launch(kern, p, clusters, kThreads, wide_smem<NT>(pairs, unit_bytes(GROUP, ZEROS)), stream);
}

template <typename XT, int GROUP, bool ZEROS>
int launch_cols(W4Params p, int64_t M, cudaStream_t stream) {
  // As many MMA columns at a time as the wide kernel's shared memory takes for
  // this matrix (32, 24 or 16), else the narrow kernel's 8.
  constexpr int kUnitB = unit_bytes(GROUP, ZEROS), kParts = parts<XT>();
  const int pairs = ((p.units + p.split - 1) / p.split + 1) / 2;
  const int most = wide_smem<4>(pairs, kUnitB) <= kWideSmem   ? 32
                   : wide_smem<3>(pairs, kUnitB) <= kWideSmem ? 24
                   : wide_smem<2>(pairs, kUnitB) <= kWideSmem ? 16
                                                              : 8;
  const int y_size = p.y_dtype == PQ2_F32 ? 4 : 2;
  for (int64_t m = 0; m < M; m += most / kParts) {
    W4Params q = p;
    q.M = (int)std::min<int64_t>(most / kParts, M - m);
    q.x = static_cast<const XT*>(p.x) + m * p.ldx;
    q.y = static_cast<uint8_t*>(p.y) + m * p.N * y_size;
    const int cols = q.M * kParts;
    const int st = cols <= 8    ? launch_narrow<XT, GROUP, ZEROS>(q, stream)
                   : cols <= 16 ? launch_wide<XT, 2, GROUP, ZEROS>(q, stream)
                   : cols <= 24 ? launch_wide<XT, 3, GROUP, ZEROS>(q, stream)
                                : launch_wide<XT, 4, GROUP, ZEROS>(q, stream);
    if (st) return st;
  }
  return PQ2_OK;
}

template <typename XT>
int launch_x(W4Params p, int64_t M, int group, bool zeros, cudaStream_t stream) {
  p.vector_x = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx * sizeof(XT) % 16 == 0;
  switch (group * 2 + zeros) {
    case 256: return launch_cols<XT, 128, false>(p, M, stream);
    case 257: return launch_cols<XT, 128, true>(p, M, stream);
    case 128: return launch_cols<XT, 64, false>(p, M, stream);
    case 129: return launch_cols<XT, 64, true>(p, M, stream);
    case 64: return launch_cols<XT, 32, false>(p, M, stream);
    default: return launch_cols<XT, 32, true>(p, M, stream);
  }
}

}  // namespace

size_t w4_plane_bytes(int64_t N, int64_t K, int group, bool zeros) {
  const int64_t tiles = (N + kTileRows - 1) / kTileRows, units = (K + kUnitK - 1) / kUnitK;
  return (size_t)tiles * (size_t)units * (size_t)unit_bytes(group, zeros);
}

int launch_w4_prepare(const uint8_t* codes, int64_t ldc, const uint16_t* scales,
                      const uint8_t* zeros, int64_t N, int64_t K, int group, uint8_t* plane,
                      cudaStream_t stream) {
  W4PrepParams p{codes, scales, zeros, plane, ldc, N, K, (K + kUnitK - 1) / kUnitK, 0, group};
  p.total = (N + kTileRows - 1) / kTileRows * p.units;
  const int64_t blocks = (p.total + 7) / 8;
  if (blocks > 0x7FFFFFFF) return PQ2_ERR_SHAPE;
  w4_prepare_kernel<<<(unsigned)blocks, 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PQ2_OK : PQ2_ERR_LAUNCH;
}

int launch_w4_mmv(const void* x, int x_dtype, int64_t ldx, int64_t M, int64_t N, int64_t K,
                  int group, bool zeros, const uint8_t* plane, void* y, int y_dtype,
                  int overlap, int sm_count, cudaStream_t stream) {
  const int64_t tiles = (N + kTileRows - 1) / kTileRows;
  W4Params p{};
  p.x = x, p.plane = plane, p.y = y, p.ldx = ldx, p.N = N, p.K = (int)K, p.y_dtype = y_dtype;
  p.tiles = (int)tiles, p.units = (int)((K + kUnitK - 1) / kUnitK), p.overlap = overlap;
  const W4Split split = w4_split(p.tiles, p.units, sm_count);
  p.split = split.split, p.warps = split.warps;
  if (x_dtype == PQ2_BF16) return launch_x<__nv_bfloat16>(p, M, group, zeros, stream);
  if (x_dtype == PQ2_F16) return launch_x<__half>(p, M, group, zeros, stream);
  return launch_x<float>(p, M, group, zeros, stream);
}

}  // namespace pq2
