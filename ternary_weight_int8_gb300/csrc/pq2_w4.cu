// pq2_w4.cu — matrix-vector products with 4-bit weights and group scales
// (pq2_w4_prepare, pq2_w4_mmv):
//   y[m][n] = sum_g s[n][g] * sum_{k in g} (c[n][k] - z[n][g]) * x[m][k]
//
// Plane layout.  Rows go in tiles of 16 and columns in units of 128; a unit
// (tile, 128 columns) is one contiguous block in the order in which a warp's
// mma.sync.m16n8k16 takes it as the A operand:
//   512 B   lane l's 16 bytes: words of MMA steps 0..3
//   512 B   lane l's 16 bytes: words of MMA steps 4..7
//   per group of the unit: 8 x (scale of row i, scale of row i + 8), fp16
//   with zero points, per group: 8 x (zero of row i | zero of row i + 8 << 4)
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
  for (int e = lane; e < groups * 16; e += 32) {  // e = group, pair, half
    const int64_t g = u * groups + e / 16, n = tile * kTileRows + (e % 16) / 2 + 8 * (e & 1);
    scales[e] = g < row_groups && n < p.N ? p.scales[n * row_groups + g] : 0;
  }
  if (p.zeros)
    for (int e = lane; e < groups * 8; e += 32) {
      const int64_t g = u * groups + e / 8, n = tile * kTileRows + e % 8;
      uint32_t z = 0;
      if (g < row_groups && n < p.N) z = p.zeros[n * row_groups + g] & 15u;
      if (g < row_groups && n + 8 < p.N) z |= (p.zeros[(n + 8) * row_groups + g] & 15u) << 4;
      zeros[e] = (uint8_t)z;
    }
}

// ---------------------------------------------------------------------------
// Product.

struct W4Params {
  const void* x;
  const uint8_t* plane;
  void* y;
  int64_t ldx, N;
  int M, K, units, y_dtype;
};

// x as MMA columns: 16-bit types are taken as they are; a 32-bit x is the sum
// of three bf16 parts (24 bits of mantissa), each a column of its own.
template <typename XT>
struct Operand {
  using T = XT;
  static constexpr int kParts = 1;
};
template <>
struct Operand<float> {
  using T = __nv_bfloat16;
  static constexpr int kParts = 3;
};

template <typename T>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The offset that turns a code into c - z in the operand type: a code OR-ed
// into the mantissa of 128 (bf16) or 1024 (fp16) is exactly 128 + c or
// 1024 + c, and subtracting 128 + z or 1024 + z is exact.
template <typename T>
struct Magic;
template <>
struct Magic<__nv_bfloat16> {
  static constexpr uint32_t kBits = 0x43004300u;
  static __device__ __forceinline__ uint32_t sub(uint32_t v, uint32_t off) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v),
                                     *reinterpret_cast<__nv_bfloat162*>(&off));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct Magic<__half> {
  static constexpr uint32_t kBits = 0x64006400u;
  static __device__ __forceinline__ uint32_t sub(uint32_t v, uint32_t off) {
    const __half2 r =
        __hsub2(*reinterpret_cast<__half2*>(&v), *reinterpret_cast<__half2*>(&off));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

// The A fragment (rows i and i + 8) of one step's word.
template <typename T>
__device__ __forceinline__ void decode(uint32_t w, uint32_t off0, uint32_t off1, uint32_t* a) {
  a[0] = Magic<T>::sub((w & 0x000F000Fu) | Magic<T>::kBits, off0);
  a[1] = Magic<T>::sub(((w >> 4) & 0x000F000Fu) | Magic<T>::kBits, off1);
  a[2] = Magic<T>::sub(((w >> 8) & 0x000F000Fu) | Magic<T>::kBits, off0);
  a[3] = Magic<T>::sub(((w >> 12) & 0x000F000Fu) | Magic<T>::kBits, off1);
}

// Part `part` of the 8 consecutive elements x[0..8) of one column as the two
// B register pairs of two steps; zeros where the column does not exist.
template <typename XT>
__device__ __forceinline__ uint4 load_b(const XT* x, int part, bool on) {
  uint32_t r[4] = {};
  if (on) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (std::is_same<XT, float>::value) {
        float v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float f = x[2 * e + h];
          for (int q = 0; q < part; ++q) f -= __bfloat162float(__float2bfloat16(f));
          v[h] = f;
        }
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[0], v[1]);
        r[e] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        const uint16_t* xb = reinterpret_cast<const uint16_t*>(x);
        r[e] = xb[2 * e] | (uint32_t)xb[2 * e + 1] << 16;
      }
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ void store_y(void* y, int dtype, int64_t at, float v) {
  if (dtype == PQ2_F32) reinterpret_cast<float*>(y)[at] = v;
  else if (dtype == PQ2_BF16) reinterpret_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16(v);
  else reinterpret_cast<__half*>(y)[at] = __float2half(v);
}

constexpr int kWarps = 8;

// One CTA per tile: its warps take the tile's units in turn, and their sums
// are added through shared memory in warp order.
template <typename XT, int NT, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kWarps * 32) w4_mmv_kernel(W4Params p) {
  using T = typename Operand<XT>::T;
  constexpr int kParts = Operand<XT>::kParts;
  constexpr int kGroups = kUnitK / GROUP, kSteps = GROUP / 16;
  __shared__ float red[kWarps][kTileRows][8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float acc[NT][4] = {};
  for (int u = warp; u < p.units; u += kWarps) {
    const uint8_t* unit =
        p.plane + ((int64_t)blockIdx.x * p.units + u) * unit_bytes(GROUP, ZEROS);
    const uint4 c0 = reinterpret_cast<const uint4*>(unit)[lane];
    const uint4 c1 = reinterpret_cast<const uint4*>(unit + 512)[lane];
    const uint32_t words[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    uint4 b[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int v = 8 * nt + i, m = v / kParts;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = u * kUnitK + 32 * j + 8 * t;
        const bool on = m < p.M && k < p.K;
        b[nt][j] = load_b(static_cast<const XT*>(p.x) + (on ? m * p.ldx + k : 0), v % kParts, on);
      }
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const uint32_t sc = reinterpret_cast<const uint32_t*>(unit + kUnitCodeBytes)[8 * g + i];
      const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&sc));
      uint32_t z0 = 8, z1 = 8;
      if (ZEROS) {
        const uint32_t z = unit[kUnitCodeBytes + 32 * kGroups + 8 * g + i];
        z0 = z & 15, z1 = z >> 4;
      }
      const uint32_t off0 = Magic<T>::kBits + z0 * 0x10001u, off1 = Magic<T>::kBits + z1 * 0x10001u;
      float d[NT][4] = {};
#pragma unroll
      for (int s2 = 0; s2 < kSteps; ++s2) {
        const int step = g * kSteps + s2;
        uint32_t a[4];
        decode<T>(words[step], off0, off1, a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 bb = b[nt][step / 2];
          mma16816<T>(d[nt], a, step % 2 ? bb.z : bb.x, step % 2 ? bb.w : bb.y);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        acc[nt][0] = fmaf(s.x, d[nt][0], acc[nt][0]);
        acc[nt][1] = fmaf(s.x, d[nt][1], acc[nt][1]);
        acc[nt][2] = fmaf(s.y, d[nt][2], acc[nt][2]);
        acc[nt][3] = fmaf(s.y, d[nt][3], acc[nt][3]);
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    red[warp][i][8 * nt + 2 * t] = acc[nt][0];
    red[warp][i][8 * nt + 2 * t + 1] = acc[nt][1];
    red[warp][i + 8][8 * nt + 2 * t] = acc[nt][2];
    red[warp][i + 8][8 * nt + 2 * t + 1] = acc[nt][3];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kTileRows * p.M; e += kWarps * 32) {
    const int m = e / kTileRows, r = e % kTileRows;
    const int64_t n = (int64_t)blockIdx.x * kTileRows + r;
    if (n >= p.N) continue;
    float sum = 0.f;
    for (int q = kParts - 1; q >= 0; --q)  // the smallest part first
      for (int w = 0; w < kWarps; ++w) sum += red[w][r][m * kParts + q];
    store_y(p.y, p.y_dtype, (int64_t)m * p.N + n, sum);
  }
}

template <typename XT, int NT, int GROUP, bool ZEROS>
int launch_one(const W4Params& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((p.N + kTileRows - 1) / kTileRows));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, w4_mmv_kernel<XT, NT, GROUP, ZEROS>, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  return PQ2_OK;
}

template <typename XT, int NT>
int launch_nt(const W4Params& p, int group, bool zeros, cudaStream_t stream) {
  if (group == 128) return zeros ? launch_one<XT, NT, 128, true>(p, stream) : launch_one<XT, NT, 128, false>(p, stream);
  if (group == 64) return zeros ? launch_one<XT, NT, 64, true>(p, stream) : launch_one<XT, NT, 64, false>(p, stream);
  return zeros ? launch_one<XT, NT, 32, true>(p, stream) : launch_one<XT, NT, 32, false>(p, stream);
}

template <typename XT>
int launch_x(W4Params p, int64_t M, int group, bool zeros, cudaStream_t stream) {
  // At most 32 MMA columns at a time: 32 columns of x, or 10 of a 32-bit x.
  constexpr int kMost = 32 / Operand<XT>::kParts;
  const int y_size = p.y_dtype == PQ2_F32 ? 4 : 2;
  for (int64_t m = 0; m < M; m += kMost) {
    W4Params q = p;
    q.M = (int)std::min<int64_t>(kMost, M - m);
    q.x = static_cast<const XT*>(p.x) + m * p.ldx;
    q.y = static_cast<uint8_t*>(p.y) + m * p.N * y_size;
    int st;
    switch ((q.M * Operand<XT>::kParts + 7) / 8) {
      case 1: st = launch_nt<XT, 1>(q, group, zeros, stream); break;
      case 2: st = launch_nt<XT, 2>(q, group, zeros, stream); break;
      case 3: st = launch_nt<XT, 3>(q, group, zeros, stream); break;
      default: st = launch_nt<XT, 4>(q, group, zeros, stream); break;
    }
    if (st) return st;
  }
  return PQ2_OK;
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
  W4Params p{x, plane, y, ldx, N, (int)M, (int)K, (int)((K + kUnitK - 1) / kUnitK), y_dtype};
  if (x_dtype == PQ2_BF16) return launch_x<__nv_bfloat16>(p, M, group, zeros, stream);
  if (x_dtype == PQ2_F16) return launch_x<__half>(p, M, group, zeros, stream);
  return launch_x<float>(p, M, group, zeros, stream);
}

}  // namespace pq2
