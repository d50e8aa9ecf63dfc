// pq2_kv.cu — the key-value cache as it is written and read back.
//
// A row (the token of a sequence) has 2 * heads units of D elements, its keys
// and then its values.  8-bit caches hold q = clamp(rne(x / s), +-127) with
// s = max|x| / 127 over a unit, pq2_quantize_act's rule with D in the place of
// 128; 16-bit caches x rounded to nearest even.
//
// Bound: HBM.  A warp takes kUnits loads of 32 x 8 elements of one row, all
// in flight before the first is used; D / 8 lanes share a unit, so its maximum
// is a few shuffles inside them and nothing passes through shared memory.  The
// row's sequence is found by the whole warp, 32 probes of cu at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pq2_internal.h"

namespace pq2 {
namespace {

constexpr int kUnits = 4;    // loads of a lane in flight
constexpr int kThreads = 256;

struct CacheView {
  uint8_t *k, *v;
  float *k_scales, *v_scales;
  int64_t page_stride, head_stride, token_stride;  // elements
  int pages, heads, page_size;
};

struct KvParams {
  CacheView c;
  KvBatch b;
  KvRows k, v;  // the packed rows
  int chunks;   // warps that share a row
};

// Page and slot of the row, or false where it has none; `mine` is false if it
// belongs to no sequence at all.  The whole warp calls it.
__device__ __forceinline__ bool locate(const KvParams& p, int64_t row, int lane, bool* mine,
                                       int64_t* page, int* slot) {
  const KvBatch& s = p.b;
  int b, n;
  int64_t first;
  if (s.cu) {
    // How many of the B + 1 sums are <= row.
    int lo = 0, hi = s.B + 1;
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const int c = __popc(__ballot_sync(~0u, at < hi && __ldg(s.cu + at) <= row));
      if (!c) break;
      const int end = lo + c * step;
      lo += (c - 1) * step + 1;
      hi = end < hi ? end : hi;
    }
    b = lo - 1;
    *mine = b >= 0 && b < s.B;
    if (!*mine) return false;
    first = __ldg(s.cu + b);
    n = (int)(__ldg(s.cu + b + 1) - first);
  } else {
    n = (int)(s.rows / s.B);
    b = (int)(row / n);
    first = (int64_t)b * n;
    *mine = true;
  }
  const int64_t pos = (int64_t)__ldg(s.lens + b) - n + (row - first);
  if (pos < 0) return false;
  const int64_t at = pos / p.c.page_size;
  if (at >= s.table_width) return false;
  const int pg = __ldg(s.table + (int64_t)b * s.table_stride + at);
  *page = pg, *slot = (int)(pos - at * p.c.page_size);
  return pg >= 0 && pg < p.c.pages;
}

template <typename T> __device__ __forceinline__ float widen(T x);
template <> __device__ __forceinline__ float widen(float x) { return x; }
template <> __device__ __forceinline__ float widen(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ float narrow(float x) { return x; }
template <> __device__ __forceinline__ __half narrow(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 narrow(float x) {
  return __float2bfloat16_rn(x);
}

template <typename T> struct alignas(sizeof(T) * 8 > 16 ? 16 : sizeof(T) * 8) Eight { T x[8]; };

// The larger of both magnitudes, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct Unit {
  bool values;
  int head;
};

// XT: the packed rows' type; CT: the cache's; D: elements of a unit; VEC: the
// rows' pointers and strides are multiples of 16 bytes.
template <typename XT, typename CT, int D, bool VEC, bool STORE>
__global__ void __launch_bounds__(kThreads) kv_kernel(const KvParams p) {
  constexpr int L = D / 8, kPer = 32 / L;  // lanes of a unit, units of one load
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = item / p.chunks;
  if (row >= p.b.rows) return;
  const int unit0 = (int)(item % p.chunks) * (kPer * kUnits) + lane / L, d = (lane % L) * 8;
  bool mine;
  int64_t page = 0;
  int slot = 0;
  const bool there = locate(p, row, lane, &mine, &page, &slot);
  if (STORE ? !there : !mine) return;
  const int64_t base = page * p.c.page_stride + (int64_t)slot * p.c.token_stride + d;
  const int64_t side = page * p.c.heads * p.c.page_size + slot;
  const auto unit = [&](int i) {
    const int u = unit0 + i * kPer;
    return Unit{u >= p.c.heads, u >= p.c.heads ? u - p.c.heads : u};
  };
  const auto cached = [&](Unit u) {
    return reinterpret_cast<Eight<CT>*>(reinterpret_cast<CT*>(u.values ? p.c.v : p.c.k) + base +
                                        u.head * p.c.head_stride);
  };
  const auto scale_at = [&](Unit u) {
    return (u.values ? p.c.v_scales : p.c.k_scales) + side + (int64_t)u.head * p.c.page_size;
  };
  const auto packed = [&](Unit u) {
    const KvRows& r = u.values ? p.v : p.k;
    return static_cast<XT*>(r.p) + row * r.token_stride + u.head * r.head_stride + d;
  };
  if constexpr (STORE) {
    Eight<XT> x[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const Unit u = unit(i);
      if (u.head >= p.c.heads) break;
      const XT* from = packed(u);
      if constexpr (VEC) {
        x[i] = *reinterpret_cast<const Eight<XT>*>(from);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i].x[j] = from[j];
      }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const Unit u = unit(i);
      const bool live = u.head < p.c.heads;
      Eight<CT> y;
      if constexpr (sizeof(CT) == 1) {
        float top = 0.f;
        if (live) {
#pragma unroll
          for (int j = 0; j < 8; ++j) top = max_nan(top, fabsf(widen(x[i].x[j])));
        }
#pragma unroll
        for (int o = L / 2; o; o /= 2) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
        const float s = __fdiv_rn(top, 127.f), by = s > 0.f ? s : 1.f;
        if (live) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int q = __float2int_rn(__fdiv_rn(widen(x[i].x[j]), by));
            y.x[j] = (CT)min(max(q, -127), 127);
          }
          if (d == 0) *scale_at(u) = s;
        }
      } else if (live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y.x[j] = narrow<CT>(widen(x[i].x[j]));
      }
      if (live) *cached(u) = y;
    }
  } else {
    Eight<CT> x[kUnits];
    float s[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const Unit u = unit(i);
      if (u.head >= p.c.heads) break;
      if (there) {
        x[i] = *cached(u);
        if constexpr (sizeof(CT) == 1) s[i] = *scale_at(u);
      } else {
        x[i] = Eight<CT>{}, s[i] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const Unit u = unit(i);
      if (u.head >= p.c.heads) break;
      Eight<XT> y;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (sizeof(CT) == 1)
          y.x[j] = narrow<XT>((float)x[i].x[j] * s[i]);
        else
          y.x[j] = narrow<XT>(widen(x[i].x[j]));
      }
      *reinterpret_cast<Eight<XT>*>(packed(u)) = y;
    }
  }
}

template <typename XT, typename CT, int D, bool VEC, bool STORE>
int launch(KvParams& p, cudaStream_t stream) {
  constexpr int kPer = 32 / (D / 8) * kUnits;
  p.chunks = (2 * p.c.heads + kPer - 1) / kPer;
  const int64_t blocks = (p.b.rows * p.chunks + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffff) return PQ2_ERR_SHAPE;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv_kernel<XT, CT, D, VEC, STORE>, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  return PQ2_OK;
}

template <typename XT, typename CT, bool VEC, bool STORE>
int launch_dim(KvParams& p, int dim, cudaStream_t stream) {
  if (dim == 64) return launch<XT, CT, 64, VEC, STORE>(p, stream);
  if (dim == 128) return launch<XT, CT, 128, VEC, STORE>(p, stream);
  return launch<XT, CT, 256, VEC, STORE>(p, stream);
}

template <typename XT, bool VEC, bool STORE>
int launch_cache(KvParams& p, const pq2_kv_cache& c, cudaStream_t stream) {
  if (c.dtype == PQ2_I8) return launch_dim<XT, int8_t, VEC, STORE>(p, (int)c.dim, stream);
  if (c.dtype == PQ2_F16) return launch_dim<XT, __half, VEC, STORE>(p, (int)c.dim, stream);
  return launch_dim<XT, __nv_bfloat16, VEC, STORE>(p, (int)c.dim, stream);
}

template <bool VEC, bool STORE>
int launch_type(KvParams& p, const pq2_kv_cache& c, int dtype, cudaStream_t stream) {
  if (dtype == PQ2_BF16) return launch_cache<__nv_bfloat16, VEC, STORE>(p, c, stream);
  if (dtype == PQ2_F16) return launch_cache<__half, VEC, STORE>(p, c, stream);
  return launch_cache<float, VEC, STORE>(p, c, stream);
}

CacheView view(const pq2_kv_cache& c) {
  return {static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.k_scales, c.v_scales,
          c.page_stride, c.head_stride, c.token_stride, (int)c.pages, (int)c.heads,
          (int)c.page_size};
}

}  // namespace

int launch_kv_store(KvRows k, KvRows v, int dtype, const pq2_kv_cache& c, const KvBatch& b,
                    cudaStream_t stream) {
  KvParams p{view(c), b, k, v, 0};
  const int e = dtype == PQ2_F32 ? 4 : 2;
  const uint64_t bits = reinterpret_cast<uintptr_t>(k.p) | reinterpret_cast<uintptr_t>(v.p) |
                        (uint64_t)(k.token_stride | k.head_stride | v.token_stride |
                                   v.head_stride) * e;
  return bits % 16 ? launch_type<false, true>(p, c, dtype, stream)
                   : launch_type<true, true>(p, c, dtype, stream);
}

int launch_kv_load(const pq2_kv_cache& c, const KvBatch& b, void* k, void* v, int dtype,
                   cudaStream_t stream) {
  const int64_t row = c.heads * c.dim;
  KvParams p{view(c), b, {k, row, c.dim}, {v, row, c.dim}, 0};
  return launch_type<true, false>(p, c, dtype, stream);
}

}  // namespace pq2
