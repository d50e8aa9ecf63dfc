// pq2_kv.cu — the key-value cache as it is written and read back.
//
// A row (the token of a sequence) has 2 * heads units of D elements, its keys
// and then its values.  8-bit caches hold q = clamp(rne(x / s), +-127) with
// s = max|x| / 127 over a unit, pq2_quantize_act's rule with D in the place of
// 128; 16-bit caches x rounded to nearest even.
//
// Bound: HBM.  A CTA takes up to 16 consecutive rows with all their units, so
// that both sides are long runs: a head's slots in a page, and whole rows of
// the packed side (one row a CTA: twice the time).  Its first threads find the
// rows' places (a search of cu, one look at lens and at the table) once for all
// units; then D / 8 threads share a unit, 8 elements each, and its maximum is a
// few shuffles inside them.  Eight CTAs an SM have enough loads in flight; 2 or
// 4 a thread, for which fewer threads fit, were slower.  131072 tokens of 8 heads of
// 128: from bf16 into 8 bits 222 us (0.54 of the copy rate: the codes' arithmetic),
// back 145 (0.82), 16 bits 164 and 162 (0.97).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "pq2_internal.h"

namespace pq2 {
namespace {

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
  int shift;    // a CTA's rows: 1 << shift
};

// Where the row lies in the cache, in elements of k and of its scales; -1 if
// it is in no page, -2 if it belongs to no sequence.
struct Place {
  int64_t at, side;
};
__device__ __forceinline__ Place locate(const KvParams& p, int64_t row) {
  const KvBatch& s = p.b;
  int b, n;
  int64_t first;
  if (row >= s.rows) return {-2, 0};
  if (s.cu) {
    int lo = 0, hi = s.B + 1;  // how many of the B + 1 sums are <= row
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(s.cu + mid) <= row) lo = mid + 1; else hi = mid;
    }
    b = lo - 1;
    if (b < 0 || b >= s.B) return {-2, 0};
    first = __ldg(s.cu + b);
    n = (int)(__ldg(s.cu + b + 1) - first);
  } else {
    n = (int)(s.rows / s.B);
    b = (int)(row / n);
    first = (int64_t)b * n;
  }
  const int64_t pos = (int64_t)__ldg(s.lens + b) - n + (row - first);
  if (pos < 0) return {-1, 0};
  const int64_t at = pos / p.c.page_size, slot = pos - at * p.c.page_size;
  if (at >= s.table_width) return {-1, 0};
  const int64_t page = __ldg(s.table + (int64_t)b * s.table_stride + at);
  if (page < 0 || page >= p.c.pages) return {-1, 0};
  return {page * p.c.page_stride + slot * p.c.token_stride,
          page * p.c.heads * p.c.page_size + slot};
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

// (a0, a1) * (b, b) + (c0, c1), two IEEE results.
__device__ __forceinline__ float2 fma2(float2 a, float b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\t"
      "mov.b64 c, {%5, %6};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b), "f"(c.x), "f"(c.y));
  return r;
}
// The largest magnitude of eight elements, NaN if one is.
__device__ __forceinline__ float largest(const Eight<float>& x) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(x.x[e]));
  return top;
}
template <typename T, typename T2>
__device__ __forceinline__ float largest_of_pairs(const Eight<T>& x) {
  const T2* y = reinterpret_cast<const T2*>(&x);
  const T2 top = __hmax2_nan(__hmax2_nan(__habs2(y[0]), __habs2(y[1])),
                             __hmax2_nan(__habs2(y[2]), __habs2(y[3])));
  return max_nan(widen(top.x), widen(top.y));
}
__device__ __forceinline__ float largest(const Eight<__half>& x) {
  return largest_of_pairs<__half, __half2>(x);
}
__device__ __forceinline__ float largest(const Eight<__nv_bfloat16>& x) {
  return largest_of_pairs<__nv_bfloat16, __nv_bfloat162>(x);
}

template <typename XT> __device__ __forceinline__ float clamped(float x) {
  return sizeof(XT) == 4 ? fminf(fmaxf(x, -127.f), 127.f) : x;
}

// Eight codes of a unit: q = clamp(rne(x / s)).  The quotient is first taken as
// t = x * (1 / s), which is within 3e-5 of it (|t| <= 127, three roundings) and
// so rounds alike unless it lies within 1e-4 of a half: then the warp divides.
// t + 1.5 * 2^23 rounds t to nearest even and has the code in its low byte.  The
// clamp has something to do for subnormal s only, by which the warp divides: s is a
// coarse rounding of max|x| / 127 then, and |x / s| passes 127.5 in fp32 (not in
// bf16: max|x| >= 2^-133 leaves s 516 steps of 2^-149, and |x / s| below 127.13).
template <typename XT>
__device__ __forceinline__ uint2 quantise(const Eight<XT>& x, float s) {
  constexpr float kRound = 12582912.f;
  const float by = s > 0.f ? s : 1.f, inv = __frcp_rn(by);
  float2 t[4], r[4];
  float off = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    t[e] = fma2(make_float2(widen(x.x[2 * e]), widen(x.x[2 * e + 1])), inv, make_float2(-0.f, -0.f));
    r[e] = fma2(t[e], 1.f, make_float2(kRound, kRound));
    const float2 n = fma2(r[e], 1.f, make_float2(-kRound, -kRound)), f = fma2(n, -1.f, t[e]);
    off = fmaxf(off, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  // Or the reciprocal is out of range, the scale infinite or NaN.
  if (__any_sync(~0u, off > 0.4999f || !(by > 0x1p-120f && by < 0x1p120f))) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r[e].x = clamped<XT>(__fdiv_rn(widen(x.x[2 * e]), by)) + kRound;
      r[e].y = clamped<XT>(__fdiv_rn(widen(x.x[2 * e + 1]), by)) + kRound;
    }
  }
  const auto four = [](float2 a, float2 b) {
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
  };
  return make_uint2(four(r[0], r[1]), four(r[2], r[3]));
}
// Byte i of u, 128 above its code, as that code: 2^23 + u exactly, less 2^23 +
// 128 (a conversion of integers has a quarter of the rate).
template <int I>
__device__ __forceinline__ float code_value(uint32_t u) {
  return __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540 | I)) - 8388736.f;
}

// XT: the packed rows' type; CT: the cache's; D: elements of a unit; VEC: the
// rows' pointers and strides are multiples of 16 bytes.
template <typename XT, typename CT, int D, bool VEC, bool STORE>
__global__ void __launch_bounds__(kThreads, 8) kv_kernel(const KvParams p) {
  constexpr int L = D / 8, kPer = kThreads / L;  // threads of a unit, units at a time
  __shared__ Place places[16];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t row0 = (int64_t)blockIdx.x << p.shift;
  if (threadIdx.x < 1 << p.shift) places[threadIdx.x] = locate(p, row0 + threadIdx.x);
  __syncthreads();
  // A thread keeps its row and columns and steps through the heads, those of
  // the keys and then those of the values.
  const int d = threadIdx.x % L * 8, r = threadIdx.x / L & ((1 << p.shift) - 1);
  const int unit0 = threadIdx.x / L >> p.shift, step = kPer >> p.shift, units = 2 * p.c.heads;
  const Place at = places[r];
  const bool there = at.at >= 0, live = STORE ? there : at.at != -2;
  const auto cached = [&](int u) {
    const bool values = u >= p.c.heads;
    return reinterpret_cast<CT*>(values ? p.c.v : p.c.k) + at.at + d +
           (u - (values ? p.c.heads : 0)) * p.c.head_stride;
  };
  const auto scale = [&](int u) {
    const bool values = u >= p.c.heads;
    return (values ? p.c.v_scales : p.c.k_scales) + at.side +
           (int64_t)(u - (values ? p.c.heads : 0)) * p.c.page_size;
  };
  const auto packed = [&](int u) {
    const bool values = u >= p.c.heads;
    const KvRows& rows = values ? p.v : p.k;
    return static_cast<XT*>(rows.p) + (row0 + r) * rows.token_stride + d +
           (u - (values ? p.c.heads : 0)) * rows.head_stride;
  };
  for (int u = unit0; __any_sync(~0u, u < units); u += step) {
    const bool mine = live && u < units;
    if constexpr (STORE) {
      Eight<XT> x{};
      if (mine) {
        const XT* from = packed(u);
        if constexpr (VEC) {
          x = *reinterpret_cast<const Eight<XT>*>(from);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x.x[e] = from[e];
        }
      }
      if constexpr (sizeof(CT) == 1) {
        float top = largest(x);
#pragma unroll
        for (int o = L / 2; o; o /= 2) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
        // A unit that is not finite reads back as NaN.
        const float s = top < INFINITY ? __fdiv_rn(top, 127.f) : __uint_as_float(0x7FC00000u);
        const uint2 q = quantise(x, s);
        if (mine) {
          *reinterpret_cast<uint2*>(cached(u)) = q;
          if (d == 0) *scale(u) = s;
        }
      } else if (mine) {
        Eight<CT> y;
#pragma unroll
        for (int e = 0; e < 8; ++e) y.x[e] = narrow<CT>(widen(x.x[e]));
        *reinterpret_cast<Eight<CT>*>(cached(u)) = y;
      }
    } else if (mine) {
      Eight<CT> x{};
      float s = 0.f;
      if (there) {
        x = *reinterpret_cast<const Eight<CT>*>(cached(u));
        if constexpr (sizeof(CT) == 1) s = *scale(u);
      }
      Eight<XT> y;
      if constexpr (sizeof(CT) == 1) {
        const uint2 w = *reinterpret_cast<const uint2*>(&x);
        const uint32_t a = w.x ^ 0x80808080u, b = w.y ^ 0x80808080u;
        y.x[0] = narrow<XT>(code_value<0>(a) * s), y.x[1] = narrow<XT>(code_value<1>(a) * s);
        y.x[2] = narrow<XT>(code_value<2>(a) * s), y.x[3] = narrow<XT>(code_value<3>(a) * s);
        y.x[4] = narrow<XT>(code_value<0>(b) * s), y.x[5] = narrow<XT>(code_value<1>(b) * s);
        y.x[6] = narrow<XT>(code_value<2>(b) * s), y.x[7] = narrow<XT>(code_value<3>(b) * s);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y.x[e] = narrow<XT>(widen(x.x[e]));
      }
      *reinterpret_cast<Eight<XT>*>(packed(u)) = y;
    }
  }
}

template <typename XT, typename CT, int D, bool VEC, bool STORE>
int launch(KvParams& p, int sm_count, cudaStream_t stream) {
  // As many rows a CTA as leave two CTAs for every SM, 16 (8 of 256 columns) at
  // most.
  p.shift = 0;
  while (1 << p.shift < std::min(16, kThreads / (D / 8)) && p.b.rows >> (p.shift + 2) >= sm_count) ++p.shift;
  const int64_t blocks = (p.b.rows + (1 << p.shift) - 1) >> p.shift;
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
int launch_dim(KvParams& p, int dim, int sm_count, cudaStream_t stream) {
  if (dim == 64) return launch<XT, CT, 64, VEC, STORE>(p, sm_count, stream);
  if (dim == 128) return launch<XT, CT, 128, VEC, STORE>(p, sm_count, stream);
  return launch<XT, CT, 256, VEC, STORE>(p, sm_count, stream);
}

template <typename XT, bool VEC, bool STORE>
int launch_cache(KvParams& p, const pq2_kv_cache& c, int sm_count, cudaStream_t stream) {
  if (c.dtype == PQ2_I8) return launch_dim<XT, int8_t, VEC, STORE>(p, (int)c.dim, sm_count, stream);
  if (c.dtype == PQ2_F16) return launch_dim<XT, __half, VEC, STORE>(p, (int)c.dim, sm_count, stream);
  return launch_dim<XT, __nv_bfloat16, VEC, STORE>(p, (int)c.dim, sm_count, stream);
}

template <bool VEC, bool STORE>
int launch_type(KvParams& p, const pq2_kv_cache& c, int dtype, int sm_count,
                cudaStream_t stream) {
  if (dtype == PQ2_BF16) return launch_cache<__nv_bfloat16, VEC, STORE>(p, c, sm_count, stream);
  if (dtype == PQ2_F16) return launch_cache<__half, VEC, STORE>(p, c, sm_count, stream);
  return launch_cache<float, VEC, STORE>(p, c, sm_count, stream);
}

CacheView view(const pq2_kv_cache& c) {
  return {static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.k_scales, c.v_scales,
          c.page_stride, c.head_stride, c.token_stride, (int)c.pages, (int)c.heads,
          (int)c.page_size};
}

}  // namespace

int launch_kv_store(KvRows k, KvRows v, int dtype, const pq2_kv_cache& c, const KvBatch& b,
                    int sm_count, cudaStream_t stream) {
  KvParams p{view(c), b, k, v, 0};
  const int e = dtype == PQ2_F32 ? 4 : 2;
  const uint64_t bits = reinterpret_cast<uintptr_t>(k.p) | reinterpret_cast<uintptr_t>(v.p) |
                        (uint64_t)(k.token_stride | k.head_stride | v.token_stride |
                                   v.head_stride) * e;
  return bits % 16 ? launch_type<false, true>(p, c, dtype, sm_count, stream)
                   : launch_type<true, true>(p, c, dtype, sm_count, stream);
}

int launch_kv_load(const pq2_kv_cache& c, const KvBatch& b, void* k, void* v, int dtype,
                   int sm_count, cudaStream_t stream) {
  const int64_t row = c.heads * c.dim;
  KvParams p{view(c), b, {k, row, c.dim}, {v, row, c.dim}, 0};
  return launch_type<true, false>(p, c, dtype, sm_count, stream);
}

}  // namespace pq2
