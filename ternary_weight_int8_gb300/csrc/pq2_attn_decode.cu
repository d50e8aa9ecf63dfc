// pq2_attn_decode.cu — attention of new tokens over a paged cache.
//
// A warp takes one query row and walks its keys with the running maximum m
// and sum l of a softmax: for a score s (in units of ln 2) the new maximum is
// M = max(m, s), and l and the output sum are scaled by 2^(m - M) before
// 2^(s - M) and 2^(s - M) v are added.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pq2_internal.h"

namespace pq2 {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(int8_t x) { return (float)x; }
template <typename T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ __half narrow(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 narrow(float x) {
  return __float2bfloat16_rn(x);
}

// key(j, &k, &v, &ks, &vs): the addresses and scales of position j, false if
// it reads as zeros.
template <typename QT, typename CT, int D, typename Key>
__device__ __forceinline__ void row(const QT* q, float scale, int64_t most, Key key, QT* out,
                                    float* lse) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  float x[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = widen(q[lane * E + e]) * (scale * kLog2e);
  for (int64_t j = 0; j < most; ++j) {
    const CT *k, *v;
    float ks, vs, s = 0.f;
    const bool there = key(j, &k, &v, &ks, &vs);
    if (there) {
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(x[e], widen(k[lane * E + e]), s);
    }
#pragma unroll
    for (int i = 16; i; i /= 2) s += __shfl_xor_sync(~0u, s, i);
    if (there) s *= ks;
    const float top = fmaxf(m, s), old = m > -INFINITY ? exp2f(m - top) : 0.f;
    const float p = top > -INFINITY ? exp2f(s - top) : 0.f;
    l = l * old + p;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = fmaf(p, there ? widen(v[lane * E + e]) * vs : 0.f, o[e] * old);
    m = top;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane * E + e] = narrow<QT>(most > 0 ? o[e] / l : 0.f);
  if (lse && lane == 0) *lse = most > 0 ? m * kLn2 + logf(l) : -INFINITY;
}

template <typename QT, typename CT, int D>
__global__ void __launch_bounds__(128) decode_kernel(const DecodeParams p, const pq2_kv_cache c) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (int64_t)p.batch.B * p.T * p.q_heads) return;
  const int h = (int)(item % p.q_heads), t = (int)(item / p.q_heads % p.T);
  const int64_t b = item / p.q_heads / p.T;
  const int64_t kh = h / (p.q_heads / (int)c.heads);
  const int64_t most = (int64_t)__ldg(p.batch.lens + b) - p.T + t + 1;
  const auto key = [&](int64_t j, const CT** k, const CT** v, float* ks, float* vs) {
    const int64_t at = j / c.page_size, slot = j % c.page_size;
    if (at >= p.batch.table_width) return false;
    const int64_t page = __ldg(p.batch.table + b * p.batch.table_stride + at);
    if (page < 0 || page >= c.pages) return false;
    const int64_t o = page * c.page_stride + kh * c.head_stride + slot * c.token_stride;
    *k = static_cast<const CT*>(c.k) + o, *v = static_cast<const CT*>(c.v) + o;
    *ks = *vs = 1.f;
    if (sizeof(CT) == 1) {
      const int64_t s = (page * c.heads + kh) * c.page_size + slot;
      *ks = c.k_scales[s], *vs = c.v_scales[s];
    }
    return true;
  };
  row<QT, CT, D>(static_cast<const QT*>(p.q) + b * p.batch_stride + t * p.token_stride +
                     h * p.head_stride,
                 p.scale, most, key, static_cast<QT*>(p.out) + item * D,
                 p.lse ? p.lse + item : nullptr);
}

template <typename K, typename... A>
int launch(K kernel, int64_t rows, cudaStream_t stream, const A&... args) {
  if ((rows + 3) / 4 > 0x7fffffff) return PQ2_ERR_SHAPE;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  return PQ2_OK;
}

template <typename QT, typename CT>
int launch_decode(const DecodeParams& p, const pq2_kv_cache& c, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.batch.B * p.T * p.q_heads;
  if (c.dim == 64) return launch(decode_kernel<QT, CT, 64>, rows, stream, p, c);
  if (c.dim == 128) return launch(decode_kernel<QT, CT, 128>, rows, stream, p, c);
  return launch(decode_kernel<QT, CT, 256>, rows, stream, p, c);
}

}  // namespace

size_t attn_decode_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 16; }

int launch_attn_decode(const DecodeParams& p, const pq2_kv_cache& c, int sm_count,
                       cudaStream_t stream) {
  (void)sm_count;
  if (p.dtype == PQ2_BF16)
    return c.dtype == PQ2_I8 ? launch_decode<__nv_bfloat16, int8_t>(p, c, stream)
                             : launch_decode<__nv_bfloat16, __nv_bfloat16>(p, c, stream);
  return c.dtype == PQ2_I8 ? launch_decode<__half, int8_t>(p, c, stream)
                           : launch_decode<__half, __half>(p, c, stream);
}

}  // namespace pq2
