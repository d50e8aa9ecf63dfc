// pq2_norm.cu — the norms after a block and before the next one, fused with
// the block's gate and residual scale (pq2_norm_gate_residual):
//   p  = z / sqrt(mean z^2 + eps) * (w_post + o)   (or z without w_post)
//   h' = h + alpha * gate * p
//   n  = h' / sqrt(mean h'^2 + eps) * (w_pre + o)
// in fp32, each output rounded once.
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

constexpr int kThreads = 256;

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float v, float* o) { *o = v; }
__device__ __forceinline__ void narrow(float v, __half* o) { *o = __float2half_rn(v); }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16* o) { *o = __float2bfloat16_rn(v); }

__device__ __forceinline__ float block_sum(float v, float* buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) v += buf[w];
  __syncthreads();
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_kernel(NormParams p) {
  __shared__ float buf[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = blockIdx.x;
  const T* z = static_cast<const T*>(p.z) + row * p.ldz;
  const T* h = static_cast<const T*>(p.h) + row * p.ldh;
  const T* gate = p.gate ? static_cast<const T*>(p.gate) + row / p.rows_per_gate * p.ldg : nullptr;
  const T* w_post = static_cast<const T*>(p.w_post);
  float inv = 1.f;
  if (p.z && w_post) {
    float s = 0.f;
    for (int64_t j = threadIdx.x; j < p.K; j += kThreads) s = fmaf(widen(z[j]), widen(z[j]), s);
    inv = 1.f / sqrtf(block_sum(s, buf) / (float)p.K + p.eps);
  }
  // h' is formed again after its norm: h_out may be h, so it is written last.
  auto sum = [&](int64_t j) {
    float v = widen(h[j]);
    if (!p.z) return v;
    float q = widen(z[j]);
    if (w_post) q = q * inv * (widen(w_post[j]) + p.w_offset);
    if (gate) q *= widen(gate[j]);
    return fmaf(p.alpha, q, v);
  };
  float s = 0.f;
  for (int64_t j = threadIdx.x; j < p.K; j += kThreads) {
    const float v = sum(j);
    s = fmaf(v, v, s);
  }
  const float inv_n = 1.f / sqrtf(block_sum(s, buf) / (float)p.K + p.eps);
  for (int64_t j = threadIdx.x; j < p.K; j += kThreads) {
    const float v = sum(j);
    if (p.h_out) narrow(v, static_cast<T*>(p.h_out) + row * p.K + j);
    if (p.n_out)
      narrow(v * inv_n * (widen(static_cast<const T*>(p.w_pre)[j]) + p.w_offset),
             static_cast<T*>(p.n_out) + row * p.K + j);
  }
}

template <typename T>
int launch_type(const NormParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.M);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, norm_kernel<T>, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  return PQ2_OK;
}

}  // namespace

int launch_norm(const NormParams& p, int dtype, int sm_count, cudaStream_t stream) {
  if (dtype == PQ2_BF16) return launch_type<__nv_bfloat16>(p, stream);
  if (dtype == PQ2_F16) return launch_type<__half>(p, stream);
  return launch_type<float>(p, stream);
}

}  // namespace pq2
