// pq2_logprobs.cu — log-probabilities of given tokens, entropy and top
// alternatives of each row of logits (pq2_token_logprobs).
//
// With t = scale * x, m = max t over the row, u = t - m, S = sum exp(u) and
// W = sum exp(u) u:
//   log p_j = u_j - log S,    H = -sum p log p = log S - W / S.
// Logits of -inf are excluded (p = 0, and 0 log 0 = 0).
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

struct LogprobParams {
  const void* logits;
  const int64_t* tokens;
  float* token_lp;
  float* entropy;
  int64_t* top_ids;
  float* top_lp;
  int64_t ldl, V, T;
  float scale;
  int k;
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

// The order of the alternatives as one number: by value (-0 = +0, NaN below
// -inf), equal values by the lower index.  0 is below every element's key.
__device__ __forceinline__ uint64_t order_key(float v, uint32_t index) {
  v += 0.f;
  const uint32_t b = __float_as_uint(v);
  const uint32_t o = v != v ? 1u : (b >> 31 ? ~b : b | 0x80000000u);
  return (uint64_t)o << 32 | (0xFFFFFFFFu - index);
}

constexpr int kThreads = 256;

template <typename V>
__device__ __forceinline__ V block_reduce(V v, V* buf, V (*op)(V, V)) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = buf[0];
  for (int w = 1; w < kThreads / 32; ++w) v = op(v, buf[w]);
  __syncthreads();
  return v;
}
__device__ float op_max(float a, float b) { return fmaxf(a, b); }
__device__ float op_sum(float a, float b) { return a + b; }
__device__ unsigned long long op_umax(unsigned long long a, unsigned long long b) { return a > b ? a : b; }

template <typename XT>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(LogprobParams p) {
  __shared__ float fbuf[kThreads / 32];
  __shared__ unsigned long long kbuf[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = blockIdx.x;
  const XT* x = static_cast<const XT*>(p.logits) + row * p.ldl;
  float m = -INFINITY;
  for (int64_t j = threadIdx.x; j < p.V; j += kThreads) m = fmaxf(m, widen(x[j]));
  m = block_reduce<float>(m, fbuf, op_max);
  float S = 0.f, W = 0.f;
  for (int64_t j = threadIdx.x; j < p.V; j += kThreads) {
    const float v = widen(x[j]);
    if (v == -INFINITY) continue;
    const float u = (v - m) * p.scale, e = expf(u);
    S += e;
    W += e > 0.f ? e * u : 0.f;
    if (u != u) S = u;
  }
  S = block_reduce<float>(S, fbuf, op_sum);
  W = block_reduce<float>(W, fbuf, op_sum);
  // Nothing left: no token has a probability.  A NaN, if any, makes S NaN.
  const bool none = S == 0.f;
  const float log_s = logf(S);
  if (p.entropy && threadIdx.x == 0) p.entropy[row] = none ? 0.f : log_s - W / S;
  for (int64_t j = threadIdx.x; j < p.T; j += kThreads) {
    const int64_t id = p.tokens[row * p.T + j];
    p.token_lp[row * p.T + j] = id < 0      ? 0.f
                                : id >= p.V ? NAN
                                : none      ? -INFINITY
                                            : (widen(x[id]) - m) * p.scale - log_s;
  }
  unsigned long long last = ~0ull;
  for (int i = 0; i < p.k; ++i) {
    unsigned long long best = 0;
    for (int64_t j = threadIdx.x; j < p.V; j += kThreads) {
      const unsigned long long key = order_key(widen(x[j]), (uint32_t)j);
      if (key < last && key > best) best = key;
    }
    last = best = block_reduce<unsigned long long>(best, kbuf, op_umax);
    if (threadIdx.x == 0) {
      const int64_t id = 0xFFFFFFFFu - (uint32_t)best;
      p.top_ids[row * p.k + i] = id;
      p.top_lp[row * p.k + i] = none ? -INFINITY : (widen(x[id]) - m) * p.scale - log_s;
    }
  }
}

template <typename XT>
int launch_type(const LogprobParams& p, int64_t M, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)M);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, logprobs_kernel<XT>, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  return PQ2_OK;
}

}  // namespace

int launch_token_logprobs(const void* logits, int dtype, int64_t ldl, int64_t M, int64_t V,
                          float scale, const int64_t* tokens, int64_t T, float* token_lp,
                          float* entropy, int k, int64_t* top_ids, float* top_lp, int sm_count,
                          cudaStream_t stream) {
  const LogprobParams p{logits, tokens, token_lp, entropy, top_ids, top_lp, ldl, V, T, scale, k};
  if (dtype == PQ2_BF16) return launch_type<__nv_bfloat16>(p, M, stream);
  if (dtype == PQ2_F16) return launch_type<__half>(p, M, stream);
  return launch_type<float>(p, M, stream);
}

}  // namespace pq2
