// pq2_norm.cu — the norms after a block and before the next one, fused with
// the block's gate and residual scale (pq2_norm_gate_residual):
//   p  = z / sqrt(mean z^2 + eps) * (w_post + o)   (or z without w_post)
//   h' = h + alpha * gate * p
//   n  = h' / sqrt(mean h'^2 + eps) * (w_pre + o)
// in fp32, each output rounded once.
//
// Bound by memory: z, h (and a gate per token) are read and h', n written once.
// A CTA takes a row and keeps it in registers between the two sums.  Several
// CTAs share an SM, so that some rows' loads are in flight while others wait
// for their sums.  (4096 rows of 5120 bf16, a gate per token: 36.4 us, 0.85 of
// the measured copy rate; persistent CTAs with the next two rows' copies in a
// shared-memory ring took 39.4 us, 160 instead of 320 threads a row 38.3 us.)
// The choices were made at that width.  Rows of more than 8192 16-bit elements
// (4096 32-bit ones) load the weights after the first sum, those of more than
// 16384 (8192) have an SM to themselves, and 64 registers do not hold them
// whole: 12 to 72 bytes a thread spill with four groups, 204 to 432 with eight
// (32-bit rows beyond 16384).  Rows, strides or pointers that are not multiples
// of 16 bytes use narrower accesses.  (500 rows of 20000 bf16 26.7 us, 0.55 of
// the copy rate; of 20000 fp32 64.4 us, 0.46; of 19999 bf16 70.9 us, 0.21; 4096
// rows of 5119 bf16 66.6 us, 0.46.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "pq2.h"
#include "pq2_device.cuh"
#include "pq2_internal.h"

namespace pq2 {
namespace {

// 16 bytes of a row: E elements in fp32 and back (rounded to nearest even).
template <typename T>
struct Pack;
template <>
struct Pack<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void widen(uint4 v, float* f) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 narrow(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};
template <>
struct Pack<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void widen(uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 narrow(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Pack<__half> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void widen(uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = p.x, f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint4 narrow(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// The block's sum of v, in a fixed order; `buf` holds a float per warp and is
// used once.
__device__ __forceinline__ float block_sum(float v, float* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  v = lane < (int)blockDim.x >> 5 ? buf[lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A thread's elements of a row: groups of E, each loaded as E / W pieces of W
// elements (16 bytes where rows, K and pointers are multiples of that, else
// the largest power of two that they are multiples of).  Piece c of group i is
// at ((i * E / W + c) * threads + tid) * W.
template <typename T, int W>
struct Slice {
  using P = Pack<T>;
  static constexpr int E = P::E, kPieces = E / W, kBytes = W * (int)sizeof(T);
  using Piece = typename std::conditional<
      kBytes == 16, uint4,
      typename std::conditional<kBytes == 8, uint2,
                                typename std::conditional<kBytes == 4, uint32_t, uint16_t>::type>::
          type>::type;
  // Where element e of group i is; a piece is in the row as a whole or not.
  static __device__ __forceinline__ int at(int i, int e) {
    return ((i * kPieces + e / W) * (int)blockDim.x + (int)threadIdx.x) * W + e % W;
  }
  // Group i; zeros beyond K.
  static __device__ __forceinline__ uint4 load(const T* row, int K, int i) {
    if constexpr (kBytes == 16) {
      return at(i, 0) < K ? *reinterpret_cast<const uint4*>(row + at(i, 0)) : make_uint4(0, 0, 0, 0);
    } else {
      uint32_t w[4] = {};
#pragma unroll
      for (int e = 0; e < E; e += W) {
        if constexpr (kBytes == 8) {
          const uint2 v = at(i, e) < K ? *reinterpret_cast<const uint2*>(row + at(i, e)) : make_uint2(0, 0);
          w[e * 4 / E] = v.x, w[e * 4 / E + 1] = v.y;
        } else {
          if (at(i, e) < K)
            w[e * 4 / E] |= (uint32_t) reinterpret_cast<const Piece*>(row)[at(i, e) / W]
                            << (8 * e * sizeof(T) % 32);
        }
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  static __device__ __forceinline__ void store(T* row, int K, int i, uint4 v) {
    if constexpr (kBytes == 16) {
      if (at(i, 0) < K) *reinterpret_cast<uint4*>(row + at(i, 0)) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < E; e += W) {
        if constexpr (kBytes == 8) {
          if (at(i, e) < K)
            *reinterpret_cast<uint2*>(row + at(i, e)) = make_uint2(w[e * 4 / E], w[e * 4 / E + 1]);
        } else {
          if (at(i, e) < K)
            reinterpret_cast<Piece*>(row)[at(i, e) / W] =
                (Piece)(w[e * 4 / E] >> (8 * e * sizeof(T) % 32));
        }
      }
    }
  }
};

// Threads of a CTA, at most: small CTAs, so that several rows share an SM.
constexpr int threads_of(int v) { return v > 2 ? 1024 : v == 1 ? 256 : 512; }

// A thread's groups of a row, and of the weights.
template <int V>
struct Row {
  uint4 z[V], h[V], gate[V];
};
template <int V>
struct Weights {
  uint4 post[V], pre[V];
};

// One row in registers.  EARLY: the weights are in registers too, else they
// are loaded group by group.
template <typename T, int V, int W, bool EARLY>
__device__ __forceinline__ void do_row(const NormParams& p, int64_t row, const Row<V>& in,
                                       const Weights<V>& w, float (*buf)[32]) {
  using S = Slice<T, W>;
  using P = Pack<T>;
  constexpr int E = P::E;
  const int K = (int)p.K;
  float inv = 1.f;
  if (p.w_post) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float z[E];
      P::widen(in.z[i], z);
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(z[e], z[e], s);
    }
    inv = rsqrtf(fmaf(block_sum(s, buf[0]), p.one_over_k, p.eps));
  }
  float v[V][E], s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    P::widen(in.h[i], v[i]);
    if (p.z) {
      float q[E], f[E];
      P::widen(in.z[i], q);
      if (p.w_post) {
        P::widen(EARLY ? w.post[i] : S::load(static_cast<const T*>(p.w_post), K, i), f);
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = q[e] * inv * (f[e] + p.w_offset);
      }
      if (p.gate) {
        P::widen(in.gate[i], f);
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] *= f[e];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = fmaf(p.alpha, q[e], v[i][e]);
    }
    if (p.h_out) S::store(static_cast<T*>(p.h_out) + row * p.K, K, i, P::narrow(v[i]));
    // Places beyond K hold zeros, or what alpha makes of them.
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (S::at(i, e / W * W) < K) s = fmaf(v[i][e], v[i][e], s);
  }
  if (!p.n_out) return;
  inv = rsqrtf(fmaf(block_sum(s, buf[1]), p.one_over_k, p.eps));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f[E];
    P::widen(EARLY ? w.pre[i] : S::load(static_cast<const T*>(p.w_pre), K, i), f);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = v[i][e] * inv * (f[e] + p.w_offset);
    S::store(static_cast<T*>(p.n_out) + row * p.K, K, i, P::narrow(f));
  }
}

template <typename T>
__device__ __forceinline__ const T* gate_row(const NormParams& p, int64_t row) {
  const uint32_t r = p.rows_per_gate == 1 ? (uint32_t)row : (uint32_t)row / p.rows_per_gate;
  return static_cast<const T*>(p.gate) + r * p.ldg;
}

// A row a CTA.
template <typename T, int V, int W>
__global__ void __launch_bounds__(threads_of(V), 1024 / threads_of(V)) norm_kernel(const NormParams p) {
  using S = Slice<T, W>;
  constexpr bool kEarly = W == S::E && V <= 2;
  __shared__ float buf[2][32];
  const int K = (int)p.K;
  const int64_t row = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Row<V> in;
  Weights<V> w;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    in.h[i] = S::load(static_cast<const T*>(p.h) + row * p.ldh, K, i);
    if (p.z) in.z[i] = S::load(static_cast<const T*>(p.z) + row * p.ldz, K, i);
    if (p.gate) in.gate[i] = S::load(gate_row<T>(p, row), K, i);
    if (kEarly && p.w_post) w.post[i] = S::load(static_cast<const T*>(p.w_post), K, i);
    if (kEarly && p.n_out) w.pre[i] = S::load(static_cast<const T*>(p.w_pre), K, i);
  }
  do_row<T, V, W, kEarly>(p, row, in, w, buf);
}

template <typename T, int V, int W>
int launch_one(const NormParams& p, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.M);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, norm_kernel<T, V, W>, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  return PQ2_OK;
}

template <typename T, int W>
int launch_slices(const NormParams& p, cudaStream_t stream) {
  // Groups of 16 bytes a thread; eight are for fp32 rows beyond 16384 columns
  // alone.
  constexpr int E = 16 / sizeof(T);
  const int groups = (int)((p.K + E - 1) / E);
  const auto threads = [&](int v) { return ((groups + v - 1) / v + 31) / 32 * 32; };
  if (threads(1) <= threads_of(1)) return launch_one<T, 1, W>(p, threads(1), stream);
  if (threads(2) <= threads_of(2)) return launch_one<T, 2, W>(p, threads(2), stream);
  if (sizeof(T) == 2 || threads(4) <= threads_of(4))
    return launch_one<T, 4, W>(p, threads(4), stream);
  return launch_one<T, sizeof(T) == 4 ? 8 : 4, W>(p, threads(8), stream);
}

template <typename T>
int launch_type(const NormParams& p, cudaStream_t stream) {
  // The lowest bit set in any address or row length, in bytes.
  uint64_t bits = 16;
  for (const void* q : {p.z, p.h, p.gate, p.w_post, p.w_pre, (const void*)p.h_out, (const void*)p.n_out})
    bits |= reinterpret_cast<uintptr_t>(q);
  bits |= (uint64_t)(p.K | p.ldh | (p.z ? p.ldz : 0) | (p.gate ? p.ldg : 0)) * sizeof(T);
  switch (bits & -bits) {
    case 16: return launch_slices<T, 16 / sizeof(T)>(p, stream);
    case 8: return launch_slices<T, 8 / sizeof(T)>(p, stream);
    case 4: return launch_slices<T, 4 / sizeof(T)>(p, stream);
    default: return launch_slices<T, 1>(p, stream);
  }
}

}  // namespace

int launch_norm(const NormParams& p, int dtype, cudaStream_t stream) {
  if (dtype == PQ2_BF16) return launch_type<__nv_bfloat16>(p, stream);
  if (dtype == PQ2_F16) return launch_type<__half>(p, stream);
  return launch_type<float>(p, stream);
}

}  // namespace pq2
