// pq2_logprobs.cu — log-probabilities of given tokens, entropy and top
// alternatives of each row of logits (pq2_token_logprobs), in one pass.
//
// With t = scale * x, a reference r near the row's maximum, u = t - scale r,
// S = sum exp(u) and W = sum exp(u) u:
//   log p_j = u_j - log S,    H = -sum p log p = log S - W / S,
// kept in base 2 (u2 = u / ln 2) for the exponential instruction.  A thread's
// reference moves only when an element exceeds it by more than 2^8 in p (the
// published lazy form of a running maximum): S' = a S, W' = a (W + d S) with d =
// u2 of the old reference, a = 2^d.  The exponential is the approximate
// instruction (2^-22 of a term) and u2 carries three roundings (2^-23 |u2|), as
// more would make the pass, bound by its instructions, longer.
// Logits of -inf have u2 clamped to -200, where 2^u2 is 0, so they add 0 to
// both sums; a NaN stays a NaN.
//
// Top alternatives: the pass keeps each thread's two largest vector maxima and
// where the larger was.  With n threads known to hold an element of some key
// (value, then lower index) or better, the n-th key of the row is at least
// that; so a few of the warps' best threads give a limit, and only the threads
// whose best reaches it (about 2 k of them) read that vector once more, or all
// of theirs if the second reaches it too.  What reaches the limit there is
// sorted.  (2048 rows of 131072 bf16: 83 us without alternatives, 92 us with
// one, 99 us with 20; 0.96 .. 0.80 of the measured copy rate.  Lists kept during
// the pass cost 122 us.)  Logits of -inf stay out of this: a row with fewer than k others
// takes its first ones at the end (one warp, in order: a row of NaN alone is
// walked twice, 32 rows of 131072 in 1.04 ms).
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

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnroll = 4;       // 16-byte vectors a thread holds
constexpr int kMaxCluster = 16;
constexpr int kFlush = 32;       // pending keys that are merged
constexpr float kLn2 = 0.693147180559945309f;

struct LogprobParams {
  const void* logits;
  const int64_t* tokens;
  float* token_lp;
  float* entropy;
  int64_t* top_ids;
  float* top_lp;
  int64_t ldl, V, T;
  float scale;
  int k, split;
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

// The order of the alternatives as a whole number: by value (-0 = +0, NaN
// below -inf); 0 is below every element.
__device__ __forceinline__ uint32_t order_of(float v) {
  v += 0.f;
  const uint32_t b = __float_as_uint(v);
  return v != v ? 1u : (b >> 31 ? ~b : b | 0x80000000u);
}
constexpr uint32_t kOrderOfMinusInf = 0x007FFFFFu;
__device__ __forceinline__ float value_of(uint32_t order) {
  return order <= 1u ? -INFINITY
                     : __uint_as_float(order >> 31 ? order & 0x7FFFFFFFu : ~order);
}
// Value, then the lower index.
__device__ __forceinline__ uint64_t key_of(uint32_t order, uint32_t index) {
  return (uint64_t)order << 32 | (0xFFFFFFFFu - index);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// A 16-byte vector of logits: its elements in fp32 and its maximum (NaN
// ignored).
template <typename XT>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kElems = 4;
  static __device__ __forceinline__ void widen(uint4 v, float* f) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float most(uint4 v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                 fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static constexpr uint32_t kNone = 0xFF800000u;  // -inf in every element
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kElems = 8;
  static __device__ __forceinline__ void widen(uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ float most(uint4 v) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__bfloat162float(m.x), __bfloat162float(m.y));
  }
  static constexpr uint32_t kNone = 0xFF80FF80u;
};
template <>
struct Vec<__half> {
  static constexpr int kElems = 8;
  static __device__ __forceinline__ void widen(uint4 v, float* f) {
    const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(h[i]);
      f[2 * i] = p.x, f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ float most(uint4 v) {
    const __half2* h = reinterpret_cast<const __half2*>(&v);
    const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__half2float(m.x), __half2float(m.y));
  }
  static constexpr uint32_t kNone = 0xFC00FC00u;
};

// Two fp32 values in one register pair, for the two-wide operations.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Sums over some elements, relative to `ref`.
struct Sums {
  float ref, S, W;
  // To another reference.
  __device__ __forceinline__ void move(float to, float c2) {
    const float d = fmaxf((ref - to) * c2, -200.f), a = ex2(d);
    W = a * fmaf(d, S, W);
    S *= a;
    ref = to;
  }
  // The sum over the warp's lanes (over groups of N lanes).
  template <int N>
  __device__ __forceinline__ void join(float c2) {
    float r = ref;
#pragma unroll
    for (int o = N / 2; o; o >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
    move(r, c2);
#pragma unroll
    for (int o = N / 2; o; o >>= 1) {
      S += __shfl_xor_sync(0xffffffffu, S, o);
      W += __shfl_xor_sync(0xffffffffu, W, o);
    }
  }
};

// One thread's sums, in two halves.
struct Running {
  float ref;
  uint64_t S, W;
  // Move the reference up to `most` if that exceeds it by more than `slack`.
  __device__ __forceinline__ void refer(float most, float slack, float c2) {
    if (most > ref + slack) {
      const float d = fmaxf((ref - most) * c2, -200.f), a = ex2(d);
      W = mul2(pair(a, a), fma2(pair(d, d), S, W));
      S = mul2(pair(a, a), S);
      ref = most;
    }
  }
  __device__ __forceinline__ void add(float x0, float x1, float c2) {
    const float2 v = unpair(mul2(add2(pair(x0, x1), pair(-ref, -ref)), pair(c2, c2)));
    const float u0 = max_nan(v.x, -200.f), u1 = max_nan(v.y, -200.f);
    const uint64_t e = pair(ex2(u0), ex2(u1));
    S = add2(S, e);
    W = fma2(e, pair(u0, u1), W);
  }
  __device__ __forceinline__ Sums sum() const {
    const float2 s = unpair(S), w = unpair(W);
    return {ref, s.x + s.y, w.x + w.y};
  }
};

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t min64(uint64_t a, uint64_t b) { return a < b ? a : b; }

// A bitonic sequence over the lanes, sorted descending.
__device__ __forceinline__ uint64_t sort_bitonic(uint64_t v, int lane) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
    v = lane & o ? min64(v, w) : max64(v, w);
  }
  return v;
}
// Any sequence over the lanes, sorted descending.  (Functions of their own, as
// each runs a few times at most: a kernel that starts cold pays for the code it
// fetches.)
__device__ __noinline__ uint64_t sort_any(uint64_t v, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
    for (int o = n >> 1; o; o >>= 1) {
      const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
      v = ((lane & o) != 0) != ((lane & n) != 0) ? min64(v, w) : max64(v, w);
    }
  return v;
}
// The 32 best of two descending sequences, descending.
__device__ __noinline__ uint64_t merge_sorted(uint64_t a, uint64_t b, int lane) {
  return sort_bitonic(max64(a, __shfl_sync(0xffffffffu, b, 31 - lane)), lane);
}

// A warp's best keys.
struct Best {
  uint64_t list;  // this lane's key, descending over the lanes
  uint64_t last;  // the k-th key: what a new one has to exceed
  int pending;    // keys in the buffer
};
struct Keys {
  uint64_t list, last;
};

struct Shared {
  uint64_t buffer[kWarps][64];
  uint64_t lists[kMaxCluster][32];
  uint64_t few[kWarps * 32];  // keys that no list holds yet
  uint64_t mine[32];          // this CTA's list, for the cluster
  Sums sums[kWarps];
  Sums total;
  uint64_t posted[kWarps];  // the key of each warp's quota-th thread
  int pending[kWarps];      // keys not in the list yet, or -1 if it is in use
};

// The first 32 of the warp's pending keys into its list.
__device__ __noinline__ Keys flush_keys(uint64_t list, int pending, int k, uint64_t* buffer) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  const uint64_t v = lane < pending ? buffer[lane] : 0;
  const uint64_t more = lane + 32 < pending ? buffer[lane + 32] : 0;
  __syncwarp();
  if (lane + 32 < pending) buffer[lane] = more;
  Keys r;
  r.list = merge_sorted(list, sort_any(v, lane), lane);
  r.last = __shfl_sync(0xffffffffu, r.list, k - 1);
  __syncwarp();
  return r;
}
__device__ __forceinline__ void flush(Best& b, int k, Shared& s, int warp) {
  const Keys r = flush_keys(b.list, b.pending, k, s.buffer[warp]);
  b.list = r.list, b.last = r.last;
  b.pending = max(b.pending - 32, 0);
}
// Offers one key per lane (0: none).
__device__ __forceinline__ void offer(Best& b, uint64_t key, int k, Shared& s, int warp, int lane) {
  const bool take = key > b.last;
  const uint32_t who = __ballot_sync(0xffffffffu, take);
  if (!who) return;
  if (take) s.buffer[warp][b.pending + __popc(who & ((1u << lane) - 1))] = key;
  b.pending += __popc(who);
  if (b.pending >= kFlush) flush(b, k, s, warp);
}
// The quota-th largest of the lanes' keys (0 if there are fewer), quota =
// k / kWarps rounded up.
__device__ __forceinline__ uint64_t quota_th(uint64_t key, int k) {
  uint64_t found = 0;
#pragma unroll 1
  for (int q = 0; q < k; q += kWarps) {
    const uint32_t high = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32));
    const uint32_t low =
        __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32) == high ? (uint32_t)key : 0);
    found = (uint64_t)high << 32 | low;
    if (key == found) key = 0;
  }
  return found;
}
// The largest key that n quotas making k are known to reach, by the keys the
// warps posted: the n-th largest of them.
__device__ __forceinline__ uint64_t limit_of(int k, const uint64_t* posted) {
  const int lane = threadIdx.x & 31, quota = (k + kWarps - 1) / kWarps;
  const uint64_t mine = posted[lane % kWarps];
  int above = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const uint64_t other = posted[w];
    above += other > mine || (other == mine && w < lane % kWarps);
  }
  const uint32_t who = __ballot_sync(0xffffffffu, above == (k + quota - 1) / quota - 1);
  return __shfl_sync(0xffffffffu, mine, __ffs(who) - 1);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
template <typename T>
__device__ __forceinline__ T remote(const T* p, int rank) {
  T v;
  if constexpr (sizeof(T) == 8)
    asm volatile(
        "{\n\t.reg .u32 at;\n\tmapa.shared::cluster.u32 at, %1, %2;\n\t"
        "ld.shared::cluster.b64 %0, [at];\n\t}"
        : "=l"(v)
        : "r"(smem_u32(p)), "r"(rank)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .u32 at;\n\tmapa.shared::cluster.u32 at, %1, %2;\n\t"
        "ld.shared::cluster.f32 %0, [at];\n\t}"
        : "=f"(v)
        : "r"(smem_u32(p)), "r"(rank)
        : "memory");
  return v;
}

// Merges `count` lists in s.lists pairwise until one is left; every thread of
// the block calls it.
__device__ __forceinline__ void merge_lists(Shared& s, int count, int warp, int lane) {
  while (count > 1) {
    const int half = (count + 1) / 2;
    for (int i = warp; i + half < count; i += kWarps)
      s.lists[i][lane] = merge_sorted(s.lists[i][lane], s.lists[i + half][lane], lane);
    count = half;
    __syncthreads();
  }
}

// Fills a list of n < k keys up to k with the row's first logits of -inf, then
// NaN; one warp.
template <typename XT>
__device__ __noinline__ void fill_list(const XT* x, int64_t V, int n, int k, uint64_t* list) {
  const int lane = threadIdx.x & 31;
  for (int nan = 0; nan < 2; ++nan)
    for (int64_t base = 0; base < V && n < k; base += 32) {
      const float v = base + lane < V ? widen(x[base + lane]) : 0.f;
      const bool take = nan ? v != v : v == -INFINITY;
      const uint32_t who = __ballot_sync(0xffffffffu, take);
      const int at = n + __popc(who & ((1u << lane) - 1));
      if (take && at < k) list[at] = key_of(nan ? 1u : kOrderOfMinusInf, (uint32_t)(base + lane));
      n += __popc(who);
    }
  __syncwarp();
}

template <typename XT, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LogprobParams p) {
  constexpr int E = Vec<XT>::kElems;
  __shared__ Shared s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % p.split;
  const int64_t row = blockIdx.x / p.split;
  const XT* x = static_cast<const XT*>(p.logits) + row * p.ldl;
  const float c2 = p.scale * 1.44269504088896341f, slack = 8.f / c2;

  // The row as a few elements up to a 16-byte boundary, vectors, a few
  // elements after them; the vectors are shared among the CTAs of the cluster.
  const int64_t head = min((int64_t)(16 - reinterpret_cast<uintptr_t>(x) % 16) % 16 / (int)sizeof(XT), p.V);
  const int64_t vectors = (p.V - head) / E, body_end = head + vectors * E;
  const int64_t v0 = vectors * rank / p.split, v1 = vectors * (rank + 1) / p.split;
  const uint4* body = reinterpret_cast<const uint4*>(x + head);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // The row's first vectors are on their way before anything is waited for.
  uint4 next[kUnroll];
  auto load = [&](int64_t base) {
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int64_t v = base + j * kThreads + tid;
      next[j] = v < v1 ? body[v]
                       : make_uint4(Vec<XT>::kNone, Vec<XT>::kNone, Vec<XT>::kNone, Vec<XT>::kNone);
    }
  };
  load(v0);

  Running sums{-3.402823466e38f, 0, 0};
  Best best{};

  // The first tokens' logits, while the row streams.
  int64_t token = -1;
  float token_x = 0.f;
  if (rank == 0 && tid < p.T) {
    token = p.tokens[row * p.T + tid];
    if (token >= 0 && token < p.V) token_x = widen(x[token]);
  }

  // The elements outside the vectors, one per lane of the first warp.
  const int64_t single = warp                              ? -1
                         : rank == 0 && lane < head        ? lane
                         : rank == p.split - 1 && lane >= 16 && body_end + lane - 16 < p.V
                             ? body_end + lane - 16
                             : -1;
  float single_x = -INFINITY;
  if (warp == 0) {
    if (single >= 0) single_x = widen(x[single]);
    sums.refer(single_x, slack, c2);
    sums.add(single_x, -INFINITY, c2);
  }

  float high = -INFINITY, second = -INFINITY;  // largest vector maxima
  int where = 0, at = 0;                       // the vector of `high`
  for (int64_t base = v0; base < v1; base += kUnroll * kThreads) {
    uint4 cur[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) cur[j] = next[j];
    load(base + kUnroll * kThreads);
    float most[kUnroll], top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      most[j] = Vec<XT>::most(cur[j]);
      top = fmaxf(top, most[j]);
      if (TOP) {
        if (most[j] > high) where = at + j;
        second = fmaxf(second, fminf(high, most[j]));
        high = fmaxf(high, most[j]);
      }
    }
    at += kUnroll;
    sums.refer(top, slack, c2);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      float f[E];
      Vec<XT>::widen(cur[j], f);
#pragma unroll
      for (int e = 0; e < E; e += 2) sums.add(f[e], f[e + 1], c2);
    }
  }

  // The CTA's sums and list.
  Sums part = sums.sum();
  const bool clean = part.S == part.S;
  part.join<32>(c2);
  if (lane == 0) s.sums[warp] = part;
  if (TOP) {
    // This thread's best: its order and the indexes it may have (0: nothing
    // above -inf, or unknown, where a NaN or +inf may hide among its elements).
    const int count = v0 + tid < v1 ? (int)((v1 - v0 - tid + kThreads - 1) / kThreads) : 0;
    const int64_t best_v = v0 + tid + (int64_t)where * kThreads, first = head + best_v * E;
    const uint32_t order = clean && count && high > -INFINITY ? order_of(high) : 0;
    const uint64_t q = quota_th(order ? key_of(order, (uint32_t)(first + E - 1)) : 0, p.k);
    if (lane == 0) s.posted[warp] = q;
    __syncthreads();
    const uint64_t limit = max64(limit_of(p.k, s.posted), (uint64_t)(kOrderOfMinusInf + 1) << 32);
    if (warp == 0) {
      const uint64_t key = single >= 0 ? key_of(order_of(single_x), (uint32_t)single) : 0;
      offer(best, key >= limit ? key : 0, p.k, s, warp, lane);
    }
    // Each lane's vector v, if `in`.
    const float least = value_of((uint32_t)(limit >> 32));
    auto look = [&](int64_t v, bool in) {
      const uint4 c = in ? body[v] : make_uint4(0, 0, 0, 0);
      float f[E];
      Vec<XT>::widen(c, f);
      uint32_t any = 0;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (!(f[e] < least)) any |= 1u << e;
      if (!in) any = 0;
#pragma unroll 1
      while (__any_sync(0xffffffffu, any)) {
        uint64_t key = 0;
        if (any) {
          const int64_t i = head + v * E + __ffs(any) - 1;
          any &= any - 1;
          key = key_of(order_of(widen(x[i])), (uint32_t)i);
        }
        offer(best, key >= limit ? key : 0, p.k, s, warp, lane);
      }
    };
    const bool hit = count && (!clean || (order && key_of(order, (uint32_t)first) >= limit));
    // The first place where a vector other than the best can be.
    const int64_t other = head + (v0 + tid + (where ? 0 : kThreads)) * E;
    const bool whole =
        hit && (!clean || key_of(order_of(second), (uint32_t)other) >= limit);
    // First the lanes that need one vector, then one whole thread after
    // another, 32 vectors at a time.
    uint32_t rest = __ballot_sync(0xffffffffu, whole);
    int64_t v = best_v;
    bool in = hit && !whole;
    int n = 0, i = 0, who = 0;
#pragma unroll 1
    for (;;) {
      if (__any_sync(0xffffffffu, in)) look(v, in);
      i += 32;
      if (i >= n) {
        if (!rest) break;
        who = __ffs(rest) - 1;
        rest &= rest - 1;
        n = __shfl_sync(0xffffffffu, count, who);
        i = 0;
      }
      v = v0 + warp * 32 + who + (int64_t)(i + lane) * kThreads;
      in = i + lane < n;
    }
    const bool used = __any_sync(0xffffffffu, best.list != 0);
    while (best.pending > 32 || (best.pending && used)) flush(best, p.k, s, warp);
    if (lane == 0) s.pending[warp] = used ? -1 : best.pending;
    s.lists[warp][lane] = best.list;
  }
  __syncthreads();
  Sums total = s.sums[lane % kWarps];
  total.join<kWarps>(c2);
  if (TOP) {
    // The keys that no list holds yet, 32 to a list; or, where a warp had more
    // of them, every warp's list.
    int n = 0, from = 0;
    bool few = true;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int c = s.pending[w];
      few = few && c >= 0;
      n += max(c, 0);
      if (w < warp) from = n;
    }
    if (few) {
      if (lane < best.pending) s.few[from + lane] = s.buffer[warp][lane];
      __syncthreads();
      if (warp * 32 < n || warp == 0)
        s.lists[warp][lane] = sort_any(tid < n ? s.few[tid] : 0, lane);
    } else if (best.pending) {
      flush(best, p.k, s, warp);
      s.lists[warp][lane] = best.list;
    }
    __syncthreads();
    merge_lists(s, few ? (n + 31) / 32 : kWarps, warp, lane);
  }

  if (p.split > 1) {
    if (tid == 0) s.total = total;
    if (TOP && tid < 32) s.mine[tid] = s.lists[0][tid];
    cluster_sync();
    if (rank == 0) {
      const int r = lane % p.split;  // a power of two, at most 16
      total.ref = remote(&s.total.ref, r);
      total.S = remote(&s.total.S, r);
      total.W = remote(&s.total.W, r);
      if (lane >= p.split) total.S = total.W = 0.f;
      total.join<32>(c2);
      if (TOP) {
        for (int i = tid; i < p.split * 32; i += kThreads)
          s.lists[i >> 5][i & 31] = remote(&s.mine[i & 31], i >> 5);
        __syncthreads();
        merge_lists(s, p.split, warp, lane);
      }
    }
    cluster_sync();
    if (rank) return;
  }

  // A NaN makes S NaN; S = 0 is a row with nothing left.
  const bool none = total.S == 0.f;
  const float log_s = logf(total.S);
  auto logprob = [&](float v) {
    return none ? -INFINITY : fmaf(v - total.ref, p.scale, -log_s);
  };
  if (p.entropy && tid == 0)
    p.entropy[row] = none ? 0.f : fmaf(total.W / total.S, -kLn2, log_s);
  for (int64_t j = tid; j < p.T; j += kThreads) {
    if (j >= kThreads) {
      token = p.tokens[row * p.T + j];
      if (token >= 0 && token < p.V) token_x = widen(x[token]);
    }
    p.token_lp[row * p.T + j] = token < 0 ? 0.f : token >= p.V ? NAN : logprob(token_x);
  }
  if (TOP && warp == 0) {
    const int n = __popc(__ballot_sync(0xffffffffu, s.lists[0][lane] != 0));
    if (n < p.k) fill_list(x, p.V, n, p.k, s.lists[0]);
  }
  if (TOP && tid < p.k) {
    const uint64_t key = s.lists[0][tid];
    p.top_ids[row * p.k + tid] = 0xFFFFFFFFu - (uint32_t)key;
    p.top_lp[row * p.k + tid] = logprob(value_of((uint32_t)(key >> 32)));
  }
}

template <typename XT, bool TOP>
int launch_one(LogprobParams p, int64_t M, int sms, cudaStream_t stream) {
  auto kern = logprobs_kernel<XT, TOP>;
  // CTAs a row: enough to give every SM one, of at least 2048 elements each;
  // two where that gives every SM two.  (32 rows of 131072: 10.3 us in 256 CTAs,
  // 14.6 us in 512; 300 rows of 100003: 21 us in 300 CTAs, 20 us in 600.)
  p.split = 1;
  while (p.split < kMaxCluster && M * p.split < (p.split == 1 ? 2 : 1) * sms &&
         p.V / (2 * p.split) >= 2048)
    p.split *= 2;
  if (M * p.split > 0x7FFFFFFF) return PQ2_ERR_SHAPE;
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PQ2_ERR_CUDA;
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
        cudaSuccess) {
      cudaGetLastError();
      return PQ2_ERR_CUDA;
    }
    ready.fetch_or((uint64_t)1 << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(M * p.split));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    cudaGetLastError();
    return PQ2_ERR_LAUNCH;
  }
  return PQ2_OK;
}

template <typename XT>
int launch_type(const LogprobParams& p, int64_t M, int sms, cudaStream_t stream) {
  return p.k ? launch_one<XT, true>(p, M, sms, stream) : launch_one<XT, false>(p, M, sms, stream);
}

}  // namespace

int launch_token_logprobs(const void* logits, int dtype, int64_t ldl, int64_t M, int64_t V,
                          float scale, const int64_t* tokens, int64_t T, float* token_lp,
                          float* entropy, int k, int64_t* top_ids, float* top_lp, int sm_count,
                          cudaStream_t stream) {
  const LogprobParams p{logits, tokens, token_lp, entropy, top_ids, top_lp,
                        ldl,    V,      T,        scale,   k,       1};
  if (dtype == PQ2_BF16) return launch_type<__nv_bfloat16>(p, M, sm_count, stream);
  if (dtype == PQ2_F16) return launch_type<__half>(p, M, sm_count, stream);
  return launch_type<float>(p, M, sm_count, stream);
}

}  // namespace pq2
