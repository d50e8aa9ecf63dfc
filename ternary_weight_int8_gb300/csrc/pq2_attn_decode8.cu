// pq2_attn_decode8.cu — the kernels of pq2_attn_decode.cuh over 8-bit caches.
#include "pq2_attn_decode.cuh"

namespace pq2 {

int launch_attn_decode8(AttnDecode& p, int sm_count, cudaStream_t stream) {
  return p.a.dtype == PQ2_BF16 ? launch_dim<__nv_bfloat16, int8_t>(p, sm_count, stream)
                               : launch_dim<__half, int8_t>(p, sm_count, stream);
}

}  // namespace pq2
