// pq2_attn_decode.cu — attention of the newest tokens over a paged cache
// (pq2_attn_decode.cuh): workspace, choice of the kernel, and the kernels over
// 16-bit caches (pq2_attn_decode8.cu has those over 8-bit ones; two units only
// for the time that they take to compile).
#include "pq2_attn_decode.cuh"

namespace pq2 {
namespace {

// Rows of a CTA, as launch_rows chooses them.
int group_rows(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }
bool in_clusters(int64_t B, int64_t rows, int64_t heads, int64_t positions) {
  const int n = group_rows(rows);
  return B * heads * ((rows + n - 1) / n) <= kClusterItems && positions <= kClusterPositions;
}

}  // namespace

size_t attn_decode_workspace_bytes(int64_t B, int64_t T, int64_t q_heads, int64_t heads,
                                   int64_t dim, int64_t positions) {
  const int64_t rows = T * (q_heads / heads);
  if (in_clusters(B, rows, heads, positions)) return 0;
  return kMaxCtas * sizeof(int4) + (size_t)2 * kMaxCtas * group_rows(rows) * (dim + 3) * sizeof(float);
}

int launch_attn_decode(const DecodeParams& a, const pq2_kv_cache& c, int sm_count,
                       cudaStream_t stream) {
  AttnDecode p{};
  p.a = a, p.cache = c;
  p.group = a.q_heads / (int)c.heads;
  p.rows = a.T * p.group;
  p.c = a.scale * kLog2e;
  p.cluster = in_clusters(a.batch.B, p.rows, c.heads, a.batch.table_width * c.page_size);
  if (c.dtype == PQ2_I8) return launch_attn_decode8(p, sm_count, stream);
  if (a.dtype == PQ2_BF16)
    return launch_dim<__nv_bfloat16, __nv_bfloat16>(p, sm_count, stream);
  return launch_dim<__half, __half>(p, sm_count, stream);
}

}  // namespace pq2
