// pq2_attn_decode.cu — attention of the newest tokens over a paged cache
// (pq2_attn_decode.cuh): workspace, choice of the kernel, and the kernels over
// 16-bit caches (pq2_attn_decode8.cu has those over 8-bit ones; two units only
// for the time that they take to compile).
#include "pq2_attn_decode.cuh"

namespace pq2 {
namespace {

// Rows of a CTA, as launch_rows chooses them.
int group_rows(int64_t rows, int64_t dim) {
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 24 && dim == 256 ? 24 : 32;
}
// How many CTAs take an item together, in a cluster that joins its parts through
// distributed shared memory, or one alone; 0: even shares of all SMs, which need a
// workspace and a second kernel.  The table bounds the lengths.  An SM begins in
// 4 us and reads at 45 GB/s when all do; 14 clusters of 8, 32 of 4, 72 of 2 or 152
// CTAs run at once (16 of 8 took two rounds: 13.4 us against 7.4 for 15).  Even
// shares read at 6.7 TB/s, half of the table as lengths differ, begin in 8 us, and
// their second launch and workspace take the host 6 us more.  Heads of 128, bf16,
// full tables, replayed (called in a loop): 1 x 512 tokens, 8 key heads 6.6 (11.3) us in
// clusters of 8 against 8.3 (16) in even shares; 4 x 1024 6.9 (11.1) in clusters of
// 4 against 9.8 (16); 8 x 1500 9.9 (11.1) in clusters of 2 against 11.3 (16); 16 x 700
// 8.6 (11.1) alone against 12.5 (16); 1 x 8192 11.0 (12.0) against 10.3 (16).
int cluster_of(int64_t B, int64_t rows, int64_t heads, int64_t dim, int64_t positions) {
  const int n = group_rows(rows, dim);
  const int64_t items = B * heads * ((rows + n - 1) / n);
  const double bytes = (double)positions * (double)dim * 4;  // of an item, 16 bits
  double least = (double)items * bytes / 2 / 6.7e6 + 14;
  int best = 0, at_once[4] = {152, 72, 32, 14};
  for (int i = 0; i < 4; ++i) {
    const double us = (double)((items + at_once[i] - 1) / at_once[i]) * (4 + bytes / (1 << i) / 45e3);
    if (us < least) least = us, best = 1 << i;
  }
  return best;
}
static_assert(kCluster == 8, "cluster_of");

}  // namespace

size_t attn_decode_workspace_bytes(int64_t B, int64_t T, int64_t q_heads, int64_t heads,
                                   int64_t dim, int64_t positions) {
  const int64_t rows = T * (q_heads / heads);
  if (cluster_of(B, rows, heads, dim, positions)) return 0;
  return kMaxCtas * sizeof(int4) + (size_t)2 * kMaxCtas * group_rows(rows, dim) * (dim + 3) * sizeof(float);
}

int launch_attn_decode(const DecodeParams& a, const pq2_kv_cache& c, int sm_count,
                       cudaStream_t stream) {
  AttnDecode p{};
  p.a = a, p.cache = c;
  p.group = a.q_heads / (int)c.heads;
  p.rows = a.T * p.group;
  p.c = a.scale * kLog2e;
  p.cluster = cluster_of(a.batch.B, p.rows, c.heads, c.dim, a.batch.table_width * c.page_size);
  if ((int64_t)p.cluster * a.batch.B * c.heads * ((p.rows + 7) / 8) > 0x7fffffff) return PQ2_ERR_SHAPE;
  if (c.dtype == PQ2_I8) return launch_attn_decode8(p, sm_count, stream);
  if (a.dtype == PQ2_BF16)
    return launch_dim<__nv_bfloat16, __nv_bfloat16>(p, sm_count, stream);
  return launch_dim<__half, __half>(p, sm_count, stream);
}

}  // namespace pq2
