"""The flags of pq2_w4_mmv on both kernels, with and without a split of K over
a cluster, and in calls of several launches: the bits are those of a call that
waits for everything before it, and a buffer that the call before still reads
is written only after it."""
import pytest
import torch

from ternary_weight_int8_gb300 import pq2

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pq2.lib()
    yield
    torch.cuda.synchronize()


def plane(N, K, G, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand((N, K // G), generator=g, device="cuda") * 0.002 + 0.001).half()
    return pq2.pq2_w4_prepare(codes, scales, group=G)


# M = 3 is the narrow kernel, 24 the wide one (or, with 32-bit x or K = 17408,
# several launches); K = 2048 has no split, 5120 and 17408 one of five.
@pytest.mark.parametrize("M", [3, 24])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,K", [(2048, 2048), (5120, 5120), (5120, 17408)])
def test_flags(M, dtype, N, K):
    G, rows = 64, 30000
    reader, writer = plane(rows, N, G, seed=1), plane(N, K, G, seed=2)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn((M, K), generator=g, device="cuda").to(dtype)
    before = torch.randn((M, N), generator=g, device="cuda").to(dtype)
    want_read = pq2.pq2_w4_mmv(before, reader, rows, G)
    want = pq2.pq2_w4_mmv(x, writer, N, G, out_dtype=dtype)
    torch.cuda.synchronize()
    want_after = pq2.pq2_w4_mmv(want, reader, rows, G)
    torch.cuda.synchronize()
    buf, read = torch.empty_like(before), torch.empty_like(want_read)
    after = torch.empty_like(want_read)

    def chain():
        buf.copy_(before)
        # reads buf, which the flagged call then writes, and the last one reads
        pq2.pq2_w4_mmv(buf, reader, rows, G, y=read)
        pq2.pq2_w4_mmv(x, writer, N, G, y=buf, flags=pq2.PQ2_MMV_INDEPENDENT)
        pq2.pq2_w4_mmv(buf, reader, rows, G, y=after, flags=pq2.PQ2_MMV_OVERLAP_WEIGHTS)

    def check():
        torch.cuda.synchronize()
        assert torch.equal(read, want_read) and torch.equal(buf, want)
        assert torch.equal(after, want_after)

    for _ in range(3):
        chain()
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(3):
        graph.replay()
        check()
