"""Calls with ``stream``: a block that the current stream has let go of, with work
on it still queued there, does not become the call's workspace or output."""
import pytest
import torch

from ternary_weight_int8_gb300 import pq2
import attn_util as A

pytestmark = pytest.mark.gpu

BF16 = A.BF16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pq2.lib()
    yield
    torch.cuda.synchronize()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def while_the_current_stream_is_busy(nbytes, call):
    """A copy of `nbytes` bytes of 7 waits on the current stream behind 0.1 s of
    work, its source is let go of, and the call runs on another stream meanwhile:
    its outputs are those of the same call alone, and the copy is all 7."""
    want = call(None)
    side = torch.cuda.Stream()
    source = torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda")
    copy = torch.zeros_like(source)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    copy.copy_(source)
    del source
    got = call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    assert bool((copy == 7).all())


@pytest.mark.parametrize("given", [True, False])
def test_prefill(given):
    nq, nk, H, G, D = 60, 9000, 2, 2, 128
    q, k, v = (torch.randn((n, h, D), generator=A.gen(n + h), device="cuda").to(BF16)
               for n, h in ((nq, H * G), (nk, H), (nk, H)))
    cu = ints([0, nq]), ints([0, nk])
    out = torch.empty_like(q) if given else None
    nbytes = pq2.lib().pq2_attn_prefill_workspace_bytes(1, nq, nk, H * G, H, D)
    assert nbytes
    call = lambda s: [pq2.pq2_attn_prefill(q, k, v, *cu, out=out, stream=s).clone()  # noqa: E731
                      if s is None else pq2.pq2_attn_prefill(q, k, v, *cu, out=out, stream=s)]
    while_the_current_stream_is_busy(nbytes if given else q.numel() * 2, call)


@pytest.mark.parametrize("given", [True, False])
def test_decode_and_load(given):
    n, H, G, D, width = 3000, 4, 5, 128, 10000
    cache, table, _ = A.make_cache(2, [n, 77], H, 16, D, BF16, seed=1, width=width)
    q = torch.randn((2, H * G, D), generator=A.gen(3), device="cuda").to(BF16)
    lens = ints([n, 77])
    out = torch.empty_like(q) if given else None
    nbytes = pq2.lib().pq2_attn_decode_workspace_bytes(2, 1, H * G, H, D, width * 16)
    assert nbytes
    call = lambda s: [pq2.pq2_attn_decode(q, cache, table, lens, out=out, stream=s).clone()  # noqa: E731
                      if s is None else
                      pq2.pq2_attn_decode(q, cache, table, lens, out=out, stream=s)]
    while_the_current_stream_is_busy(nbytes if given else q.numel() * 2, call)
    cu = ints([0, n, n + 77])
    load = lambda s: pq2.pq2_kv_load(cache, table, lens, cu=cu, tokens=n + 77, stream=s)  # noqa: E731
    while_the_current_stream_is_busy((n + 77) * H * D * 2, load)


def test_captured_prefills_replayed_at_once():
    """Two graphs whose calls have workspaces (keys in parts), replayed on two streams
    while eager calls run on a third."""
    nq, nk, H, G, D = 60, 9000, 2, 2, 128
    k, v = (torch.randn((nk, H, D), generator=A.gen(s), device="cuda").to(BF16) for s in (1, 2))
    qs = [torch.randn((nq, H * G, D), generator=A.gen(s), device="cuda").to(BF16) for s in (3, 4)]
    cu = ints([0, nq]), ints([0, nk])
    want = [pq2.pq2_attn_prefill(q, k, v, *cu) for q in qs]
    outs, graphs = [torch.empty_like(q) for q in qs], []
    for q, out in zip(qs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(10):
                pq2.pq2_attn_prefill(q, k, v, *cu, out=out)
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(4):
        for g, s, o in zip(graphs, streams, outs):
            with torch.cuda.stream(s):
                o.zero_()
                g.replay()
        eager = [pq2.pq2_attn_prefill(q, k, v, *cu) for q in qs * 3]
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        assert all(torch.equal(o, w) for o, w in zip(eager, want * 3))
