"""pq2_attn_prefill against the definition in 64 bits (bounds in attn_util)."""
import math

import pytest
import torch

from ternary_weight_int8_gb300 import pq2
import attn_util as A
import gpu_util as U

pytestmark = pytest.mark.gpu

BF16, F16, F32, I8 = A.BF16, A.F16, A.F32, A.I8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pq2.lib()
    yield
    torch.cuda.synchronize()


def sums(x):
    total = [0]
    for n in x:
        total.append(total[-1] + n)
    return torch.tensor(total, dtype=torch.int32, device="cuda")


def inputs(nq, nk, H, G, D, dtype, seed, spare=0):
    g = A.gen(seed)
    q = torch.randn((sum(nq) + spare, H * G, D), generator=g, device="cuda").to(dtype)
    k, v = ((torch.randn((sum(nk) + spare, H, D), generator=g, device="cuda") + b).to(dtype)
            for b in (0.0, 0.3))
    return q, k, v


def check(q, k, v, nq, nk, scale=None, causal=True, heads=None):
    out, back, guard = U.guarded(q.shape, q.dtype)
    lse, lback, lguard = U.guarded(q.shape[:-1], F32)
    back.fill_(float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu_q, cu_k = sums(nq), sums(nk)
    pq2.pq2_attn_prefill(q, k, v, cu_q, cu_k, scale=scale, causal=causal, out=out, lse=lse,
                         status=status)
    torch.cuda.synchronize()
    assert not int(status)
    assert U.guards_intact(back, guard) and U.guards_intact(lback, lguard)
    assert bool(out[sum(nq):].isnan().all()) and bool(lse[sum(nq):].isnan().all())
    verify(out, lse, q, k, v, nq, nk, scale, causal, heads)
    again = pq2.pq2_attn_prefill(q, k, v, cu_q, cu_k, scale=scale, causal=causal)
    assert torch.equal(again[:sum(nq)], out[:sum(nq)])
    return out


def verify(out, lse, q, k, v, nq, nk, scale=None, causal=True, heads=None):
    D = q.shape[2]
    G = q.shape[1] // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    a = c = 0
    for n, m in zip(nq, nk):
        most = torch.full((n,), m, device="cuda")
        if causal:
            most = m - n + 1 + torch.arange(n, device="cuda")
        for h in range(q.shape[1]) if heads is None else heads:
            ref = A.attend(q[a:a + n, h].double(), k[c:c + m, h // G].double(),
                           v[c:c + m, h // G].double(), most, scale)
            A.check_rows(out[a:a + n, h], None if lse is None else lse[a:a + n, h], ref, D, q.dtype)
        a, c = a + n, c + m


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,H,G", [
    ([1], 1, 1), ([2], 2, 5), ([37], 8, 5), ([127, 128, 129], 1, 1), ([1, 0, 255, 256, 257], 2, 2),
    ([500], 1, 6), ([33, 1, 64, 65, 100], 2, 8), ([20, 3], 1, 16), ([9], 1, 128), ([300], 1, 3),
    ([7] * 40, 2, 4), ([700, 20], 1, 1)])
def test_whole_prompts(dtype, D, nq, H, G):
    q, k, v = inputs(nq, nq, H, G, D, dtype, seed=len(nq) + D, spare=5)
    check(q, k, v, nq, nq)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H,G", [
    ([1], [1], 1, 4), ([1, 1, 1], [200, 128, 129], 2, 6), ([16, 40], [1000, 41], 2, 5),
    ([5, 300, 7], [0, 100, 7], 1, 3), ([130], [64], 2, 1), ([129, 2], [1030, 2000], 1, 8),
    ([64], [4097], 2, 2), ([0, 10, 0], [5, 10, 9], 1, 2)])
def test_chunks(dtype, D, causal, nq, nk, H, G):
    """Keys before the chunk, fewer keys than rows (rows that see none), none."""
    q, k, v = inputs(nq, nk, H, G, D, dtype, seed=sum(nk) + D)
    check(q, k, v, nq, nk, causal=causal)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long(D):
    nq = [3001, 1200]
    q, k, v = inputs(nq, nq, 2, 2, D, BF16, seed=D)
    check(q, k, v, nq, nq, heads=[0, 3])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H,G", [
    ([1], [20000], 1, 1), ([70], [9001], 2, 5), ([40, 0, 300], [6000, 50, 12000], 1, 6),
    ([3, 200], [0, 17000], 2, 3), ([700], [20000], 1, 2), ([300, 5], [70, 5000], 1, 1)])
def test_few_rows_before_many_keys(dtype, D, causal, nq, nk, H, G):
    """The keys of a tile in several parts, joined: rows that see none of a part's
    keys, or none at all, sequences with fewer key tiles than parts."""
    B, rows, keys = len(nq), sum(nq), sum(nk)
    nbytes = pq2.lib().pq2_attn_prefill_workspace_bytes(B, rows, keys, H * G, H, D)
    parts = nbytes // (rows * H * G * (D + 2) * 4)
    assert parts > 1 and parts * rows * H * G * (D + 2) * 4 == nbytes
    q, k, v = inputs(nq, nk, H, G, D, dtype, seed=sum(nk) + D, spare=3)
    check(q, k, v, nq, nk, causal=causal, heads=[0, H * G - 1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_seen_in_parts(D, bad):
    """A later token's value that is not finite stays out of the rows before it in
    the join too, and is in the rows that see it."""
    nq, nk = [60], [9000]
    q, k, v = inputs(nq, nk, 1, 2, D, BF16, seed=5, spare=64)
    v[8970, 0, 5:9], v[9000:], k[9000:] = bad, bad, bad
    out = pq2.pq2_attn_prefill(q, k, v, sums(nq), sums(nk))
    most = 8970 - (9000 - 60)  # rows before it
    ref = out[:most].clone()
    verify(ref, None, q[:most], k, v, [most], [8970])
    assert not bool(out[most:60, :, 5:9].isfinite().any())
    assert bool(out[most:60, :, 9:].isfinite().all())
    k[10] = float("nan")
    assert bool(pq2.pq2_attn_prefill(q, k, v, sums(nq), sums(nk))[:60].isnan().all())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_no_keys_at_all(D):
    q, k, v = inputs([5, 3], [0, 0], 2, 3, D, BF16, seed=1)
    assert k.shape[0] == 0
    out = check(q, k, v, [5, 3], [0, 0])
    assert not out.any()


@pytest.mark.parametrize("nk", [60, 9000])
def test_rows_before_the_first_sequence(nk):
    """Sums that begin above 0: those rows stay as they were, with keys in one part
    and in several."""
    q, k, v = inputs([40], [nk], 2, 2, 128, BF16, seed=1)
    want = pq2.pq2_attn_prefill(q[7:], k[9:], v[9:], sums([33]), sums([nk - 9]))
    out = torch.full_like(q, float("nan"))
    cu_q, cu_k = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([7, 40], [9, nk]))
    pq2.pq2_attn_prefill(q, k, v, cu_q, cu_k, out=out)
    assert bool(out[:7].isnan().all())
    tol = 2.0 ** -7 * float(v.float().abs().max())
    assert float((out[7:].float() - want.float()).abs().max()) <= tol


def test_a_stream_given_by_name():
    nq, nk = [40], [9000]
    q, k, v = inputs(nq, nk, 2, 2, 128, BF16, seed=1)
    want = pq2.pq2_attn_prefill(q, k, v, sums(nq), sums(nk))
    torch.cuda.synchronize()
    side, cu = torch.cuda.Stream(), (sums(nq), sums(nk))
    torch.cuda.synchronize()
    outs = [torch.empty_like(q) for _ in range(8)]
    for out in outs:  # the workspaces are let go of while that stream still uses them
        pq2.pq2_attn_prefill(q, k, v, *cu, out=out, stream=side)
        torch.empty(1 << 22, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)


def test_a_workspace_of_the_callers():
    nq, nk = [50, 9], [9000, 5000]
    q, k, v = inputs(nq, nk, 2, 4, 128, F16, seed=2)
    want = check(q, k, v, nq, nk)
    nbytes = pq2.lib().pq2_attn_prefill_workspace_bytes(2, 59, 14000, 8, 2, 128)
    back = torch.full((nbytes + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    got = pq2.pq2_attn_prefill(q, k, v, sums(nq), sums(nk), workspace=back[256:256 + nbytes])
    assert torch.equal(got, want)
    assert bool((back[:256] == 0x5A).all()) and bool((back[256 + nbytes:] == 0x5A).all())
    with pytest.raises(pq2.Pq2Error):
        pq2.pq2_attn_prefill(q, k, v, sums(nq), sums(nk), workspace=back[256:256 + nbytes - 16])


@pytest.mark.parametrize("B", [1000, 2500])
def test_many_sequences(B):
    nq = [(7 * b) % 4 for b in range(B)]
    q, k, v = inputs(nq, nq, 1, 2, 64, F16, seed=1)
    out = pq2.pq2_attn_prefill(q, k, v, sums(nq))
    few = sum(nq[:300])
    verify(out[:few], None, q[:few], k[:few], v[:few], nq[:300], nq[:300])
    last = sum(nq[:-200])
    verify(out[last:], None, q[last:], k[last:], v[last:], nq[-200:], nq[-200:])


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 4.0])
def test_scales_of_the_scores(scale):
    nq = [300, 45]
    q, k, v = inputs(nq, nq, 2, 2, 64, F16, seed=7)
    check(q, k, v, nq, nq, scale=scale)


@pytest.mark.parametrize("order", ["rising", "falling", "late"])
@pytest.mark.parametrize("D", [64, 256])
def test_orders_of_the_scores(order, D):
    n = 700
    j = torch.arange(n, device="cuda")
    size = {"rising": j / n * 200, "falling": 200 - j / n * 200,
            "late": torch.where(j >= n - 130, 300.0, 0.0)}[order]
    q, k, v = inputs([n], [n], 1, 4, D, BF16, seed=2)
    k.zero_()
    k[:, 0, 0] = size.bfloat16()
    q.zero_()
    q[..., 0] = torch.tensor([1.0, 0.5, -1.0, 0.0], device="cuda")
    check(q, k, v, [n], [n], scale=1.0)
    check(q, k, v, [n], [n], scale=1.0, causal=False)


def test_strides():
    """q, k and v as columns of one projection's rows, and head-major tensors."""
    T, H, G, D = 150, 2, 3, 128
    qkv = torch.full((T, (H * G + 2 * H) * D + 8), float("nan"), dtype=BF16, device="cuda")
    nq = [100, 50]
    q0, k0, v0 = inputs(nq, nq, H, G, D, BF16, seed=4)
    cuts = [0, H * G * D, (H * G + H) * D, (H * G + 2 * H) * D]
    q, k, v = (qkv[:, a:b].unflatten(1, (-1, D)) for a, b in zip(cuts, cuts[1:]))
    for x, y in ((q, q0), (k, k0), (v, v0)):
        x.copy_(y)
    want = check(q, k, v, nq, nq)
    turned = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q0, k0, v0)]
    assert torch.equal(check(*turned, nq, nq), want)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_seen_takes_no_part(D, bad):
    """Keys and values of other sequences, behind the last one and after the row
    itself, that are infinite or NaN."""
    nq = [70, 60, 90]
    q, k, v = inputs(nq, nq, 1, 2, D, BF16, seed=5, spare=64)
    clean = pq2.pq2_attn_prefill(q, k, v, sums(nq))
    k[70:130], v[70:130], k[220:], v[220:] = bad, bad, bad, bad
    q[70:130] = bad
    out = pq2.pq2_attn_prefill(q, k, v, sums(nq))
    assert torch.equal(out[:70], clean[:70]) and torch.equal(out[130:220], clean[130:220])
    # a later token of the same prompt
    q, k, v = inputs(nq, nq, 1, 2, D, BF16, seed=5, spare=64)
    v[40, 0, 3], v[200] = bad, bad
    k[215] = float("nan")
    out = pq2.pq2_attn_prefill(q, k, v, sums(nq))
    verify(out[:40], None, q, k, v, [40], [40])
    w = v.clone()
    w[40, 0, 3] = 0
    part = pq2.pq2_attn_prefill(q, k, w, sums(nq))
    assert bool((out[40:70, :, 3] != out[40:70, :, 3]).all() if bad != bad
                else (out[40:70, :, 3] == bad).all())
    assert torch.equal(out[70:200], part[70:200])
    verify(out[130:200], None, q[130:], k[130:], v[130:], [70], [70])
    assert bool(out[215:220].isnan().all())


def test_a_cache_read_back_for_the_next_chunk():
    """A chunk through the cache as a server runs it: stored, read back with its
    prefix, attended; the last token of each prompt is the decode's too."""
    H, G, D, page = 2, 5, 128, 16
    past, new = [100, 0, 37], [30, 17, 1]
    lens = [p + n for p, n in zip(past, new)]
    g = A.gen(3)
    pages = sum(-(-n // page) for n in lens)
    cache = pq2.kv_cache(pages, H, page, D, torch.int8)
    table = torch.zeros((3, 9), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // page)
        table[b, :m] = torch.arange(at, at + m, dtype=torch.int32)
        at += m
    for rows, have in ((past, past), (new, lens)):
        k, v = (torch.randn((sum(rows), H, D), generator=g, device="cuda").bfloat16()
                for _ in range(2))
        pq2.pq2_kv_store(k, v, cache, table, sums(have).diff(), cu=sums(rows))
    n = sums(lens).diff()
    k, v = pq2.pq2_kv_load(cache, table, n, cu=sums(lens), tokens=sum(lens))
    q = torch.randn((sum(new), H * G, D), generator=g, device="cuda").bfloat16()
    out = check(q, k, v, new, lens)
    last = (sums(new)[1:] - 1).long()
    one = pq2.pq2_attn_decode(q[last], cache, table, n)
    # the same keys and values, rounded once more on the prefill's way
    assert float((one.float() - out[last].float()).abs().max()) <= \
        2.0 ** -7 * 2 * float(v.float().abs().max())


def test_streams_and_a_captured_graph():
    nq = [90, 33]
    q, k, v = inputs(nq, nq, 2, 3, 128, BF16, seed=1)
    want = check(q, k, v, nq, nq)
    side = torch.cuda.Stream()
    cu = sums(nq)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = [pq2.pq2_attn_prefill(q, k, v, cu) for _ in range(4)]
    outs += [pq2.pq2_attn_prefill(q, k, v, cu) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.full_like(q, float("nan"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pq2.pq2_attn_prefill(q, k, v, cu, out=out)
    cu.copy_(sums([20, 70]))
    graph.replay()
    torch.cuda.synchronize()
    verify(out[:90], None, q, k, v, [20, 70], [20, 70])
    assert bool(out[90:].isnan().all())
