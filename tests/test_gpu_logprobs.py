"""pq2_token_logprobs against the definition in 64 bits.

Tolerance (fixed before the first run): u = (x - max) * scale has two
roundings, 2^-23 |u| with |u| <= 104 where exp(u) counts; exp and log are
within 2^-22; S and W are sums of terms of one sign, at most V / 256 in a row
and a tree above, so their relative error is at most (V / 256 + 32) * 2^-24.
With eps = (V / 256 + 512) * 2^-24:
  |log p - exact| <= eps + 2^-22 |log p|,   |H - exact| <= eps (2 + 2 H).
The ids are exact: the order of a stable descending sort."""
import math

import pytest
import torch

from ternary_weight_int8_gb300 import pq2
import gpu_util as U

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pq2.lib()
    yield
    torch.cuda.synchronize()


def logits(M, V, dtype, seed, spread=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((M, V), generator=g, device="cuda") * spread
    tokens = torch.randint(0, V, (M, 2), generator=g, device="cuda")
    return x.to(dtype), tokens


def exact(x, tokens, k, scale):
    t = x.double() * scale
    logp = torch.log_softmax(t, 1)
    logp[torch.isneginf(t).all(1)] = -INF
    p = logp.exp()
    H = -torch.where(p > 0, p * logp, 0.0).sum(1)
    ids = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :k]
    return logp.gather(1, tokens), H, ids, logp.gather(1, ids)


def near(a, b, tol):
    a, b = a.double(), b.double()
    fine = b.isfinite()
    assert torch.equal(fine, a.isfinite())
    assert bool((a[~fine] == b[~fine]).all())
    off = ((a - b).abs() - tol(b.abs()))[fine]
    assert not off.numel() or bool((off <= 0).all()), float(off.max())


def check(x, tokens, k, scale=1.0):
    M, V = x.shape
    T = tokens.shape[1]
    bufs = [U.guarded((M, T), F32), U.guarded((M,), F32),
            U.guarded((max(M * k, 1),), torch.int32), U.guarded((M, max(k, 1)), F32)]
    ids_back = torch.full((M * k + 16,), -77, dtype=torch.int64, device="cuda")
    ids_buf = ids_back[8:8 + M * k].view(M, k)
    out = (bufs[0][0], bufs[1][0], ids_buf, bufs[3][0][:, :k].contiguous() if not k else bufs[3][0])
    lp, H, ids, top = pq2.pq2_token_logprobs(x, tokens, k, scale=scale, out=out)
    torch.cuda.synchronize()
    assert bool((ids_back[:8] == -77).all()) and bool((ids_back[8 + M * k:] == -77).all())
    for _, back, guard in (bufs[0], bufs[1], bufs[3]):
        assert U.guards_intact(back, guard)
    e_lp, e_H, e_ids, e_top = exact(x, tokens, k, scale)
    assert torch.equal(ids, e_ids)
    eps = (V / 256 + 512) * 2.0 ** -24
    near(lp, e_lp, lambda b: eps + 2.0 ** -22 * b)
    near(top, e_top, lambda b: eps + 2.0 ** -22 * b)
    near(H, e_H, lambda b: eps * (2 + 2 * b))
    again = pq2.pq2_token_logprobs(x, tokens, k, scale=scale)
    assert torch.equal(again[0], lp) and torch.equal(again[1], H) and torch.equal(again[3], top)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,V,k", [(1, 1, 1), (2, 7, 7), (3, 32, 32), (5, 33, 32), (4, 1000, 8),
                                   (1, 4096, 1), (300, 1003, 5), (2, 8191, 20), (1, 100003, 32),
                                   (7, 131072, 20), (33, 50001, 0), (160, 16384, 3),
                                   (700, 5000, 1), (1, 1 << 20, 8), (17, 262147, 32)])
def test_values_and_order(dtype, M, V, k):
    x, tokens = logits(M, V, dtype, seed=M + V)
    check(x, tokens, k)


@pytest.mark.parametrize("scale", [0.05, 0.7, 1.25, 30.0])
def test_scale(scale):
    x, tokens = logits(6, 20011, BF16, seed=1)
    check(x, tokens, 5, scale)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("pad,shift", [(5, 0), (8, 0), (1, 3), (0, 1), (64, 7)])
def test_strides_and_alignments(dtype, pad, shift):
    M, V = 9, 10007
    x, tokens = logits(M, V, dtype, seed=2)
    back = torch.full((M * (V + pad) + shift,), float("nan"), dtype=dtype, device="cuda")
    view = back[shift:].view(M, V + pad)[:, :V]
    view.copy_(x)
    check(view, tokens, 6)


@pytest.mark.parametrize("V", [100, 5000, 70001])
@pytest.mark.parametrize("k", [1, 7, 32])
def test_orders_and_ties(V, k):
    """Constant, rising, falling, few-valued rows, both zeros, a late and an
    early maximum."""
    j = torch.arange(V, device="cuda")
    rows = [torch.zeros(V, device="cuda"), j / V * 10, -j / V * 10, (j % 3).float(),
            (j // 64 % 2).float() * 4, torch.where(j % 2 == 0, -0.0, 0.0),
            torch.where(j == V - 1, 9.0, (j % 5).float()), torch.where(j == 0, 9.0, 0.0),
            torch.full((V,), -3.0e38, device="cuda"), torch.full((V,), 3.0e38, device="cuda")]
    x = torch.stack(rows)
    tokens = torch.randint(0, V, (len(rows), 2), device="cuda",
                           generator=torch.Generator("cuda").manual_seed(3))
    check(x, tokens, k)
    check(x[:8].to(BF16), tokens[:8], k)
    check(x[:8].half(), tokens[:8], k)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("V,k", [(64, 5), (5003, 32), (100003, 20), (131072, 1)])
def test_masked_rows(dtype, V, k):
    """-inf in most places: rows that leave everything, many, few, one (first,
    last, inside) and none; the type's lowest value as a mask."""
    x, tokens = logits(9, V, dtype, seed=4)
    g = torch.Generator("cuda").manual_seed(5)
    keep = torch.rand((9, V), generator=g, device="cuda") < \
        torch.tensor([1, 0.5, 0.01, 3 / V, 0, 0, 0, 0, 0.02], device="cuda")[:, None]
    keep[4, 0] = keep[5, V - 1] = keep[6, V // 2] = True
    low = torch.finfo(dtype).min
    x = torch.where(keep, x, torch.where(torch.arange(9, device="cuda")[:, None] == 8, low, -INF)
                    .to(dtype))
    assert bool(torch.isneginf(x[7]).all())
    check(x, tokens, k)


@pytest.mark.parametrize("V", [10, 4097, 100003])
def test_nan_and_infinity(V):
    """NaN or +inf anywhere makes the row's numbers NaN and leaves its
    neighbours alone; the ids stay in range and distinct, NaN last."""
    k = 5
    x, tokens = logits(5, V, F32, seed=6)
    clean = pq2.pq2_token_logprobs(x, tokens, k)
    x[1, V // 2] = float("nan")
    x[2, V - 1] = INF
    x[3] = float("nan")
    lp, H, ids, top = pq2.pq2_token_logprobs(x, tokens, k)
    for r in (0, 4):
        assert torch.equal(lp[r], clean[0][r]) and torch.equal(ids[r], clean[2][r])
        assert H[r] == clean[1][r] and torch.equal(top[r], clean[3][r])
    assert bool(lp[1:4].isnan().all()) and bool(H[1:4].isnan().all())
    assert bool(top[1:4].isnan().all())
    order = torch.where(x[1].isnan(), -INF, x[1])
    assert torch.equal(ids[1], torch.sort(order, descending=True, stable=True).indices[:k])
    assert int(ids[2, 0]) == V - 1
    assert torch.equal(ids[3], torch.arange(k, device="cuda"))


def test_tokens_outside_the_vocabulary():
    x, _ = logits(2, 500, BF16, seed=7)
    tokens = torch.tensor([[-1, 3, 500], [-(1 << 40), 1 << 40, 499]], device="cuda")
    lp, *_ = pq2.pq2_token_logprobs(x, tokens)
    assert lp[0, 0] == 0 and lp[1, 0] == 0
    assert bool(lp[0, 2].isnan()) and bool(lp[1, 1].isnan())
    want = torch.log_softmax(x.double(), 1)
    assert abs(float(lp[0, 1] - want[0, 3])) < 1e-4 and abs(float(lp[1, 2] - want[1, 499])) < 1e-4


def test_optional_parts():
    x, tokens = logits(4, 3001, F16, seed=8)
    lp, H, ids, top = pq2.pq2_token_logprobs(x, tokens, 4)
    a = pq2.pq2_token_logprobs(x, None, 0)
    assert a[0].shape == (4, 0) and torch.equal(a[1], H) and a[2].shape == (4, 0)
    b = pq2.pq2_token_logprobs(x, tokens[:, 0].contiguous(), 2, entropy=False)
    assert b[1] is None and torch.equal(b[0][:, 0], lp[:, 0]) and torch.equal(b[2], ids[:, :2])
    many = torch.arange(3001, device="cuda").repeat(4, 1)
    c = pq2.pq2_token_logprobs(x, many)
    assert abs(float(c[0][1].double().exp().sum()) - 1) < 1e-3


def test_rows_do_not_depend_on_their_number():
    x, tokens = logits(400, 20000, BF16, seed=9)
    ids = pq2.pq2_token_logprobs(x, tokens, 9)[2]
    for a, b in ((0, 1), (5, 7), (100, 164)):
        assert torch.equal(pq2.pq2_token_logprobs(x[a:b], tokens[a:b], 9)[2], ids[a:b])


def test_matrix_beyond_32_bits():
    M, V = 70000, 40009
    x = torch.empty((M, V), dtype=BF16, device="cuda")
    x.random_(0, 100)
    assert x.numel() > 1 << 31
    tokens = torch.full((M, 1), 5, device="cuda")
    lp, H, ids, top = pq2.pq2_token_logprobs(x, tokens, 2)
    rows = torch.tensor([0, 1, 53000, M - 1], device="cuda")
    e_lp, e_H, e_ids, _ = exact(x[rows], tokens[rows], 2, 1.0)
    assert torch.equal(ids[rows], e_ids)
    assert float((lp[rows].double() - e_lp).abs().max()) < 1e-3
    assert float((H[rows].double() - e_H).abs().max()) < 1e-3


def test_streams_and_capture():
    x, tokens = logits(3, 131072, F32, seed=10)
    want = pq2.pq2_token_logprobs(x, tokens, 8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [pq2.pq2_token_logprobs(x, tokens, 8) for _ in range(3)]
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(pq2.pq2_token_logprobs(x, tokens, 8))
    graph.replay()
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_refusals():
    x, tokens = logits(2, 50, F32, seed=11)
    for bad in (lambda: pq2.pq2_token_logprobs(x, tokens, 33),
                lambda: pq2.pq2_token_logprobs(x[:, :10], tokens, 11),
                lambda: pq2.pq2_token_logprobs(x, tokens, 1, scale=0.0),
                lambda: pq2.pq2_token_logprobs(x, tokens, 1, scale=-1.0),
                lambda: pq2.pq2_token_logprobs(x, tokens, 1, scale=float("nan")),
                lambda: pq2.pq2_token_logprobs(x[:0], None, 1)):
        with pytest.raises(pq2.Pq2Error):
            bad()
    for bad in (lambda: pq2.pq2_token_logprobs(x, tokens.int(), 1),
                lambda: pq2.pq2_token_logprobs(x, tokens[:1], 1),
                lambda: pq2.pq2_token_logprobs(x.t(), None, 1)):
        with pytest.raises(ValueError):
            bad()
