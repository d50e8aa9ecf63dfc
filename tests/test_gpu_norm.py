"""pq2_norm_gate_residual against the definition in 64 bits.

Tolerance (fixed before the first run): a mean of K squares in fp32 is within
(K / 256 + 32) * 2^-24 of its value (terms of one sign, at most K / 256 in a
row and a tree above), its inverse square root within half of that and two
roundings; each further operation adds 2^-24.  With e = (K / 256 + 64) * 2^-24:
  |h' - exact| <= e (|h| + |alpha g p|),
  |n - exact|  <= e (|h| + |alpha g p|) |inv (w + o)| + e |n|
(h' carries its own error into the mean, which the last term covers twice
over), and half a unit in the last place for a 16-bit output."""
import pytest
import torch

from ternary_weight_int8_gb300 import pq2
import gpu_util as U

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 0.0}  # half a unit over the value, at most


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pq2.lib()
    yield
    torch.cuda.synchronize()


def tensors(M, K, dtype, seed, gates=0, pad=0, shift=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def mk(rows, spread, mean=0.0):
        v = (torch.randn((rows, K), generator=g, device="cuda") * spread + mean).to(dtype)
        back = torch.full((rows * (K + pad) + shift,), float("nan"), dtype=dtype, device="cuda")
        view = back[shift:].view(rows, K + pad)[:, :K]
        view.copy_(v)
        return view
    return {"z": mk(M, 3), "h": mk(M, 10), "w_post": mk(1, 0.2, 1)[0].contiguous(),
            "w_pre": mk(1, 0.2, 1)[0].contiguous(), "gate": mk(gates, 1) if gates else None}


def check(t, rows_per_gate=1, alpha=1.0, eps=1e-6, w_offset=0.0, post=True, in_place=False):
    M, K = t["h"].shape
    dtype = t["h"].dtype
    z, h = (t["z"].double() if t["z"] is not None else None), t["h"].double()
    add = torch.zeros_like(h)
    if z is not None:
        if post:
            z = z * torch.rsqrt(z.square().mean(1, keepdim=True) + eps) * \
                (t["w_post"].double() + w_offset)
        if t["gate"] is not None:
            z = z * t["gate"].double().repeat_interleave(rows_per_gate, 0)[:M]
        add = alpha * z
    e_h = h + add
    inv = torch.rsqrt(e_h.square().mean(1, keepdim=True) + eps)
    w = t["w_pre"].double() + w_offset
    e_n = e_h * inv * w
    nb, n_back, guard = U.guarded((M, K), dtype)
    hb, h_back, _ = U.guarded((M, K), dtype)
    src = t["h"]
    if in_place:
        hb.copy_(src)
        src = hb
    h_out, n_out = pq2.pq2_norm_gate_residual(
        t["z"], src, t["w_pre"], w_post=t["w_post"] if post else None, gate=t["gate"],
        rows_per_gate=rows_per_gate, alpha=alpha, eps=eps, w_offset=w_offset,
        h_out=hb if t["z"] is not None else None, n_out=nb)
    torch.cuda.synchronize()
    assert U.guards_intact(n_back, guard) and U.guards_intact(h_back, guard)
    e = (K / 256 + 64) * 2.0 ** -24
    mag = h.abs() + add.abs()
    half = HALF[dtype]
    tiny = 2.0 ** -25 if dtype == F16 else 0.0
    off_n = (n_out.double() - e_n).abs() - (
        (e * mag * (inv * w).abs() + e * e_n.abs()) * (1 + half) + half * e_n.abs() * 1.01 + tiny)
    assert bool((off_n <= 0).all()), float(off_n.max())
    if t["z"] is None:
        assert h_out is None
        return
    off_h = (h_out.double() - e_h).abs() - (
        e * mag * (1 + half) + half * e_h.abs() * 1.01 + tiny)
    assert bool((off_h <= 0).all()), float(off_h.max())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (2, 100), (1, 1000), (5, 1024), (1, 5120),
                                 (40, 5119), (700, 2048), (3, 8200), (2, 17408), (1, 32768),
                                 (513, 4096), (2, 30001), (9, 12288)])
def test_within_bound(dtype, M, K):
    check(tensors(M, K, dtype, seed=M + K, gates=1), rows_per_gate=M)
    check(tensors(M, K, dtype, seed=M + K, gates=M), alpha=0.5, w_offset=1.0)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (3, 1), (0, 1), (0, 4)])
def test_strides_and_alignments(dtype, pad, shift):
    for K in (1280, 1283):
        t = tensors(6, K, dtype, seed=K, gates=2, pad=pad, shift=shift)
        check(t, rows_per_gate=3)
        w = torch.empty(K + 1, dtype=dtype, device="cuda")[1:]
        w.copy_(t["w_pre"])
        t["w_pre"] = w
        check(t, rows_per_gate=4)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [640, 5120, 20000])
def test_parts(dtype, K):
    """No post norm, no gate, no block output at all, in place, one output."""
    t = tensors(11, K, dtype, seed=K)
    check(t, post=False, alpha=-0.25)
    check(t, in_place=True)
    check({**t, "z": None}, post=False)
    h, n = pq2.pq2_norm_gate_residual(t["z"], t["h"], t["w_pre"], w_post=t["w_post"])
    h1, n1 = pq2.pq2_norm_gate_residual(t["z"], t["h"], None, w_post=t["w_post"])
    assert n1 is None and torch.equal(h1, h)
    assert torch.equal(pq2.pq2_norm_gate_residual(t["z"], t["h"], t["w_pre"],
                                                  w_post=t["w_post"])[1], n)


def test_special_rows():
    """A zero row stays zero (eps > 0); a NaN shows in its own row only; large
    and small magnitudes keep their precision."""
    t = tensors(5, 3000, F32, seed=1)
    t["z"][0] = 0
    t["h"][0] = 0
    t["z"][1] *= 1e15
    t["z"][2] *= 1e-15
    t["h"][2] *= 1e-15
    check(t, eps=1e-35)
    h0, n0 = pq2.pq2_norm_gate_residual(t["z"], t["h"], t["w_pre"], w_post=t["w_post"])
    assert not h0[0].any() and not n0[0].any()
    t["z"][3, 17] = float("nan")
    h1, n1 = pq2.pq2_norm_gate_residual(t["z"], t["h"], t["w_pre"], w_post=t["w_post"])
    keep = [0, 1, 2, 4]
    assert torch.equal(h1[keep], h0[keep]) and torch.equal(n1[keep], n0[keep])
    assert bool(h1[3].isnan().all()) and bool(n1[3].isnan().all())


def test_row_bits_do_not_depend_on_the_batch():
    t = tensors(300, 5120, BF16, seed=2, gates=300)
    h, n = pq2.pq2_norm_gate_residual(t["z"], t["h"], t["w_pre"], w_post=t["w_post"],
                                      gate=t["gate"])
    for a, b in ((0, 1), (7, 12), (200, 300)):
        h1, n1 = pq2.pq2_norm_gate_residual(t["z"][a:b], t["h"][a:b], t["w_pre"],
                                            w_post=t["w_post"], gate=t["gate"][a:b])
        assert torch.equal(h1, h[a:b]) and torch.equal(n1, n[a:b])


def test_offsets_beyond_32_bits():
    M, K = 140000, 16384
    h = torch.ones((M, K), dtype=BF16, device="cuda")
    h[M - 1] = 3
    _, n = pq2.pq2_norm_gate_residual(None, h, torch.ones(K, dtype=BF16, device="cuda"))
    assert h.numel() > 1 << 31
    assert bool((n[0] == 1).all()) and bool((n[M - 1] == 1).all()) and bool((n[M // 2] == 1).all())


def test_chain_on_another_stream():
    t = tensors(4, 5120, BF16, seed=3)
    want = []
    h, n = t["h"], t["z"]
    for _ in range(5):
        h, n = pq2.pq2_norm_gate_residual(n, h, t["w_pre"], w_post=t["w_post"])
        torch.cuda.synchronize()
        want.append((h, n))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        h, n = t["h"].clone(), t["z"]
        for _ in range(5):
            h, n = pq2.pq2_norm_gate_residual(n, h, t["w_pre"], w_post=t["w_post"], h_out=h)
    s.synchronize()
    assert torch.equal(h, want[-1][0]) and torch.equal(n, want[-1][1])


def test_refusals():
    t = tensors(2, 64, BF16, seed=4)
    big = torch.zeros((1, 32769), dtype=BF16, device="cuda")
    for bad in (lambda: pq2.pq2_norm_gate_residual(None, big, big[0]),
                lambda: pq2.pq2_norm_gate_residual(None, t["h"], None),
                lambda: pq2.pq2_norm_gate_residual(None, t["h"], t["w_pre"], w_post=t["w_post"]),
                lambda: pq2.pq2_norm_gate_residual(t["z"], t["h"], t["w_pre"], eps=-1.0),
                lambda: pq2.pq2_norm_gate_residual(t["z"], t["h"], t["w_pre"], eps=float("nan"))):
        with pytest.raises(pq2.Pq2Error):
            bad()
    for bad in (lambda: pq2.pq2_norm_gate_residual(t["z"].float(), t["h"], t["w_pre"]),
                lambda: pq2.pq2_norm_gate_residual(t["z"][:1], t["h"], t["w_pre"]),
                lambda: pq2.pq2_norm_gate_residual(t["z"], t["h"], t["w_pre"],
                                                   gate=t["z"][:1])):
        with pytest.raises(ValueError):
            bad()
