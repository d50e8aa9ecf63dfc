"""4-bit weights with group scales: pq2_w4_prepare and pq2_w4_mmv against the
definition in 64 bits.

Tolerance (fixed before the first run), with B = sum_k |s (c - z) x|:
the products are exact; a group's sum is at most 8 tensor-core steps of 16
products, each within 2^-22 of the sum of magnitudes (8 * 2^-22 = 1.9e-6); the
scaling and the at most K/128 + 32 fp32 additions of group sums are within
2^-24 each (K = 17408: 1e-5 at the very worst, a tenth of it for sums of either
sign); the 32-bit x is held to 24 bits.  fp32 y: |y - y64| <= 1e-5 B.  16-bit
y: half a unit in the last place more."""
import numpy as np
import pytest
import torch

from ternary_weight_int8_gb300 import pq2
import gpu_util as U

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pq2.lib()
    yield
    torch.cuda.synchronize()


def raw(N, K, G, zeros, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand((N, K // G), generator=g, device="cuda") * 0.045 + 0.005).half()
    z = torch.randint(0, 16, (N, K // G), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales, z if zeros else None


def dense(codes, scales, z, G):
    """The weights in 64 bits."""
    N, K = codes.shape[0], codes.shape[1] * 2
    c = torch.empty((N, K), dtype=torch.float64, device=codes.device)
    c[:, 0::2] = (codes % 16).double()
    c[:, 1::2] = (codes // 16).double()
    zero = 8.0 if z is None else z.double().repeat_interleave(G, 1)
    return (c - zero) * scales.double().repeat_interleave(G, 1)


def acts(M, K, dtype, seed, pad=0, shift=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((M, K), generator=g, device="cuda")
    x[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 20
    back = torch.full((M * (K + pad) + shift,), float("nan"), dtype=dtype, device="cuda")
    view = back[shift:].view(M, K + pad)[:, :K]
    view.copy_(x)
    return view


def check(y, x, w):
    y64 = x.double() @ w.t()
    tol = 1e-5 * (x.double().abs() @ w.abs().t())
    if y.dtype == BF16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * y64.abs()
    if y.dtype == F16:
        tol = tol * (1 + 2.0 ** -11) + 2.0 ** -11 * y64.abs() + 2.0 ** -25
    off = (y.double() - y64).abs() - tol
    assert bool((off <= 0).all()), float(off.max())


@pytest.mark.parametrize("G", [128, 64, 32])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N,K", [(16, 256), (37, 416)])
def test_every_weight_is_where_it_belongs(G, zeros, dtype, N, K):
    """x a unit vector gives s (c - z), exactly, for every column."""
    K = K // G * G
    codes, scales, z = raw(N, K, G, zeros, seed=N + G)
    plane = pq2.pq2_w4_prepare(codes, scales, z, group=G)
    w = dense(codes, scales, z, G).float()
    for a in range(0, K, 32):
        x = torch.zeros((32, K), dtype=dtype, device="cuda")
        x[torch.arange(32), torch.arange(a, a + 32)] = 1
        y = pq2.pq2_w4_mmv(x, plane, N, G, zeros=zeros)
        assert torch.equal(y, w[:, a:a + 32].t())


@pytest.mark.parametrize("M", [1, 2, 5, 8, 9, 16, 23, 32])
@pytest.mark.parametrize("N,K,G,zeros", [(1, 32, 32, True), (5, 64, 64, False),
                                         (1000, 1152, 128, False), (1003, 4160, 32, True),
                                         (153, 17408, 128, True), (10240, 5120, 64, False),
                                         (2500, 2048, 128, True)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_within_bound(M, N, K, G, zeros, dtype):
    codes, scales, z = raw(N, K, G, zeros, seed=N + K)
    plane = pq2.pq2_w4_prepare(codes, scales, z, group=G)
    w = dense(codes, scales, z, G)
    x = acts(M, K, dtype, seed=M)
    for out in (F32, BF16, F16):
        y, back, guard = U.guarded((M, N), out)
        pq2.pq2_w4_mmv(x, plane, N, G, zeros=zeros, y=y)
        torch.cuda.synchronize()
        assert U.guards_intact(back, guard)
        check(y, x, w)


@pytest.mark.parametrize("M", [3, 13, 32])
@pytest.mark.parametrize("N,K,G", [(100, 70016, 64), (64, 30720, 128), (3000, 17408, 32)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_rows(M, N, K, G, dtype):
    """Ranges of units too long for one pass, or for the wide kernel's shared
    memory."""
    codes, scales, z = raw(N, K, G, True, seed=N)
    plane = pq2.pq2_w4_prepare(codes, scales, z, group=G)
    x = acts(M, K, dtype, seed=M)
    y = pq2.pq2_w4_mmv(x, plane, N, G, zeros=True)
    check(y, x, dense(codes, scales, z, G))
    assert torch.equal(pq2.pq2_w4_mmv(x[:1], plane, N, G, zeros=True), y[:1])


def test_small_and_large_x():
    """Magnitudes far from one keep their precision: tiny, huge and mixed
    columns of x."""
    N, K, G = 50, 768, 64
    codes, scales, z = raw(N, K, G, False, seed=15)
    plane = pq2.pq2_w4_prepare(codes, scales, group=G)
    for dtype in (BF16, F32):
        x = acts(6, K, F32, seed=16)
        x[0] *= 1e-30
        x[1] *= 1e30
        x[2, ::2] *= 1e-6
        x[3, 256:512] *= 1e20
        x[4, :256] *= 1e-20
        x = x.to(dtype)
        check(pq2.pq2_w4_mmv(x, plane, N, G), x, dense(codes, scales, None, G))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (3, 1), (0, 1), (32, 4)])
def test_strides_and_alignments_of_x(dtype, pad, shift):
    N, K, G = 300, 1280, 64
    codes, scales, z = raw(N, K, G, True, seed=3)
    plane = pq2.pq2_w4_prepare(codes, scales, z, group=G)
    x = acts(5, K, dtype, seed=4, pad=pad, shift=shift)
    y = pq2.pq2_w4_mmv(x, plane, N, G, zeros=True)
    same = pq2.pq2_w4_mmv(x.contiguous(), plane, N, G, zeros=True)
    assert torch.equal(y, same)
    check(y, x, dense(codes, scales, z, G))


def test_strided_and_unaligned_codes():
    N, K, G = 70, 416, 32
    codes, scales, z = raw(N, K, G, True, seed=5)
    back = torch.zeros(N * (K // 2 + 3) + 1, dtype=torch.uint8, device="cuda")
    view = back[1:].view(N, K // 2 + 3)[:, :K // 2]
    view.copy_(codes)
    assert torch.equal(pq2.pq2_w4_prepare(view, scales, z, group=G),
                       pq2.pq2_w4_prepare(codes, scales, z, group=G))


@pytest.mark.parametrize("N,K,G", [(10240, 5120, 128), (5120, 17408, 32), (1003, 4160, 32),
                                   (40000, 1024, 64)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_batch_invariance(N, K, G, dtype):
    codes, scales, z = raw(N, K, G, True, seed=6)
    plane = pq2.pq2_w4_prepare(codes, scales, z, group=G)
    x = acts(32, K, dtype, seed=7)
    full = pq2.pq2_w4_mmv(x, plane, N, G, zeros=True)
    assert torch.equal(full, pq2.pq2_w4_mmv(x, plane, N, G, zeros=True))
    for M in (1, 3, 8, 11, 17, 31):
        assert torch.equal(pq2.pq2_w4_mmv(x[:M], plane, N, G, zeros=True), full[:M]), M
    assert torch.equal(pq2.pq2_w4_mmv(x[31:], plane, N, G, zeros=True), full[31:])


def test_special_values():
    """A zero scale, a zero x and a code equal to its zero point give exact
    zeros; the largest fp16 scale stays finite; a NaN or infinite x shows in
    its own column only."""
    N, K, G = 40, 256, 32
    codes, scales, z = raw(N, K, G, True, seed=8)
    scales[3] = 0
    scales[7] = 65504.0
    codes[9] = 0x55
    z[9] = 5
    plane = pq2.pq2_w4_prepare(codes, scales, z, group=G)
    x = acts(4, K, BF16, seed=9)
    x[1] = 0
    good = pq2.pq2_w4_mmv(x, plane, N, G, zeros=True)
    check(good, x, dense(codes, scales, z, G))
    assert not good[:, 3].any() and not good[1].any() and not good[:, 9].any()
    x[2, 100] = float("nan")
    x[3, 7] = float("inf")
    y = pq2.pq2_w4_mmv(x, plane, N, G, zeros=True)
    assert torch.equal(y[:2], good[:2])
    assert bool(y[2].isnan().all()) and not bool(y[3].isfinite().any())


@pytest.mark.parametrize("M", [4, 20])
@pytest.mark.parametrize("dtype,most", [(BF16, 3e38), (F16, 6e4), (F32, 3e38)])
def test_infinite_x(dtype, most, M):
    """An infinite x gives the formula's infinities, with their signs, and NaN
    where the formula does (a weight of zero, infinities of both signs), also
    next to the largest finite values."""
    N, K, G = 40, 512, 32
    codes, scales, z = raw(N, K, G, True, seed=11)
    scales[3] = 0
    w = dense(codes, scales, z, G)
    plane = pq2.pq2_w4_prepare(codes, scales, z, group=G)
    x = acts(M, K, dtype, seed=12)
    x[1, 7], x[1, 8], x[1, 9] = float("inf"), -most, most
    x[2, 300], x[2, 301], x[2, 20] = float("-inf"), -most, 1.0
    x[3, 7], x[3, 400] = float("inf"), float("-inf")
    want = (x.double()[1:4, None] * w).sum(2)
    y = pq2.pq2_w4_mmv(x, plane, N, G, zeros=True, out_dtype=F32)
    assert not bool(want.isfinite().any()) and bool(want.isinf().any())
    assert torch.equal(y[1:4].double().nan_to_num(7.0, 1.0, -1.0), want.nan_to_num(7.0, 1.0, -1.0))
    rest = [0] + list(range(4, M))
    check(y[rest], x[rest], w)


def test_flags_streams_and_capture():
    """Both flags, another stream and a captured graph give the same bits, in
    a chain in which each call reads what the call before it wrote."""
    N, G = 2048, 64
    codes, scales, z = raw(N, N, G, False, seed=10)
    plane = pq2.pq2_w4_prepare(codes, scales, z, group=G)
    x = acts(3, N, F32, seed=11) * 1e-3

    def chain(flags, stream=None):
        ys = [x]
        for _ in range(6):
            ys.append(pq2.pq2_w4_mmv(ys[-1], plane, N, G, flags=flags, stream=stream))
        return ys

    want = []
    for _ in range(6):
        want.append(pq2.pq2_w4_mmv(want[-1] if want else x, plane, N, G))
        torch.cuda.synchronize()
    got = chain(pq2.PQ2_MMV_OVERLAP_WEIGHTS)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = chain(pq2.PQ2_MMV_OVERLAP_WEIGHTS)
        one = pq2.pq2_w4_mmv(x, plane, N, G, flags=pq2.PQ2_MMV_INDEPENDENT)
        two = pq2.pq2_w4_mmv(x, plane, N, G, flags=pq2.PQ2_MMV_INDEPENDENT)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want))
    assert torch.equal(one, want[0]) and torch.equal(two, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(pq2.PQ2_MMV_OVERLAP_WEIGHTS)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want))


def test_plane_beyond_32_bits():
    """A plane of more than 2^32 bytes: the last rows are read where they are."""
    N, K, G = 560003, 16384, 128
    codes, scales, _ = raw(N, K, G, False, seed=12)
    plane = pq2.pq2_w4_prepare(codes, scales, group=G)
    assert plane.numel() > 1 << 32
    x = acts(2, K, BF16, seed=13)
    y = pq2.pq2_w4_mmv(x, plane, N, G)
    rows = torch.tensor([0, 1, 262144, 300001, 559985, N - 2, N - 1], device="cuda")
    check(y[:, rows], x, dense(codes[rows], scales[rows], None, G))


def test_refusals():
    N, K, G = 8, 256, 64
    codes, scales, z = raw(N, K, G, True, seed=14)
    plane = pq2.pq2_w4_prepare(codes, scales, z, group=G)
    for bad in (lambda: pq2.pq2_w4_mmv(torch.zeros((33, K), device="cuda"), plane, N, G),
                lambda: pq2.pq2_w4_mmv(torch.zeros((1, K + 1), device="cuda"), plane, N, G),
                lambda: pq2.pq2_w4_mmv(torch.zeros((1, K), device="cuda"), plane, N, 48),
                lambda: pq2.pq2_w4_mmv(torch.zeros((1, K), device="cuda"), plane, N, G, flags=4),
                lambda: pq2.pq2_w4_mmv(torch.zeros((1, K), device="cuda"), plane[1:], N, G),
                lambda: pq2.pq2_w4_mmv(torch.zeros((0, K), device="cuda"), plane, N, G),
                lambda: pq2.pq2_w4_prepare(codes, scales, z, group=G, plane=plane[16:]),
                lambda: pq2.pq2_w4_mmv(torch.zeros((1, K), device="cuda"), plane, N + 32, G)):
        with pytest.raises(pq2.Pq2Error):
            bad()
    for bad in (lambda: pq2.pq2_w4_prepare(codes, scales, z, group=128),
                lambda: pq2.pq2_w4_mmv(torch.zeros((1, K)), plane, N, G, zeros=True),
                lambda: pq2.pq2_w4_mmv(torch.zeros((2, K), device="cuda"), plane, N, G, zeros=True,
                                       y=torch.empty((1, N), device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError):
        pq2.pq2_w4_prepare(codes.t(), scales, z, group=G)
