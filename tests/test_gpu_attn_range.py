"""The attention and the cache at the ends of their ranges (bounds in attn_util)."""
import math

import pytest
import torch

from ternary_weight_int8_gb300 import pq2
import attn_util as A

pytestmark = pytest.mark.gpu

BF16, F16, F32, I8 = A.BF16, A.F16, A.F32, A.I8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pq2.lib()
    yield
    torch.cuda.synchronize()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def table_of(pages, width):
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, :pages] = torch.arange(pages, dtype=torch.int32)
    return table


def decode_and_check(q, k, v, cache_dtype, scale=1.0, wide=(False, True)):
    """One sequence of n keys k and values v [n][H][D] (fp32) through a cache, q
    [1][T][Hq][D] over it, against 64 bits: bounds of attn_util, where over 8 bits
    the weights' unit is at most the largest exp(s_j) times value scale of a row
    or, where that is less, 2^-118 exp(m).  Weights below 2^-126 are zero."""
    n, H, D = k.shape
    T, Hq = q.shape[1:3]
    G = Hq // H
    pages = -(-n // 16)
    cache = pq2.kv_cache(pages, H, 16, D, cache_dtype)
    table = table_of(pages, pages)
    pq2.pq2_kv_store(k, v, cache, table, ints([n]))
    dense = [x.double().transpose(0, 1)
             for x in pq2.pq2_kv_load(cache, table, ints([n]), tokens=n, out_dtype=F32)]
    for w in wide:
        lse = torch.empty(q.shape[:-1], device="cuda")
        out = pq2.pq2_attn_decode(q, cache, table_of(pages, 10000 if w else pages), ints([n]),
                                  scale=scale, lse=lse)
        assert not w or pq2.lib().pq2_attn_decode_workspace_bytes(1, T, Hq, H, D, 160000)
        most = (n - T + 1 + torch.arange(T, device="cuda")).repeat_interleave(G)
        for h in sorted({0, H // 3, H - 1}):
            at = slice(h * G, h * G + G)
            rows, kk, vv = q[0, :, at].double().reshape(T * G, D), dense[0][h], dense[1][h]
            ref = A.attend(rows, kk, vv, most, scale)
            small = None
            if cache_dtype == I8:
                unit = cache.v_scales.view(pages, H, 16)[:, h].reshape(-1)[:n].double()
                seen = torch.arange(n, device="cuda")[None, :] < most[:, None]
                z = torch.where(seen, rows @ kk.t() * scale, -math.inf)
                e = torch.where(seen, torch.exp(z - z.amax(1, keepdim=True)), 0.0)
                largest = (e * unit).amax(1) + 2.0 ** -118
                small = (2 * 127 * n * largest)[:, None]
            else:
                small = ref[3]
            # what weights that are flushed to zero leave out
            small = small + 2.0 ** (25 - 117) * ref[3]
            A.check_rows(out[0, :, at].reshape(T * G, D), lse[0, :, at].reshape(T * G), ref, D,
                         F16 if cache_dtype == I8 else q.dtype, small)


def queries(T, Hq, D, dtype):
    q = torch.zeros((1, T, Hq, D), dtype=dtype, device="cuda")
    q[..., 0] = torch.tensor([1.0, 0.5, -1.0, 0.0], device="cuda").repeat(Hq // 4 + 1)[:Hq]
    return q


def keys_of(sizes, D, H=1):
    """Keys with these scores under a query of one."""
    k = torch.zeros((len(sizes), H, D), device="cuda")
    k[..., 0] = sizes.float()[:, None]
    return k


@pytest.mark.parametrize("q_dtype,cache_dtype", [(BF16, I8), (F16, I8), (BF16, BF16)])
@pytest.mark.parametrize("D,T,G", [(128, 1, 4), (64, 4, 5), (256, 4, 6), (256, 1, 32)])
@pytest.mark.parametrize("n,H", [(700, 1), (2500, 100)])
@pytest.mark.parametrize("rise", [84, 86, 100, 300, 1000])
@pytest.mark.parametrize("order", ["late", "rising", "steps"])
def test_scores_that_rise_far(q_dtype, cache_dtype, D, T, G, n, H, rise, order):
    """A row's maximum rises by more than fp32 has powers of two, at the end, with
    every key or between slices: of several warps or CTAs (one head), and of one
    warp that has seen the keys before (many)."""
    j = torch.arange(n, device="cuda")
    size = {"late": torch.where(j == n - T, float(rise), 0.0), "rising": j / n * rise,
            "steps": (j // (n // 7)) * (rise / 7)}[order]
    for spread in (1.0, 400.0):  # value scales near 0.02 and 8
        v = torch.randn((n, H, D), generator=A.gen(8), device="cuda") * spread
        decode_and_check(queries(T, G * H, D, q_dtype), keys_of(size, D, H), v, cache_dtype)


@pytest.mark.parametrize("q_dtype", [BF16, F16])
@pytest.mark.parametrize("D,Hq", [(128, 4), (64, 12), (256, 24)])
@pytest.mark.parametrize("low", [20, 60, 75, 80, 86, 100, 120])
@pytest.mark.parametrize("at,H", [(3, 1), (300, 1), (3, 90), (1400, 90)])
def test_a_value_of_zero_takes_the_softmax(q_dtype, D, Hq, low, at, H):
    """A key with a value of zero lies `low` nats above all others, which are the
    whole output; normal keys of its score come after them, or do not."""
    n = 500 if H == 1 else 2000
    size = torch.zeros(n, device="cuda")
    v = torch.randn((n, H, D), generator=A.gen(3), device="cuda")
    size[at], v[at] = low, 0
    decode_and_check(queries(1, Hq * H, D, q_dtype), keys_of(size, D, H), v, I8)
    size[n - 60:n - 20] = low
    v[n - 60:n - 20] = 50 * 127 * torch.rand(D, generator=A.gen(4), device="cuda")
    decode_and_check(queries(1, Hq * H, D, q_dtype), keys_of(size, D, H), v, I8)
    # and those before it far below
    size[:at] = -2.0 * low
    decode_and_check(queries(1, Hq * H, D, q_dtype), keys_of(size, D, H), v, I8)


@pytest.mark.parametrize("q_dtype", [BF16])
@pytest.mark.parametrize("exponent", [-136, -130, -126, -100, -40, 40, 100, 117])
@pytest.mark.parametrize("rise", [0, 50, 200, -50, -200])
def test_value_scales_at_the_ends_of_fp32(q_dtype, exponent, rise):
    """Values of this power of two, before and after normal ones; bf16 outputs hold
    them all."""
    D = 128
    for n, H in ((300, 1), (2000, 80)):
        j = torch.arange(n, device="cuda")
        v = torch.randn((n, H, D), generator=A.gen(5), device="cuda").clamp(-4, 4)
        far = v * 2.0 ** exponent
        half = torch.where(j[:, None, None] < n // 2, far, v)
        for values in (far, half, half.flip(0)):
            decode_and_check(queries(1, 4 * H, D, q_dtype), keys_of(j / n * rise, D, H), values, I8)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_codes_of_subnormal_scales(dtype, D):
    """Units whose largest magnitude is a few powers of two above the smallest
    number: s = max|x| / 127 is rounded coarsely there and |x / s| passes 127."""
    tops = torch.cat([torch.arange(1, 700), torch.arange(700, 17000, 61),
                      torch.tensor([16065, 16066, 16128, 16384])]).to(torch.int32)
    step = 1 if dtype == F32 else 1 << 16  # bf16's smallest number is 2^-133
    if dtype == BF16:
        tops = tops[:127]
    x = (torch.rand((len(tops), 2, D), generator=torch.Generator().manual_seed(D)) * 2 - 1)
    x = (x * tops[:, None, None]).round().to(torch.int32)
    x[:, 0, 5], x[:, 1, 7] = tops, -tops
    x[:, 0, 9], x[:, 1, 11] = -tops, tops
    bits = x.abs() * step  # the bits of a subnormal number are its multiple of 2^-149
    bits = torch.where(x < 0, bits - (1 << 31), bits)
    k = bits.to(torch.int32).view(F32)
    assert float(k.abs().max()) < 2.0 ** -118
    if dtype == BF16:
        assert torch.equal(k.to(BF16).float(), k)
    top = k.abs().amax(-1)
    s = torch.from_numpy(top.numpy() / torch.tensor(127.0).numpy())
    q = torch.from_numpy(k.numpy() / torch.where(s > 0, s, torch.ones(()))[..., None].numpy())
    assert dtype == BF16 or float(q.abs().max()) > 128
    q = q.round().clamp(-127, 127).to(I8)
    pages = -(-len(tops) // 16)
    cache = pq2.kv_cache(pages, 2, 16, D)
    pq2.pq2_kv_store(k.to(dtype).cuda(), -k.to(dtype).cuda(), cache, table_of(pages, pages),
                     ints([len(tops)]))
    for t, scales, want in ((cache.k, cache.k_scales, q), (cache.v, cache.v_scales, -q)):
        got = t.transpose(1, 2).reshape(-1, 2, D)[:len(tops)].cpu()
        assert torch.equal(scales.transpose(1, 2).reshape(-1, 2)[:len(tops)].cpu(), s)
        assert torch.equal(got, want)


def sums(x):
    return torch.tensor([0, *x], dtype=torch.int32, device="cuda").cumsum(0).int()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,nk", [(300, 300), (60, 9000)])
def test_infinities_and_nan_seen_and_not(dtype, D, nq, nk):
    """Columns with an infinity, with both, with NaN, and with one that only later
    rows see; the key of the first has no weight that 16 bits could hold."""
    g = A.gen(D + nq)
    q = torch.randn((nq, 4, D), generator=g, device="cuda").to(dtype)
    k = torch.randn((nk, 2, D), generator=g, device="cuda").to(dtype)
    v = torch.randn((nk, 2, D), generator=g, device="cuda").to(dtype)
    q[..., 0], k[..., 0] = 8.0, 0.0
    k[5, :, 0] = -8.0 * D ** 0.5  # 64 nats below the others
    late = nk - nq + 40
    clean = v.clone()
    clean[:, :, [3, 5, 7, 9]] = 0
    v[5, :, 3], v[5, :, 5], v[8, :, 5] = float("inf"), float("inf"), -float("inf")
    v[9, :, 7], v[late, :, 9] = float("nan"), -float("inf")
    cu_q, cu_k = sums([nq]), sums([nk])
    t = torch.arange(nq, device="cuda")
    for causal in (True, False):
        out = pq2.pq2_attn_prefill(q, k, v, cu_q, cu_k, causal=causal)
        most = nk - nq + 1 + t if causal else torch.full((nq,), nk, device="cuda")
        inf = float("inf")
        for h in range(4):
            seen = clean[:, h // 2].double()
            seen[:, [3, 5, 7, 9]] = torch.where(torch.isfinite(v[:, h // 2, [3, 5, 7, 9]]),
                                                v[:, h // 2, [3, 5, 7, 9]], 0.0).double()
            ref = A.attend(q[:, h].double(), k[:, h // 2].double(), seen, most, D ** -0.5)
            # rows that do not see what is not finite, and all other columns
            fine = torch.ones((nq, D), dtype=torch.bool, device="cuda")
            fine[:, 3], fine[:, 5], fine[:, 7] = most <= 5, most <= 5, most <= 9
            fine[:, 9] = most <= late
            got = torch.where(fine, out[:, h], torch.zeros_like(out[:, h]))
            want = (torch.where(fine, ref[0], 0.0), ref[1],
                    *(torch.where(fine, x, 0.0) for x in ref[2:4]), *ref[4:])
            A.check_rows(got, None, want, D, dtype)
            assert bool((out[most > 5, h, 3] == inf).all())
            assert bool((out[(most > 5) & (most <= 8), h, 5] == inf).all())
            assert bool(out[most > 8, h, 5].isnan().all())
            assert bool(out[most > 9, h, 7].isnan().all())
            assert bool((out[most > late, h, 9] == -inf).all())


def test_a_nan_costs_little():
    """A prompt whose first values are NaN takes no more than 30 times its time
    without (each row looks for what it sees, which ends with the first)."""
    n = 4096
    q = torch.randn((n, 8, 128), generator=A.gen(1), device="cuda").bfloat16()
    k, v = (torch.randn((n, 2, 128), generator=A.gen(s), device="cuda").bfloat16() for s in (2, 3))
    bad, out, cu = v.clone(), torch.empty_like(q), sums([n])
    bad[0] = float("nan")
    took = []
    for values in (v, bad, v, bad):
        best = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            pq2.pq2_attn_prefill(q, k, values, cu, out=out)
            b.record()
            torch.cuda.synchronize()
            best.append(a.elapsed_time(b))
        took.append(min(best))
    assert bool(out.isnan().all())
    assert took[3] <= 30 * took[2], took


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,H", [(60, 2), (3000, 2), (900, 60)])
@pytest.mark.parametrize("G", [2, 4, 6, 8, 17])
def test_decode_of_infinities_and_nan_seen_and_not(dtype, D, n, H, G):
    """Four new tokens; the newest position's values, which only the last row sees,
    and some that all rows see are not finite.  From one block of rows a warp to
    several warps a slice and several items a head."""
    T = 4
    g = A.gen(D + n)
    q = torch.randn((1, T, G * H, D), generator=g, device="cuda").to(dtype)
    k, v = (torch.randn((n, H, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    q[..., 0], k[..., 0] = 8.0, 0.0
    k[5, :, 0] = -8.0 * D ** 0.5  # 64 nats below the others
    inf = float("inf")
    v[5, :, 3], v[5, :, 5], v[8, :, 5], v[9, :, 7] = inf, inf, -inf, inf - inf
    v[n - 1, :, 9], v[n - 1, :, 20:30] = inf - inf, -inf
    pages = -(-n // 16)
    cache = pq2.kv_cache(pages, H, 16, D, dtype)
    pq2.pq2_kv_store(k, v, cache, table_of(pages, pages), ints([n]))
    lse = torch.empty(q.shape[:-1], device="cuda")
    out = pq2.pq2_attn_decode(q, cache, table_of(pages, pages), ints([n]), lse=lse)
    odd = [3, 5, 7, 9, *range(20, 30)]
    clean = torch.where(v.isfinite(), v, 0).double()
    most = n - T + 1 + torch.arange(T, device="cuda").repeat_interleave(G)
    for h in sorted({0, H // 2, H - 1}):
        at = slice(h * G, h * G + G)
        ref = A.attend(q[0, :, at].double().reshape(T * G, D), k[:, h].double(), clean[:, h], most,
                       D ** -0.5)
        o, z = out[0, :, at].reshape(T * G, D), lse[0, :, at].reshape(T * G)
        A.check_rows(o[:, 30:], z, (ref[0][:, 30:], ref[1], *(x[:, 30:] for x in ref[2:4]), *ref[4:]),
                     D, dtype)
        before = o[:G * (T - 1)]
        A.check_rows(before[:, [9, *range(20, 30)]], None,
                     tuple(x[:G * (T - 1), [9, *range(20, 30)]] if x.dim() == 2
                           else x[:G * (T - 1)] for x in ref), D, dtype)
        assert not bool(before[:, 3].isfinite().any()) and bool(o[:, [5, 7]].isnan().all())
        assert not bool(o[G * (T - 1):, odd].isfinite().any())


def test_a_nan_costs_little_in_the_decode():
    """Values of the first or of the newest position that are NaN, two new tokens:
    no more than 5 times the time without."""
    n, H = 60000, 8
    cache = pq2.kv_cache(n // 16, H, 16, 128, BF16)
    for t in cache[:2]:
        t.normal_(generator=A.gen(1))
    table = torch.arange(n // 16, dtype=torch.int32, device="cuda")[None]
    q = torch.randn((1, 2, H, 128), generator=A.gen(2), device="cuda").bfloat16()
    lens, out, took = ints([n]), torch.empty_like(q), []
    for bad in (None, (n // 16 - 1, 15), (0, 0)):
        if bad:
            cache.v[bad[0], :, bad[1]] = float("nan")
        best = []
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            pq2.pq2_attn_decode(q, cache, table, lens, out=out)
            b.record()
            torch.cuda.synchronize()
            best.append(a.elapsed_time(b))
        took.append(min(best))
        assert bool(out[:, 0].isnan().all()) == (bad == (0, 0))
        assert bool(out[:, 1].isnan().all()) == (bad is not None)
    assert max(took[1:]) <= 5 * took[0], took


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sign", [1, -1])
def test_prefill_of_scores_in_the_billions(dtype, D, sign):
    """Scales to 1e6 of products from one to some thousands, each exact: a
    sequence of one key gives its value, two of unequal scores the larger one's,
    two of equal scores their mean."""
    products = torch.cat([torch.arange(1, 400), torch.arange(400, 6000, 37)]).tolist()
    n = len(products)
    q = torch.zeros((n, 2, D), dtype=dtype, device="cuda")
    k = torch.zeros((n, 1, D), dtype=dtype, device="cuda")
    # a * 64 + b, both exact in 8 bits
    p = torch.tensor(products, device="cuda")
    q[:, :, 0], q[:, :, 1] = 64.0, 1.0
    k[:, 0, 0], k[:, 0, 1] = (p // 64).to(dtype), (p % 64).to(dtype)
    k *= sign
    v = torch.randn((n, 1, D), generator=A.gen(2), device="cuda").to(dtype)
    lse = torch.empty((n, 2), device="cuda")
    out = pq2.pq2_attn_prefill(q, k, v, sums([1] * n), scale=1e6 * sign, lse=lse)
    tol = torch.finfo(dtype).eps * v.float().abs() + 2.0 ** -20
    assert bool(((out.float() - v.float()).abs() <= tol).all())
    want = p.double()[:, None] * 1e6
    assert bool(((lse.double() - want).abs() <= 2.0 ** -21 * want).all())
    # pairs: (products[0], [1]), ...; rows see both, or the first alone
    pairs = sums([2] * (n // 2))
    for causal in (True, False):
        out = pq2.pq2_attn_prefill(q, k, v, pairs, scale=1e6 * sign, causal=causal)
        for i in range(2):
            mine = v[1:n // 2 * 2:2] if i or not causal else v[0:n // 2 * 2:2]
            tol = torch.finfo(dtype).eps * mine.float().abs() + 2.0 ** -20
            assert bool(((out[i:n // 2 * 2:2].float() - mine.float()).abs() <= tol).all())
    k[1::2] = k[0:n // 2 * 2:2]
    out = pq2.pq2_attn_prefill(q, k, v, pairs, scale=1e6 * sign, causal=False)
    a, b = v[0:n // 2 * 2:2].float(), v[1:n // 2 * 2:2].float()
    tol = torch.finfo(dtype).eps * (a.abs() + b.abs()) + 2.0 ** -20
    for i in range(2):
        assert bool(((out[i:n // 2 * 2:2].float() - (a + b) / 2).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("nq,nk", [(40, 9000), (300, 300), (700, 700)])
@pytest.mark.parametrize("order", ["rising", "falling", "steps"])
def test_prefill_of_many_keys_in_the_billions(dtype, D, nq, nk, order):
    """Maxima in the billions that rise or fall over the tiles and the parts: every
    row's output is the mean of the values of its largest scores."""
    j = torch.arange(nk, device="cuda")
    p = {"rising": 500 + j // 5, "falling": 2500 - j // 5, "steps": 1000 + (j // 190) * 3}[order]
    p = p.clamp(max=8000)
    q = torch.zeros((nq, 2, D), dtype=dtype, device="cuda")
    k = torch.zeros((nk, 1, D), dtype=dtype, device="cuda")
    q[:, :, 0], q[:, :, 1] = 64.0, 1.0
    k[:, 0, 0], k[:, 0, 1] = (p // 64).to(dtype), (p % 64).to(dtype)
    v = torch.randn((nk, 1, D), generator=A.gen(2), device="cuda").to(dtype)
    assert nk < 9000 or pq2.lib().pq2_attn_prefill_workspace_bytes(1, nq, nk, 2, 1, D)
    for causal in (True, False):
        out = pq2.pq2_attn_prefill(q, k, v, sums([nq]), sums([nk]), scale=1e6, causal=causal)
        most = nk - nq + 1 + torch.arange(nq, device="cuda") if causal else \
            torch.full((nq,), nk, device="cuda")
        seen = j[None, :] < most[:, None]
        top = torch.where(seen, p[None, :], -1).amax(1)
        w = (seen & (p[None, :] == top[:, None])).double()
        w /= w.sum(1, keepdim=True)
        want, size = w @ v[:, 0].double(), w @ v[:, 0].double().abs()
        # equal weights are powers of two of each other exactly; sums and out's rounding
        tol = torch.finfo(dtype).eps * size + 2.0 ** -18 * size.amax()
        assert bool(((out.double() - want[:, None]).abs() <= tol[:, None]).all())


@pytest.mark.parametrize("cache_dtype", [BF16, F16, I8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,H", [(700, 1), (2500, 60)])
@pytest.mark.parametrize("order", ["rising", "falling", "steps"])
def test_decode_of_scores_in_the_billions(cache_dtype, D, n, H, order):
    """A scale of 1e6 and products to some thousands, each exact: the output is the
    mean of the values of the largest score, whatever their scales are."""
    j = torch.arange(n, device="cuda")
    p = {"rising": 500 + j // 5, "falling": 2500 - j // 5, "steps": 1000 + (j // 190) * 3}[order]
    k = torch.zeros((n, H, D), device="cuda")
    k[..., 0], k[..., 1] = (p // 64).float()[:, None], (p % 64).float()[:, None]
    q = torch.zeros((1, 2 * H, D), dtype=F16 if cache_dtype == F16 else BF16, device="cuda")
    q[..., 0], q[..., 1] = 64.0, 1.0
    pages = -(-n // 16)
    cache = pq2.kv_cache(pages, H, 16, D, cache_dtype)
    v = torch.randn((n, H, D), generator=A.gen(2), device="cuda")
    v *= 2.0 ** torch.randint(-12, 8, (n, H, 1), generator=A.gen(3), device="cuda")
    pq2.pq2_kv_store(k, v, cache, table_of(pages, pages), ints([n]))
    if cache_dtype == I8:  # the keys as they are, with scales of one
        cache.k[:] = torch.cat([k, k.new_zeros(pages * 16 - n, H, D)]).to(I8) \
            .view(pages, 16, H, D).transpose(1, 2)
        cache.k_scales.fill_(1.0)
    _, v = pq2.pq2_kv_load(cache, table_of(pages, pages), ints([n]), tokens=n, out_dtype=F32)
    for m in (n, n - 1, 5 * (n // 10) + 3):
        top = p[:m] == p[:m].max()
        want = v[:m][top].double().mean(0).repeat_interleave(2, 0)
        size = v[:m][top].double().abs().amax(0).repeat_interleave(2, 0)
        # 16 bits: weights of exactly one.  8 bits: weight times scale as fp16, 2^-11
        # of it and 2^-24 of the largest scale's; then out's rounding.
        unit = v[:m].abs().amax(2).amax(0).double().repeat_interleave(2, 0)[:, None]
        tol = torch.finfo(q.dtype).eps * want.abs() + 2.0 ** -18 * size + 2.0 ** -24
        if cache_dtype == I8:
            tol = tol + 2.0 ** -11 * size + 2.0 ** -24 * unit
        for width in (pages, 10000):
            out = pq2.pq2_attn_decode(q, cache, table_of(pages, width), ints([m]), scale=1e6)
            assert bool(((out[0].double() - want).abs() <= tol).all())


def test_the_most_rows_of_a_key_head():
    """64 new tokens of 256 query heads a key head, and a few."""
    for n, T, D in ((100, 64, 64), (900, 64, 128), (40, 63, 256)):
        q = torch.randn((1, T, 256, D), generator=A.gen(n), device="cuda").to(BF16)
        k, v = (torch.randn((n, 1, D), generator=A.gen(n + s), device="cuda").to(BF16)
                for s in (1, 2))
        for cache_dtype in (BF16, I8):
            decode_and_check(q, k.float(), v.float(), cache_dtype, scale=D ** -0.5)


def test_the_most_sequences():
    """65536 of one or two tokens, or none, in the decode and the prefill."""
    B, D = 65536, 64
    lens = torch.arange(B, device="cuda").int() * 7 % 3
    k, v = (torch.randn((B * 2, 1, D), generator=A.gen(s), device="cuda").to(BF16) for s in (1, 2))
    q = torch.randn((B, 2, D), generator=A.gen(3), device="cuda").to(BF16)
    cache = pq2.kv_cache(B, 1, 16, D, BF16)
    table = torch.randperm(B, generator=A.gen(4), device="cuda").int()[:, None]
    two = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    pq2.pq2_kv_store(k, v, cache, table, two)
    out = pq2.pq2_attn_decode(q, cache, table, lens)
    kk, vv = (x.view(B, 2, D).double() for x in (k, v))
    z = torch.einsum("bhd,bjd->bhj", q.double(), kk) * D ** -0.5
    seen = torch.arange(2, device="cuda") < lens[:, None]
    z = z.masked_fill(~seen[:, None], -math.inf)
    p = torch.nan_to_num(torch.softmax(z, 2))
    want = torch.einsum("bhj,bjd->bhd", p, vv)
    tol = 2.0 ** -7 * torch.einsum("bhj,bjd->bhd", p, vv.abs()) + 2.0 ** -20
    assert bool(((out.double() - want).abs() <= tol).all())
    assert not bool(out[lens == 0].any())
    cu_q = torch.arange(B + 1, device="cuda").int()
    cu_k = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).int()
    at = seen.flatten()
    out = pq2.pq2_attn_prefill(q, k[at], v[at], cu_q, cu_k)
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("n", [1 << 22, (1 << 24) - 5])
def test_millions_of_keys(n):
    """One sequence of 4 and of 16 million positions, in the prefill and the decode."""
    D = 64
    q = torch.randn((1, 2, D), generator=A.gen(3), device="cuda").to(BF16)
    k, v = (torch.randn((n, 1, D), generator=A.gen(s), device="cuda", dtype=BF16) for s in (1, 2))
    v[::2] += 1.0
    z = torch.cat([q[0].double() @ x[:, 0].double().t() for x in k.split(1 << 20)], 1) * D ** -0.5
    p = torch.softmax(z, 1)
    want = sum(w @ x[:, 0].double() for w, x in zip(p.split(1 << 20, 1), v.split(1 << 20)))
    # The sums of n weights and values of about one, in fp32 pieces: 2^-24 sqrt(n) of
    # them each at the most likely, n 2^-24 at the very most; rounding of weights and out.
    tol = 2.0 ** -6 * want.abs() + 2.0 ** -8
    lse = torch.empty((1, 2), device="cuda")
    out = pq2.pq2_attn_prefill(q, k, v, sums([1]), sums([n]), lse=lse)
    assert bool(((out[0].double() - want).abs() <= tol).all())
    assert float((lse[0].double() - torch.logsumexp(z, 1)).abs().max()) <= 1e-3
    pages = -(-n // 16)
    cache = pq2.kv_cache(pages, 1, 16, D, BF16)
    pq2.pq2_kv_store(k, v, cache, table_of(pages, pages), ints([n]))
    out = pq2.pq2_attn_decode(q, cache, table_of(pages, pages), ints([n]), lse=lse)
    assert bool(((out[0].double() - want).abs() <= tol).all())
    assert float((lse[0].double() - torch.logsumexp(z, 1)).abs().max()) <= 1e-3


@pytest.mark.parametrize("nk", [200, 9000])
@pytest.mark.parametrize("scale", [0.1, 1e6])
def test_a_nan_key_beside_an_infinite_value(nk, scale):
    """Rows that see a key of NaN are NaN in every column, also where a value that they
    see is infinite, and with scores of any size."""
    nq = 50
    q, k, v = (torch.randn((n, 2, 128), generator=A.gen(n), device="cuda").to(BF16)
               for n in (nq, nk, nk + 1))
    v = v[:nk]
    q[..., 0], k[..., 0] = 30.0, 30.0
    v[2, :, 7], k[nk - nq + 20] = float("inf"), float("nan")
    lse = torch.empty((nq, 2), device="cuda")
    out = pq2.pq2_attn_prefill(q, k, v, sums([nq]), sums([nk]), scale=scale, lse=lse)
    assert bool(out[20:].isnan().all()) and bool(lse[20:].isnan().all())
    assert bool((out[:20, :, 7] == float("inf")).all()) and bool(lse[:20].isfinite().all())
    out[:20, :, 7] = 0
    assert bool(out[:20].isfinite().all())
