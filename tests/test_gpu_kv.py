"""The key-value cache as it is written (pq2_kv_store) and read back
(pq2_kv_load), against the rule in the library's own steps: s = max|x| / 127,
q = clamp(rne(x / s), +-127), both divisions IEEE fp32, so that codes, scales
and what they stand for are equal bit for bit."""
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


def quantised(x):
    """(codes, scales) of x [..., D] by the rule, step by step in fp32 on the host."""
    x = x.float().cpu()
    top = x.abs().amax(-1)
    s = (top.numpy() / torch.tensor(127.0).numpy())
    s = torch.from_numpy(s)
    q = (x / torch.where(s > 0, s, torch.ones(()))[..., None]).round().clamp(-127, 127)
    return q.to(I8).cuda(), s.cuda()


def case(B, new, past, heads, D, page, dtype, seed, spare=2):
    g = A.gen(seed)
    lens = [n + p for n, p in zip(new, past)]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((B, max(1, max(need))), -7, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    rows = sum(new)
    k, v = (torch.randn((rows, heads, D), generator=g, device="cuda") * s for s in (3.0, 0.01))
    k[::5] *= 1e4 if dtype != F16 else 1.0
    k[1::7, :, 3:] = 0
    v[2::7] = 0
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return k.to(dtype), v.to(dtype), pages, table, lens, cu


def place(table, lens, cu, page):
    """(page, slot) of every packed row."""
    pg, slot = [], []
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        pos = torch.arange(lens[b] - n, lens[b], device="cuda")
        pg.append(table[b].long()[pos // page])
        slot.append(pos % page)
    return torch.cat(pg), torch.cat(slot)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("cache_dtype", [I8, BF16, F16])
@pytest.mark.parametrize("B,new,past,heads,D,page", [
    (1, [1], [0], 1, 64, 16), (1, [1], [15], 8, 128, 16), (1, [1], [16], 3, 256, 16),
    (3, [0, 5, 0], [7, 0, 0], 2, 128, 32), (4, [1, 17, 33, 2], [0, 31, 100, 15], 5, 128, 48),
    (2, [300, 129], [3, 1000], 8, 64, 64), (33, [2] * 33, list(range(33)), 4, 256, 16),
    (40, [b % 3 for b in range(40)], [b * 7 % 50 for b in range(40)], 3, 64, 16),
    (1, [513], [0], 9, 128, 256)])
def test_store_and_load(dtype, cache_dtype, B, new, past, heads, D, page):
    k, v, pages, table, lens, cu = case(B, new, past, heads, D, page, dtype, seed=B + heads + D)
    cache = pq2.kv_cache(pages, heads, page, D, cache_dtype)
    for t in cache:
        if t is not None:
            t.view(torch.uint8).fill_(0x5A)
    before = [None if t is None else t.clone() for t in cache]
    pq2.pq2_kv_store(k, v, cache, table, ints(lens), cu=ints(cu))
    torch.cuda.synchronize()
    pg, slot = place(table, lens, cu, page)
    for i, x in enumerate((k, v)):
        want = before[i].clone()
        if cache_dtype == I8:
            q, s = quantised(x)
            want[pg, :, slot] = q
            side = before[2 + i].clone()
            side[pg, :, slot] = s
            assert torch.equal(cache[2 + i], side)
        else:
            want[pg, :, slot] = x.float().to(cache_dtype)
        assert torch.equal(cache[i].view(torch.uint8), want.view(torch.uint8))
    for out_dtype in (BF16, F16, F32):
        bufs = [torch.full((cu[-1] + 3, heads, D), float("nan"), dtype=out_dtype, device="cuda")
                for _ in range(2)]
        pq2.pq2_kv_load(cache, table, ints(lens), cu=ints(cu), out=bufs)
        torch.cuda.synchronize()
        for i, x in enumerate((k, v)):
            if cache_dtype == I8:
                q, s = quantised(x)
                want = (q.float() * s[..., None]).to(out_dtype)
            else:
                want = x.float().to(cache_dtype).float().to(out_dtype)
            assert torch.equal(bufs[i][:cu[-1]], want)
            assert bool(bufs[i][cu[-1]:].isnan().all())  # rows behind the last sequence


@pytest.mark.parametrize("layout", ["heads", "tokens", "both", "gaps"])
@pytest.mark.parametrize("dtype", [I8, BF16])
def test_whole_sequences_of_every_layout(layout, dtype):
    lens = [70, 0, 33, 128]
    cache, table, dense = A.make_cache(4, lens, 3, 32, 128, dtype, seed=5, layout=layout)
    cu = [0, 70, 70, 103, 231]
    k, v = pq2.pq2_kv_load(cache, table, ints(lens), cu=ints(cu), tokens=231, out_dtype=F32)
    for b in range(4):
        for got, want in zip((k, v), dense[b]):
            assert torch.equal(got[cu[b]:cu[b + 1]].transpose(0, 1), want.float())
    # and written back into another cache of that layout
    other, _, _ = A.make_cache(4, lens, 3, 32, 128, dtype, seed=5, layout=layout)
    for t in other[:2]:
        t.zero_()
    pq2.pq2_kv_store(k, v, other, table, ints(lens), cu=ints(cu))
    k2, v2 = pq2.pq2_kv_load(other, table, ints(lens), cu=ints(cu), tokens=231, out_dtype=F32)
    if dtype == I8:
        assert bool(((k2 - k).abs() <= k.abs().amax(-1, keepdim=True) / 127 * 0.51).all())
    else:
        assert torch.equal(k2, k) and torch.equal(v2, v)


@pytest.mark.parametrize("pad,shift", [(0, 0), (4, 0), (1, 3), (8, 8), (0, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_a_wider_projection(pad, shift, dtype):
    """k and v as columns of one projection's rows, of any alignment."""
    H, D, T = 3, 128, 37
    width = 2 * H * D + pad
    back = torch.randn((T * width + shift,), generator=A.gen(3), device="cuda").to(dtype)
    qkv = back[shift:].view(T, width)
    k, v = (qkv[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(2))
    table = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    cache = pq2.kv_cache(3, H, 16, D)
    pq2.pq2_kv_store(k, v, cache, table, ints([T]))
    got = pq2.pq2_kv_load(cache, table, ints([T]), tokens=T, out_dtype=F32)
    for x, y in zip((k, v), got):
        q, s = quantised(x)
        assert torch.equal(y, q.float() * s[..., None])


def test_even_split_and_places_outside_the_cache():
    """Without cu the rows split evenly; positions before the first, pages that
    are none and positions behind the table's width are not written and read as
    zeros."""
    H, D, page = 2, 64, 16
    table = torch.tensor([[0, 1], [2, 99], [-1, 3]], dtype=torch.int32, device="cuda")
    lens = ints([40, 20, 2])  # 40: behind the table; 20: page 99; 2: starts before 0
    k = torch.randn((12, H, D), device="cuda").bfloat16()
    cache = pq2.kv_cache(4, H, page, D, BF16)
    pq2.pq2_kv_store(k, k, cache, table, lens)
    torch.cuda.synchronize()
    assert not cache.k.any() and not cache.v.any()
    lens = ints([34, 18, 19])  # positions 30..33 (two of them), 14..17 (two), 15..18 (three)
    pq2.pq2_kv_store(k, k, cache, table, lens)
    got, _ = pq2.pq2_kv_load(cache, table, lens, tokens=12)
    keep = torch.tensor([1, 1, 0, 0, 1, 1, 0, 0, 0, 1, 1, 1], device="cuda").bool()
    assert torch.equal(got[keep], k[keep]) and not got[~keep].any()


def test_nothing_to_do():
    cache = pq2.kv_cache(2, 2, 16, 64)
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    none = torch.empty((0, 2, 64), device="cuda")
    pq2.pq2_kv_store(none, none, cache, table, ints([0]))
    pq2.pq2_kv_store(none, none, cache, table, ints([5]), cu=ints([0, 0]))
    k, v = pq2.pq2_kv_load(cache, table, ints([9]), tokens=0)
    torch.cuda.synchronize()
    assert k.shape == v.shape == (0, 2, 64) and not cache.k.any()


def test_rows_outside_the_sequences():
    """Sums that begin above 0 and end before the last row."""
    cache = pq2.kv_cache(4, 2, 16, 64, BF16)
    table = torch.tensor([[1, 3], [0, -1]], dtype=torch.int32, device="cuda")
    x = torch.randn((20, 2, 64), generator=A.gen(1), device="cuda").bfloat16()
    x[:3], x[16:] = float("nan"), float("nan")
    cu, lens = ints([3, 13, 16]), ints([20, 3])
    pq2.pq2_kv_store(x, -x, cache, table, lens, cu=cu)
    out = [torch.full((20, 2, 64), 7.0, dtype=F32, device="cuda") for _ in range(2)]
    pq2.pq2_kv_load(cache, table, lens, cu=cu, out=out)
    assert torch.equal(out[0][3:16], x[3:16].float()) and torch.equal(out[1][3:16], -x[3:16].float())
    for y in out:
        assert bool((y[:3] == 7).all()) and bool((y[16:] == 7).all())
    assert not cache.k.isnan().any() and not cache.v.isnan().any()


def test_what_is_not_finite_reads_back_as_nan():
    k = torch.ones((3, 2, 128), device="cuda")
    k[0, 0, 5], k[1, 1, 7], k[2, 0, 0] = float("inf"), float("nan"), -float("inf")
    cache = pq2.kv_cache(1, 2, 16, 128)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    pq2.pq2_kv_store(k, k, cache, table, ints([3]))
    got, _ = pq2.pq2_kv_load(cache, table, ints([3]), tokens=3, out_dtype=F32)
    bad = torch.tensor([[1, 0], [0, 1], [1, 0]], device="cuda").bool()
    assert bool(got[bad].isnan().all()) and bool((got[~bad] == 1).all())


def test_offsets_beyond_32_bits():
    """Pages whose elements lie more than 2^31 apart."""
    H, D, page = 1, 64, 16
    far = (1 << 31) // 2 + 64
    back = torch.zeros((2 * far + H * page * D,), dtype=I8, device="cuda")
    k = back.as_strided((3, H, page, D), (far, page * D, D, 1))
    vback = torch.zeros_like(back)
    v = vback.as_strided((3, H, page, D), (far, page * D, D, 1))
    cache = pq2.KVCache(k, v, *(torch.zeros((3, H, page), device="cuda") for _ in range(2)))
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    x = torch.randn((40, H, D), generator=A.gen(1), device="cuda")
    pq2.pq2_kv_store(x, -x, cache, table, ints([40]))
    got, minus = pq2.pq2_kv_load(cache, table, ints([40]), tokens=40, out_dtype=F32)
    q, s = quantised(x)
    assert torch.equal(got, q.float() * s[..., None]) and torch.equal(minus, -got)
