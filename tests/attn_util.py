"""Attention in 64 bits for the tests, and the bounds of its kernels.

A kernel's weight p_j = 2^(s_j - m), m a maximum among the scores so far or at
most 8 below it, is off by
  * the score: D products and sums in fp32, |ds| <= (D + 16) 2^-23 sum_d
    |q_d k_jd| scale =: ds_j (an 8-bit cache's scale is one more rounding),
    which moves a weight and the sum of the weights by at most its size;
  * 2^x and the factors of at most a few rescalings: within 2^-20 together;
  * its rounding to 16 bits: u = finfo.eps / 2 of its value, and for fp16
    2^-25 below the normal numbers.  With an 8-bit cache it is p_j s_j / S that
    is rounded, S at most twice the largest scale: 2^-25 S |q_jd| / s-units.
The sum of n weights in fp32, in pieces that each are summed one after the
other and then joined, is within n 2^-24 of its value, and so is each output's.
Then the output is rounded to q's type."""
import math

import torch

BF16, F16, F32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def attend(q, k, v, most, scale):
    """q [rows][D], k and v [keys][D] in 64 bits, row r sees its first most[r]
    keys -> (out, lse, A, N, S, L): A = sum p|v|, N = sum |v| over what is seen,
    S the largest sum |q k| scale, L = sum exp(s - max)."""
    rows, n = q.shape[0], k.shape[0]
    seen = torch.arange(n, device=q.device)[None, :] < most[:, None]
    z = torch.where(seen, (q @ k.t()) * scale, -math.inf)
    some = seen.any(1)
    top = torch.where(some, z.amax(1) if n else torch.zeros(rows, device=q.device).double(), 0.0)
    e = torch.where(seen, torch.exp(z - top[:, None]), 0.0)
    L = e.sum(1)
    p = e / torch.where(some, L, 1.0)[:, None]
    lse = torch.where(some, top + torch.log(torch.where(some, L, 1.0)), -math.inf)
    size = torch.where(seen, (q.abs() @ k.abs().t()) * abs(scale), 0.0)
    size = size.amax(1) if n else torch.zeros(rows, device=q.device).double()
    return (p @ v, lse, p @ v.abs(), seen.double() @ v.abs(), size,
            torch.where(some, L, 1.0), seen.sum(1))


def check_rows(out, lse, ref, D, weights, smallest=None):
    """out [rows][D] and lse [rows] (or None) against attend's, `weights` the
    type that the weights are rounded to; smallest: the size of 2^-25 for an
    8-bit cache, in units of v, per column."""
    o, z, A, N, S, L, n = ref
    ds = (D + 16) * 2.0 ** -23 * S
    sums = n.double() * 2.0 ** -24 + 2.0 ** -19
    u = torch.finfo(weights).eps / 2
    tol = torch.finfo(out.dtype).eps / 2 * o.abs() * 1.01 + A * (u + 2 * ds + 2 * sums)[:, None]
    if weights == F16:
        tol = tol + 2.0 ** -25 * (N if smallest is None else smallest) / L[:, None]
    tol = tol + torch.finfo(out.dtype).tiny * torch.finfo(out.dtype).eps
    empty = n == 0
    assert bool((out[empty] == 0).all())
    worst = ((out.double() - o).abs() / tol)
    assert not worst.isnan().any(), "NaN in out"
    assert worst.numel() == 0 or float(worst.max()) <= 1, float(worst.max())
    if lse is not None:
        assert bool((lse[empty] == -math.inf).all())
        d, want = lse.double()[~empty], z[~empty]
        off = (d - want).abs() - (ds + sums)[~empty] - 2.0 ** -22 * (want.abs() + S[~empty])
        assert off.numel() == 0 or float(off.max()) <= 0, float(off.max())


def make_cache(B, lens, heads, page, D, dtype, seed, layout="heads", spare=3, width=None):
    """A paged cache filled for these lengths, everything else in it NaN (8 bits:
    NaN scales), a table with entries that are no page behind the lengths, and
    the dense keys and values [heads][len][D] of each sequence in 64 bits."""
    from ternary_weight_int8_gb300 import pq2
    g = gen(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    shapes = {"heads": (pages, heads, page, D), "tokens": (pages, page, heads, D),
              "both": (pages, 2, heads, page, D), "gaps": (pages, heads + 1, page + 3, D + 16)}
    views = []
    for i in range(2):
        if layout == "both" and i:
            raw = views[0][0]
        elif dtype == I8:
            raw = torch.full(shapes[layout], 77, dtype=I8, device="cuda")
        else:
            raw = torch.full(shapes[layout], float("nan"), dtype=dtype, device="cuda")
        view = {"heads": raw, "tokens": raw.transpose(1, 2), "both": raw[:, i] if layout == "both"
                else raw, "gaps": raw[:, :heads, :page, :D]}[layout]
        views.append((raw, view))
    k, v = views[0][1], views[1][1]
    scales = [torch.full((pages, heads, page), float("nan"), device="cuda") for _ in range(2)] \
        if dtype == I8 else [None, None]
    order = torch.randperm(pages, generator=g, device="cuda").int()
    W = max(1, max(need)) if width is None else width
    table = torch.full((B, W), 0x7FFFFFFF, dtype=torch.int32, device="cuda")
    dense, at = [], 0
    for b, n in enumerate(lens):
        mine = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = mine[:W]
        pos = torch.arange(n, device="cuda")
        pg, slot = mine.long()[pos // page], pos % page
        rows = []
        for t, s, bias in ((k, scales[0], 0.0), (v, scales[1], 0.3)):
            x = torch.randn((n, heads, D), generator=g, device="cuda") + bias
            if dtype == I8:
                c = torch.randint(-127, 128, (n, heads, D), generator=g, device="cuda")
                sc = torch.rand((n, heads), generator=g, device="cuda") * 0.02 + 0.005
                t[pg, :, slot] = c.to(I8)
                s[pg, :, slot] = sc
                x = c.double() * sc.double()[..., None]
            else:
                x = x.to(dtype)
                t[pg, :, slot] = x
            rows.append(x.double().transpose(0, 1))
        dense.append(rows)
    return pq2.KVCache(k, v, *scales), table, dense
