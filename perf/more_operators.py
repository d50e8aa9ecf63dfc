"""Measured cases of a model's attention: the key-value cache as it is written
and read back, the attention of new tokens over its pages, and the attention
over whole prompts.

A case is a dict of plain values.  ``run`` computes it with elementary torch
operations in 32 bits (``own`` false) or through the package (``own`` true);
``exact`` computes the operator's definition in 64 bits."""
import itertools
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "i8": torch.int8}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "i8": 1}


def listed():
    def kv(name, B, new, last, H, D, S, x, cache, y, lens, shape):
        return {"name": name, "op": "kv", "B": B, "new": new, "last": last, "H": H, "D": D, "S": S,
                "x": x, "cache": cache, "y": y, "lens": lens, "shape": shape}

    def dec(name, B, T, Hq, H, D, S, x, cache, lens, shape, lse=False):
        return {"name": name, "op": "dec", "B": B, "T": T, "Hq": Hq, "H": H, "D": D, "S": S, "x": x,
                "cache": cache, "lens": lens, "shape": shape, "lse": lse}

    def pre(name, B, nq, nk, Hq, H, D, x, shape, causal=True, lse=False):
        return {"name": name, "op": "pre", "B": B, "nq": nq, "nk": nk, "Hq": Hq, "H": H, "D": D,
                "x": x, "shape": shape, "causal": causal, "lse": lse}

    return [
        # one token of one sequence into an 8-bit cache: launch and latency
        kv("kv_token_1", 1, 1, 1, 8, 128, 16, "bf16", "i8", "bf16", 1024, 0),
        # a chunk of four prompts into a 16-bit cache, small heads, ragged, from 32-bit keys
        kv("kv_ragged_4", 4, 700, 2000, 3, 64, 32, "f32", "f16", "f16", 2500, 1),
        # a chunk of eight prompts into an 8-bit cache, and each prompt back for its attention
        kv("kv_chunk_8", 8, 2048, 16384, 8, 128, 64, "bf16", "i8", "bf16", 16384, 0),
        # a new token of one short conversation
        dec("dec_short_1", 1, 1, 40, 8, 128, 16, "bf16", "bf16", 1024, 0),
        # a new token of one very long context
        dec("dec_long_1", 1, 1, 40, 8, 128, 64, "bf16", "bf16", 131072, 0),
        # four speculated tokens of twelve sequences of different lengths, wide heads
        dec("dec_spec_12", 12, 4, 24, 4, 256, 32, "f16", "f16", 6000, 2, lse=True),
        # a decode batch of ragged lengths (an empty one among them) over an 8-bit cache
        dec("dec_batch_32", 32, 1, 40, 8, 128, 64, "bf16", "i8", 8192, 3, lse=True),
        # a full decode batch over a long 8-bit cache
        dec("dec_batch_64", 64, 1, 32, 8, 128, 64, "f16", "i8", 16384, 0),
        # one short prompt
        pre("pre_short_1", 1, 37, 0, 40, 8, 128, "bf16", 0),
        # packed prompts of different lengths, small heads
        pre("pre_packed_16", 16, 1024, 0, 32, 8, 64, "f16", 4, lse=True),
        # the next chunk of three long prompts, wide heads
        pre("pre_chunk_3", 3, 512, 16384, 24, 4, 256, "bf16", 5),
        # a whole long prompt
        pre("pre_long_1", 1, 8192, 0, 40, 8, 128, "bf16", 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["kv", "dec", "dec", "pre", "pre"])
    D = rng.choice([64, 128, 128, 256])
    H = rng.choice([1, 2, 3, 4, 8, 8])
    shape = rng.randrange(1, 1 << 30)
    x = rng.choice(["bf16", "f16"])
    if op == "kv":
        B = _log(rng, 1, 64)
        n = _log(rng, 1, max(1, min(16384, 100_000_000 // (B * H * D))))
        return {"op": op, "B": B, "new": max(1, n // rng.choice([1, 3, 8])), "last": n, "H": H, "D": D,
                "S": rng.choice([16, 32, 48, 64, 128, 256]), "x": rng.choice(["bf16", "f16", "f32"]),
                "cache": rng.choice(["i8", "i8", "bf16", "f16"]),
                "y": rng.choice(["bf16", "f16", "f32"]), "lens": n + rng.randrange(300), "shape": shape}
    if op == "dec":
        B = _log(rng, 1, 64)
        lens = _log(rng, 1, max(2, min(131072, 500_000_000 // (B * H * D))))
        return {"op": op, "B": B, "T": rng.choice([1, 1, 1, 2, 4, 8]),
                "Hq": H * rng.choice([1, 2, 4, 5, 6, 8, 16]), "H": H, "D": D,
                "S": rng.choice([16, 32, 48, 64, 128, 256]), "x": x,
                "cache": rng.choice(["i8", x]), "lens": lens, "shape": shape,
                "lse": rng.random() < 0.3}
    G = rng.choice([1, 2, 4, 5, 6, 8])
    B = _log(rng, 1, 16)
    total = max(B, int(math.sqrt(1.6e11 / (D * H * G))))     # rows of one square of scores
    nq = _log(rng, 1, max(1, total // B))
    chunk = rng.random() < 0.3
    return {"op": op, "B": B, "nq": nq, "nk": _log(rng, nq, max(nq + 1, total // B)) if chunk else 0,
            "Hq": H * G, "H": H, "D": D, "x": x, "shape": shape,
            "causal": rng.random() < 0.8, "lse": rng.random() < 0.3}


def _lengths(case):
    """The sequences' lengths, as plain lists: all the same (shape 0) or ragged.
    kv: (new, last, lens); dec: (lens,); pre: (nq, nk)."""
    B, rng, even = case["B"], random.Random(case["shape"]), case["shape"] == 0

    def pick(most, least=0):
        return [most if even or b == 0 else rng.randint(least, most) for b in range(B)]
    if case["op"] == "kv":
        last = pick(case["last"])
        new = [min(n, l) for n, l in zip(pick(case["new"]), last)]
        return new, last, [l + (0 if even else rng.randint(0, case["lens"] - case["last"])) for l in last]
    if case["op"] == "dec":
        return (pick(case["lens"]),)
    nq = pick(case["nq"], 1)
    # a chunk comes after what its prompt has so far; a whole prompt attends itself
    return nq, [n + b for n, b in zip(nq, pick(case["nk"] - case["nq"]))] if case["nk"] else nq


def _ints(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _sums(values):
    return _ints([0, *itertools.accumulate(values)])


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _keys(g, *shape):
    """Keys or queries: a spread of their own, and a few channels that stand out."""
    D = shape[-1]
    x = torch.randn(shape, generator=g, device="cuda")
    return x.mul_(1 + 2 * (torch.rand(D, generator=g, device="cuda") < 0.03))


def _values(g, *shape):
    """Values: channels of different means and spreads."""
    D = shape[-1]
    mean = torch.randn(D, generator=g, device="cuda") * 0.3
    return torch.randn(shape, generator=g, device="cuda").mul_(
        0.5 + torch.rand(D, generator=g, device="cuda")).add_(mean)


def _pages(case, seed, lens):
    """A cache's pages, filled, and the table of each sequence's pages (those
    behind its length are no page at all)."""
    g = _gen(seed)
    S, H, D, dt = case["S"], case["H"], case["D"], DT[case["cache"]]
    need = [-(-n // S) for n in lens]
    width, pages = max(1, max(need)), sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((case["B"], width), -1, dtype=torch.int32, device="cuda")
    behind = torch.arange(width, device="cuda")[None, :] < _ints(need)[:, None]
    table[behind] = order[:sum(need)]
    s = {"table": table}
    for name, fill in (("k", _keys), ("v", _values)):
        if dt == torch.int8:
            s[name] = torch.randint(-127, 128, (pages, H, S, D), generator=g, device="cuda",
                                    dtype=torch.int8)
            s[name + "_scales"] = torch.rand((pages, H, S), generator=g, device="cuda") * 0.02 + 0.01
        else:
            s[name] = fill(g, pages, H, S, D).to(dt)
            s[name + "_scales"] = None
    return s


def prepare(case, seed):
    """What a program has before the call: its cache with the table of pages,
    the lengths on the device, and the call's tensors."""
    g, n = _gen(seed + 1), _lengths(case)
    s = {"case": case}
    H, D = case["H"], case["D"]
    if case["op"] == "kv":
        new, last, lens = n
        s |= _pages(case, seed, lens)
        s |= {"lens": _ints(lens), "cu_new": _sums(new), "cu_last": _sums(last)}
        s["new_k"] = _keys(g, sum(new), H, D).to(DT[case["x"]])
        s["new_v"] = _values(g, sum(new), H, D).to(DT[case["x"]])
        s["out"] = [torch.empty((sum(last), H, D), dtype=DT[case["y"]], device="cuda")
                    for _ in range(2)]
        return s
    dt = DT[case["x"]]
    if case["op"] == "dec":
        s |= _pages(case, seed, n[0])
        s["lens"] = _ints(n[0])
        s["q"] = _keys(g, case["B"], case["T"], case["Hq"], D).to(dt)
    else:
        nq, nk = n
        s |= {"cu_q": _sums(nq), "cu_k": _sums(nk)}
        s["q"] = _keys(g, sum(nq), case["Hq"], D).to(dt)
        s["k"] = _keys(g, sum(nk), H, D).to(dt)
        s["v"] = _values(g, sum(nk), H, D).to(dt)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["q"].shape[:-1], device="cuda") if case["lse"] else None
    return s


def run(state):
    return {"kv": _kv, "dec": _dec, "pre": _pre}[state["case"]["op"]](state, state["case"])


def _cache(s):
    from ternary_weight_int8_gb300 import pq2
    return pq2.KVCache(s["k"], s["v"], s["k_scales"], s["v_scales"])


def _kv(s, case):
    if own:
        from ternary_weight_int8_gb300 import pq2
        cache = _cache(s)
        pq2.pq2_kv_store(s["new_k"], s["new_v"], cache, s["table"], s["lens"], cu=s["cu_new"])
        k, v = pq2.pq2_kv_load(cache, s["table"], s["lens"], cu=s["cu_last"], out=s["out"])
        return {"k": k, "v": v}
    at = _places(s, s["cu_new"], s["new_k"].shape[0])
    _write(s, case, "k", at)
    _write(s, case, "v", at)
    at = _places(s, s["cu_last"], s["out"][0].shape[0])
    return {"k": _read(s, case, "k", at), "v": _read(s, case, "v", at)}


def _write(s, case, name, at):
    page, slot = at
    x = s["new_" + name].float()
    if case["cache"] == "i8":
        top = x.abs().amax(-1)
        scale = top / torch.full_like(top, 127.0)
        x = (x / torch.where(scale > 0, scale, 1.0)[..., None]).round().clamp(-127, 127)
        s[name + "_scales"][page, :, slot] = scale
    s[name][page, :, slot] = x.to(DT[case["cache"]])


def _read(s, case, name, at):
    page, slot = at
    x = s[name][page, :, slot].float()
    if case["cache"] == "i8":
        x = x * s[name + "_scales"][page, :, slot][..., None]
    return x.to(DT[case["y"]])


def _places(s, cu, rows):
    """Page and slot of each packed row: the last rows of each sequence."""
    S = s["k"].shape[2]
    row = torch.arange(rows, device=cu.device)
    b = torch.searchsorted(cu[1:], row.int(), right=True)
    at = s["lens"][b] - cu[b + 1] + row
    return s["table"][b, at // S].long(), at % S


def _softmax(scores, keep, scale):
    """The weights of scores[..., rows, keys] and their log-sum-exp."""
    scores = scores.mul_(scale).masked_fill_(~keep, -math.inf)
    top = scores.amax(-1, keepdim=True)
    some = top > -math.inf
    e = scores.sub_(torch.where(some, top, 0.0)).exp_()
    total = e.sum(-1, keepdim=True)
    lse = (torch.log(total) + torch.where(some, top, 0.0))[..., 0]
    return e.div_(torch.where(some, total, 1.0)), lse


def _dec(s, case):
    scale = 1 / math.sqrt(case["D"])
    if own:
        from ternary_weight_int8_gb300 import pq2
        out = pq2.pq2_attn_decode(s["q"], _cache(s), s["table"], s["lens"], scale=scale,
                                  out=s["out"], lse=s["lse"])
        return {"out": out, "lse": s["lse"]} if case["lse"] else {"out": out}
    B, T, Hq, H, D = (case[x] for x in ("B", "T", "Hq", "H", "D"))
    k, v = _dense(s, case, "k"), _dense(s, case, "v")
    q = s["q"].float().view(B, T, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    at = torch.arange(k.shape[2], device=q.device)
    most = s["lens"][:, None] - T + 1 + torch.arange(T, device=q.device)          # [B][T]
    keep = (at < most[..., None]).repeat_interleave(Hq // H, 1)[:, None]
    p, lse = _softmax(q @ k.transpose(2, 3), keep, scale)
    there = (at < s["lens"][:, None])[:, None, :, None]
    o = p @ torch.where(there, v, 0.0)

    def rows(x):
        return x.view(B, H, T, Hq // H, *x.shape[3:]).transpose(1, 2).reshape(B, T, Hq, *x.shape[3:])
    out = rows(o).to(s["q"].dtype)
    return {"out": out, "lse": rows(lse).contiguous()} if case["lse"] else {"out": out}


def _dense(s, case, name):
    """Each sequence's pages in a row, [B][H][tokens][D]."""
    pages = s["table"].long().clamp(min=0)
    x = s[name][pages].float()
    if case["cache"] == "i8":
        x = x * s[name + "_scales"][pages][..., None]
    return x.transpose(1, 2).reshape(case["B"], case["H"], -1, case["D"])


def _pre(s, case):
    scale = 1 / math.sqrt(case["D"])
    if own:
        from ternary_weight_int8_gb300 import pq2
        out = pq2.pq2_attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], scale=scale,
                                   causal=case["causal"], out=s["out"], lse=s["lse"])
        return {"out": out, "lse": s["lse"]} if case["lse"] else {"out": out}
    q, k, v = (s[x].float().transpose(0, 1) for x in ("q", "k", "v"))
    H, (Hq, rows, D) = case["H"], q.shape
    i, j = (torch.arange(n, device=q.device, dtype=torch.int32) for n in (rows, k.shape[1]))
    a, b = (torch.searchsorted(s[cu][1:], n, right=True) for cu, n in (("cu_q", i), ("cu_k", j)))
    keep = a[:, None] == b[None, :]
    if case["causal"]:
        # both counted from their sequence's end
        keep &= (j - s["cu_k"][b + 1])[None, :] <= (i - s["cu_q"][a + 1])[:, None]
    p, lse = _softmax(q.reshape(H, Hq // H, rows, D) @ k[:, None].transpose(2, 3), keep, scale)
    out = (p @ v[:, None]).view(Hq, rows, D).transpose(0, 1).to(s["q"].dtype).contiguous()
    return {"out": out, "lse": lse.view(Hq, rows).t().contiguous()} if case["lse"] else {"out": out}


def work(case):
    """The bytes and operations that the operator cannot do without."""
    n, H, D = _lengths(case), case["H"], case["D"]
    if case["op"] == "kv":
        new, last = sum(n[0]), sum(n[1])
        c, side = SIZE[case["cache"]], 4 if case["cache"] == "i8" else 0
        return {"bytes": 2 * H * (new * (D * (SIZE[case["x"]] + c) + side)
                                  + last * (D * (SIZE[case["y"]] + c) + side)),
                "flops": 2 * H * D * (4 * new + last) if side else 0}
    Hq, few = case["Hq"], 4 if case["lse"] else 0
    if case["op"] == "dec":
        total, rows = sum(n[0]), case["B"] * case["T"] * Hq
        side = 4 if case["cache"] == "i8" else 0
        return {"bytes": 2 * total * H * (D * SIZE[case["cache"]] + side)
                + rows * (2 * D * SIZE[case["x"]] + few),
                "flops": 4 * D * Hq * sum(max(0, l - t) for l in n[0] for t in range(case["T"]))}
    pairs = sum(a * (b - a) + a * (a + 1) // 2 if case["causal"] else a * b for a, b in zip(*n))
    return {"bytes": 2 * SIZE[case["x"]] * D * (Hq * sum(n[0]) + H * sum(n[1])) + few * Hq * sum(n[0]),
            "flops": 4 * D * Hq * pairs}


def _attend(q, k, v, most):
    """64 bits, one sequence and one head of keys: q[rows][D], k and v[keys][D],
    row r sees its first most[r] keys -> (out, lse)."""
    out, lse = torch.zeros_like(q), torch.full(q.shape[:1], -math.inf, dtype=q.dtype, device=q.device)
    step = max(1, (1 << 27) // max(1, k.shape[0]))
    for a in range(0, q.shape[0], step):
        z = torch.einsum("rd,kd->rk", q[a:a + step], k) / math.sqrt(q.shape[1])
        z = z.masked_fill(torch.arange(k.shape[0], device=q.device) >= most[a:a + step, None], -math.inf)
        seen = most[a:a + step] > 0
        lse[a:a + step][seen] = torch.logsumexp(z[seen], 1)
        out[a:a + step][seen] = torch.einsum("rk,kd->rd", torch.softmax(z[seen], 1), v)
    return out, lse


def exact(case, seed):
    """The definition in 64 bits, sequence by sequence."""
    s, n = prepare(case, seed), _lengths(case)
    H, D = case["H"], case["D"]

    def read(name, b, first, last):
        """Positions first..last of a sequence in the cache, [tokens][H][D]."""
        S = case["S"]
        at = torch.arange(first, last, device="cuda")
        page = s["table"][b].long()[torch.div(at, S, rounding_mode="floor")]
        x = s[name][page, :, at % S].double()
        return x if case["cache"] != "i8" else x * s[name + "_scales"][page, :, at % S].double()[..., None]

    if case["op"] == "kv":
        out, row = {"k": [], "v": []}, 0
        for b, (new, last, length) in enumerate(zip(*n)):
            for name in ("k", "v"):
                x = s["new_" + name][row:row + new].double()
                if case["cache"] == "i8":
                    scale = (x.abs().amax(-1, keepdim=True) / 127).float().double()
                    x = torch.round(x / scale.where(scale > 0, 1.0)) * scale
                else:
                    x = x.to(DT[case["cache"]]).double()
                out[name] += [read(name, b, length - last, length - new), x]
            row += new
        return {name: torch.cat(parts) for name, parts in out.items()}
    Hq, G = case["Hq"], case["Hq"] // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    if case["op"] == "dec":
        for b, length in enumerate(n[0]):
            if not length:
                continue
            k, v = read("k", b, 0, length), read("v", b, 0, length)
            most = length - case["T"] + 1 + torch.arange(case["T"], device="cuda").repeat_interleave(G)
            for h in range(H):
                at = slice(h * G, h * G + G)
                o, z = _attend(s["q"][b, :, at].double().reshape(-1, D), k[:, h], v[:, h], most)
                out[b, :, at], lse[b, :, at] = o.view(-1, G, D), z.view(-1, G)
    else:
        a = c = 0
        for nq, nk in zip(*n):
            most = torch.full((nq,), nk, device="cuda")
            if case["causal"]:
                most = nk - nq + 1 + torch.arange(nq, device="cuda")
            for h in range(Hq):
                k, v = (s[x][c:c + nk, h // G].double() for x in ("k", "v"))
                out[a:a + nq, h], lse[a:a + nq, h] = _attend(s["q"][a:a + nq, h].double(), k, v, most)
            a, c = a + nq, c + nk
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}

