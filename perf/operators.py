"""Measured cases of the operators a ternary model answers with: the norms
around a block with its gate and residual scale, the output head with 4-bit
weights and group scales, and the log-probabilities of the head's logits.

A case is a dict of plain values.  ``run`` computes it with elementary torch
operations in 32 bits (``own`` false) or through the package (``own`` true);
``exact`` computes the operator's definition in 64 bits."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    def w4(name, M, N, K, G, zeros, x, y):
        return {"name": name, "op": "w4", "M": M, "N": N, "K": K, "G": G, "zeros": zeros,
                "x": x, "y": y}

    def lp(name, M, V, dtype, k, T, scale, mask):
        return {"name": name, "op": "lp", "M": M, "V": V, "x": dtype, "k": k, "T": T,
                "scale": scale, "mask": mask}

    def norm(name, M, K, dtype, post, gate, alpha):
        return {"name": name, "op": "norm", "M": M, "K": K, "x": dtype, "post": post,
                "gate": gate, "alpha": alpha}

    return [
        # one token through a small projection: launch and latency
        w4("w4_small_1", 1, 1024, 1024, 128, False, "bf16", "f32"),
        # one token through an attention projection
        w4("w4_qkv_1", 1, 10240, 5120, 128, False, "bf16", "bf16"),
        # four sequences through the wide-K projection, small groups, zero points
        w4("w4_down_4", 4, 5120, 17408, 32, True, "f16", "f16"),
        # ragged sizes, 32-bit activations
        w4("w4_odd_13", 13, 5003, 4160, 32, True, "f32", "f32"),
        # the output head, one token
        w4("w4_head_1", 1, 131072, 5120, 64, False, "bf16", "f32"),
        # the output head, a full decode batch
        w4("w4_head_32", 32, 131072, 5120, 128, True, "bf16", "f32"),
        # the sampled token of one sequence with its alternatives
        lp("lp_decode_1", 1, 131072, "f32", 8, 1, 1.0, "none"),
        # a decode batch at a temperature, twenty alternatives
        lp("lp_batch_32", 32, 131072, "bf16", 20, 1, 1.25, "none"),
        # grammar-masked logits (rows that leave few tokens, one, or none), two candidates a row
        lp("lp_masked_300", 300, 100003, "f16", 5, 2, 1.0, "rows"),
        # scoring a prompt
        lp("lp_prompt_2048", 2048, 131072, "bf16", 1, 1, 1.0, "none"),
        # the norm after a block and before the next, one token
        norm("norm_decode_1", 1, 5120, "bf16", True, "column", 1.0),
        # the same over a prompt, a gate per token
        norm("norm_prompt_4096", 4096, 5120, "bf16", True, "token", 0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w4", "w4", "lp", "lp", "norm"])
    if op == "w4":
        G = rng.choice([32, 64, 128])
        x = rng.choice(["bf16", "f16", "f32"])
        K = max(1, _log(rng, 512, 17408) // G) * G
        N = min(_log(rng, 200, 131072), 131072 * 5120 // K)
        return {"op": op, "M": _log(rng, 1, 32 if x != "f32" else 20), "N": N, "K": K, "G": G,
                "zeros": rng.random() < 0.5, "x": x, "y": rng.choice(["bf16", "f16", "f32"])}
    if op == "lp":
        V = _log(rng, 1000, 200000)
        M = min(_log(rng, 1, 2048), 2048 * 131072 // (2 * V))
        return {"op": op, "M": M, "V": V, "x": rng.choice(["bf16", "f16", "f32"]),
                "k": rng.choice([0, 1, 3, 5, 8, 20, 32]), "T": rng.choice([1, 1, 2, 4]),
                "scale": rng.choice([1.0, 1.0, 0.7, 1.25]),
                "mask": rng.choice(["none", "none", "rows"])}
    K = _log(rng, 500, 20000)
    return {"op": op, "M": min(_log(rng, 1, 4096), 4096 * 5120 // (2 * K) + 1), "K": K,
            "x": rng.choice(["bf16", "f16", "f32"]), "post": rng.random() < 0.7,
            "gate": rng.choice(["none", "column", "token"]), "alpha": rng.choice([1.0, 0.5])}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _inputs(case, seed):
    """The operator's inputs on the device, made from the seed alone."""
    g, dev = _gen(seed), "cuda"
    dt = DT[case["x"]]
    M = case["M"]
    if case["op"] == "w4":
        N, K, G = case["N"], case["K"], case["G"]
        codes = torch.randint(0, 256, (N, K // 2), generator=g, device=dev, dtype=torch.uint8)
        scales = (torch.rand((N, K // G), generator=g, device=dev) * 0.045 + 0.005).half()
        zeros = torch.randint(0, 16, (N, K // G), generator=g, device=dev, dtype=torch.uint8) \
            if case["zeros"] else None
        x = torch.randn((M, K), generator=g, device=dev)
        # outlier channels, the same in every row, as activations have
        big = torch.randperm(K, generator=g, device=dev)[:max(1, K // 100)]
        x[:, big] *= 20
        return {"codes": codes, "scales": scales, "zeros": zeros, "x": x.to(dt)}
    if case["op"] == "lp":
        V = case["V"]
        x = torch.empty((M, V), device=dev, dtype=dt)
        # a broad body and a few likely tokens per row
        x.copy_(torch.randn((M, V), generator=g, device=dev).mul_(2.5))
        likely = torch.randint(0, V, (M, 12), generator=g, device=dev)
        x.scatter_(1, likely, (torch.rand((M, 12), generator=g, device=dev) * 8 + 8).to(dt))
        if case["mask"] == "rows":
            # row r keeps about V^(r%5 / 4) tokens; every fifth row one token, and row 5 none
            share = torch.tensor([1.0 / V, V ** -0.75, V ** -0.5, V ** -0.25, 1.0], device=dev)
            keep = torch.rand((M, V), generator=g, device=dev) < \
                share[torch.arange(M, device=dev) % 5][:, None]
            keep.scatter_(1, likely[:, :1], True)
            keep[5:6] = False
            x = x.masked_fill(~keep, -math.inf)
        tokens = torch.randint(0, V, (M, case["T"]), generator=g, device=dev)
        tokens[:, 0] = likely[:, 0]
        return {"logits": x, "tokens": tokens}
    K = case["K"]
    z = (torch.randn((M, K), generator=g, device=dev) * 3).to(dt)
    h = (torch.randn((M, K), generator=g, device=dev) * 10).to(dt)
    w_pre = (1 + 0.2 * torch.randn((K,), generator=g, device=dev)).to(dt)
    w_post = (1 + 0.2 * torch.randn((K,), generator=g, device=dev)).to(dt)
    gate = None
    if case["gate"] != "none":
        rows = 1 if case["gate"] == "column" else M
        gate = torch.randn((rows, K), generator=g, device=dev).to(dt)
    return {"z": z, "h": h, "w_pre": w_pre, "w_post": w_post if case["post"] else None,
            "gate": gate}


EPS = 1e-6


def prepare(case, seed):
    """A program's state before the call: its inputs, and with the package the
    prepared weights and the output buffers that it keeps."""
    s = {"case": case, **_inputs(case, seed)}
    if not own:
        return s
    from ternary_weight_int8_gb300 import pq2
    M, dev = case["M"], "cuda"
    if case["op"] == "w4":
        s["plane"] = pq2.pq2_w4_prepare(s.pop("codes"), s.pop("scales"), s.pop("zeros"),
                                        group=case["G"])
        s["y"] = torch.empty((M, case["N"]), dtype=DT[case["y"]], device=dev)
    elif case["op"] == "lp":
        k = case["k"]
        s["out"] = (torch.empty((M, case["T"]), dtype=torch.float32, device=dev),
                    torch.empty((M,), dtype=torch.float32, device=dev),
                    torch.empty((M, k), dtype=torch.int64, device=dev),
                    torch.empty((M, k), dtype=torch.float32, device=dev))
    else:
        s["h_out"] = torch.empty_like(s["h"])
        s["n_out"] = torch.empty_like(s["h"])
    return s


def run(state):
    case = state["case"]
    op = {"w4": _w4, "lp": _lp, "norm": _norm}[case["op"]]
    return op(state, case)


def _w4(s, case):
    if own:
        from ternary_weight_int8_gb300 import pq2
        return pq2.pq2_w4_mmv(s["x"], s["plane"], case["N"], case["G"], zeros=case["zeros"],
                              y=s["y"])
    N, K, G = case["N"], case["K"], case["G"]
    c = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(N, K // G, G)
    z = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    w = (c.float() - z) * s["scales"].float()[..., None]
    return (s["x"].float() @ w.view(N, K).t()).to(DT[case["y"]])


def _lp(s, case):
    k = case["k"]
    if own:
        from ternary_weight_int8_gb300 import pq2
        lp, ent, ids, top = pq2.pq2_token_logprobs(s["logits"], s["tokens"], k,
                                                   scale=case["scale"], out=s["out"])
        return {"lp": lp, "entropy": ent, "ids": ids, "top": top}
    t = s["logits"].float() * case["scale"]
    m = t.amax(1, keepdim=True)
    some = m > -math.inf
    u = t - torch.where(some, m, 0.0)
    e = torch.exp(u)
    total = e.sum(1, keepdim=True)
    log = torch.log(total)
    ent = torch.where(some, log - torch.where(e > 0, e * u, 0.0).sum(1, keepdim=True)
                      / torch.where(some, total, 1.0), 0.0)
    lp = torch.where(some, u.gather(1, s["tokens"]) - log, -math.inf)
    # The order by value, then by index, as one whole number per element.
    bits = (s["logits"].float() + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
    order -= torch.arange(case["V"], device=t.device)
    ids = torch.topk(order, k, 1).indices
    top = torch.where(some, u.gather(1, ids) - log, -math.inf)
    return {"lp": lp, "entropy": ent[:, 0], "ids": ids, "top": top}


def _norm(s, case):
    if own:
        from ternary_weight_int8_gb300 import pq2
        h, n = pq2.pq2_norm_gate_residual(
            s["z"], s["h"], s["w_pre"], w_post=s["w_post"], gate=s["gate"],
            rows_per_gate=case["M"] if case["gate"] == "column" else 1, alpha=case["alpha"],
            eps=EPS, h_out=s["h_out"], n_out=s["n_out"])
        return {"h": h, "n": n}
    p = s["z"].float()
    if s["w_post"] is not None:
        p = p / torch.sqrt((p * p).mean(1, keepdim=True) + EPS) * s["w_post"].float()
    if s["gate"] is not None:
        p = p * s["gate"].float()
    h = s["h"].float() + case["alpha"] * p
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["w_pre"].float()
    return {"h": h.to(DT[case["x"]]), "n": n.to(DT[case["x"]])}


def work(case):
    """The bytes and operations that the operator cannot do without."""
    M = case["M"]
    if case["op"] == "w4":
        N, K = case["N"], case["K"]
        side = N * (K // case["G"]) * (2.5 if case["zeros"] else 2)
        return {"bytes": N * K / 2 + side + M * K * SIZE[case["x"]] + M * N * SIZE[case["y"]],
                "flops": 2 * M * N * K}
    if case["op"] == "lp":
        out = M * (12 * case["T"] + 4 + 12 * case["k"])
        return {"bytes": M * case["V"] * SIZE[case["x"]] + out, "flops": 5 * M * case["V"]}
    K, size = case["K"], SIZE[case["x"]]
    gate = {"none": 0, "column": K, "token": M * K}[case["gate"]]
    return {"bytes": (4 * M * K + gate + (2 if case["post"] else 1) * K) * size,
            "flops": (10 if case["post"] else 6) * M * K}


def exact(case, seed):
    """The definition in 64 bits, a few rows at a time."""
    s = _inputs(case, seed)
    M = case["M"]
    if case["op"] == "w4":
        K, G, rows = case["K"], case["G"], 8192
        x = s["x"].double()
        y = torch.empty((M, case["N"]), dtype=torch.float64, device="cuda")
        for a in range(0, case["N"], rows):
            b = min(a + rows, case["N"])
            w = torch.empty((b - a, K), dtype=torch.float64, device="cuda")
            w[:, 0::2] = (s["codes"][a:b] % 16).double()
            w[:, 1::2] = (s["codes"][a:b] // 16).double()
            zero = torch.full((b - a, K // G), 8.0, dtype=torch.float64, device="cuda") \
                if s["zeros"] is None else s["zeros"][a:b].double()
            w -= zero.repeat_interleave(G, 1)
            w *= s["scales"][a:b].double().repeat_interleave(G, 1)
            y[:, a:b] = torch.einsum("mk,nk->mn", x, w)
        return y
    if case["op"] == "lp":
        parts = [_exact_lp(s["logits"][a:a + 64], s["tokens"][a:a + 64], case)
                 for a in range(0, M, 64)]
        return {key: torch.cat([p[key] for p in parts]) for key in ("lp", "entropy", "ids", "top")}
    z, h = s["z"].double(), s["h"].double()
    if s["w_post"] is not None:
        z = z * torch.rsqrt(z.square().sum(1, keepdim=True) / case["K"] + EPS) * s["w_post"].double()
    if s["gate"] is not None:
        z = z * s["gate"].double()
    h = h + case["alpha"] * z
    n = h * torch.rsqrt(h.square().sum(1, keepdim=True) / case["K"] + EPS) * s["w_pre"].double()
    return {"h": h, "n": n}


def _exact_lp(x, tokens, case):
    t = x.double() * case["scale"]
    logp = torch.log_softmax(t, 1)
    none = torch.isneginf(t).all(1)
    logp[none] = -math.inf
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    ids = torch.sort(t, dim=1, descending=True, stable=True).indices[:, :case["k"]]
    return {"lp": logp.gather(1, tokens), "entropy": entropy, "ids": ids,
            "top": logp.gather(1, ids)}
