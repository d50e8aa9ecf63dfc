"""What a call with ``stream`` allocates belongs to that stream: torch's
allocations of the binding, recorded with the stream that is current at each,
over a library that does nothing."""
import contextlib

import pytest
import torch

from ternary_weight_int8_gb300 import pq2


class Library:
    """Functions that succeed; sizes of one KB."""
    def __getattr__(self, name):
        return (lambda *a: 1024) if name.endswith("_bytes") else (lambda *a: pq2.PQ2_OK)


class Stream:
    cuda_stream = 77


@pytest.fixture
def allocated(monkeypatch):
    """[(stream that is current, shape)] of every torch.empty."""
    now, seen, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def current(stream):
        was, now[0] = now[0], stream
        yield
        now[0] = was

    def record(*a, **k):
        t = empty(*a, **k)
        seen.append((now[0], tuple(t.shape)))
        return t
    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch, "empty", record)
    monkeypatch.setattr(pq2, "_lib", Library())
    for check in ("_on_one_device", "_on_device"):
        monkeypatch.setattr(pq2, check, lambda *a: None)
    monkeypatch.setattr(pq2, "_stream", lambda s: 0 if s is None else s.cuda_stream)
    monkeypatch.setattr(pq2, "_attn_bytes", {})
    return seen


def all_on(seen, n, stream):
    assert len(seen) == n and all(s is stream for s, _ in seen), seen
    seen.clear()


@pytest.mark.parametrize("stream", [None, Stream()])
def test_the_cache_and_the_attention(allocated, stream):
    cache = pq2.kv_cache(4, 2, 16, 64, torch.bfloat16, device="cpu")
    table, lens = torch.zeros((2, 2), dtype=torch.int32), torch.tensor([3, 5], dtype=torch.int32)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 2], dtype=torch.int32)
    allocated.clear()
    pq2.pq2_kv_load(cache, table, lens, tokens=8, stream=stream)
    all_on(allocated, 2, stream)
    pq2.pq2_attn_decode(q, cache, table, lens, stream=stream)  # output, workspace
    all_on(allocated, 2, stream)
    pq2.pq2_attn_prefill(q, k, k, cu, cu, stream=stream)
    all_on(allocated, 2, stream)
    pq2.pq2_attn_prefill(q, k, k, cu, cu, out=torch.zeros_like(q), stream=stream)
    all_on(allocated, 1, stream)


def calls():
    """Every other call that takes a stream, with what it allocates."""
    def zeros(*shape, dtype=torch.uint8):
        return torch.zeros(shape, dtype=dtype)
    x = zeros(2, 256, dtype=torch.bfloat16)
    codes, scales = zeros(8, 64), zeros(8, 2, dtype=torch.float16)
    q, sx, qsum = zeros(2, 256, dtype=torch.int8), zeros(2, 2, dtype=torch.float32), zeros(2, 2)
    q8, h = zeros(2, 512), zeros(2, 256, dtype=torch.float16)
    w, sign = zeros(256, dtype=torch.bfloat16), zeros(256, dtype=torch.int8)
    raw, side = zeros(8, 68), zeros(8, 2, dtype=torch.int32)
    return [
        (2, pq2.pq2_prepare, raw, 256), (3, pq2.pq2_quantize_act, x),
        (3, pq2.pq2_quantize_act, x, pq2.PQ2_Q_F8), (3, pq2.pq2_quantize_act, x, pq2.PQ2_Q_F16),
        (1, pq2.pq2_mmv, q, sx, qsum, codes, scales),
        (1, pq2.pq2_mmv_tc, h, sx, qsum, codes, scales), (2, pq2.pq2_linear, x, codes, scales),
        (2, pq2.linear, x, codes, scales), (3, pq2.pq2_quantize_act_grouped, x, 64),
        (1, pq2.pq2_mmv_grouped, q, sx, qsum, codes, scales, 64),
        (1, pq2.pq2_debug_group_dots_grouped, q, qsum, codes, 64), (2, pq2.pq2_ptq_prepare, raw, 256),
        (1, pq2.pq2_ptq_mmv, q, sx, qsum, codes, side, 64),
        (2, pq2.pq2_ptq_linear, x, codes, side, 64),
        (1, pq2.pq2_debug_ptq_dots, q, qsum, codes, side, 64),
        (1, pq2.pq2_mmv_gated, q, sx, qsum, codes, scales),
        (2, pq2.pq2_linear_gated, x, codes, scales),
        (5, pq2.pq2_norm_hadamard_quantize, x, w, sign, 1e-6, None, pq2.PQ2_Q_PLANES, True, True),
        (1, pq2.pq2_mm_f8, q8, sx, qsum, codes, scales), (1, pq2.pq2_mm, h, sx, qsum, codes, scales),
        (1, pq2.pq2_debug_group_dots, q, codes, pq2.PQ2_PATH_MMV_PLANES),
        (1, pq2.pq2_mm_grouped, h, sx, qsum, codes, scales, 64),
        (1, pq2.pq2_mm_f8_grouped, q8, sx, qsum, codes, scales, 64),
        (1, pq2.pq2_debug_mm_dots_grouped, h, codes, pq2.PQ2_PATH_MM, 64),
        (2, pq2.pq2_linear_grouped, x, codes, scales, 64),
        (1, pq2.pq2_w4_prepare, zeros(8, 128), scales), (1, pq2.pq2_w4_mmv, x, zeros(4096), 8),
        (4, pq2.pq2_token_logprobs, x, None, 3), (2, pq2.pq2_norm_gate_residual, x, x, w)]


@pytest.mark.parametrize("stream", [None, Stream()])
def test_every_other_call(allocated, stream):
    import inspect
    made = calls()
    takes = {f for n, f in vars(pq2).items()
             if inspect.isfunction(f) and not n.startswith("_") and n != "q_buffer"
             and "stream" in inspect.signature(f).parameters}
    assert takes == {c[1] for c in made} | {pq2.pq2_kv_store, pq2.pq2_kv_load, pq2.pq2_attn_decode,
                                            pq2.pq2_attn_prefill}
    for n, f, *args in made:
        allocated.clear()
        f(*args, stream=stream)
        all_on(allocated, n, stream)
