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
