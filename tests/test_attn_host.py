"""What the key-value cache and the attention refuse, on the host: the C ABI
with addresses that are never followed, and the Python calls with host tensors
(the checks look at shapes, strides and types only)."""
import ctypes
import os

import pytest
import torch

from ternary_weight_int8_gb300 import build, pq2

A = 1 << 20   # a 16-byte aligned fake address
NULL, SHAPE, ALIGN, DTYPE = (pq2.PQ2_ERR_NULL, pq2.PQ2_ERR_SHAPE, pq2.PQ2_ERR_ALIGN,
                             pq2.PQ2_ERR_DTYPE)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(pq2.LIB_PATH):
        build.build()
    return pq2.lib()


def refused(f, ok, *changes):
    for idx, val, err in changes:
        bad = list(ok)
        bad[idx] = val
        assert f(*bad) == err, (idx, val)


def c_cache(**change):
    c = dict(k=A, v=A, k_scales=A, v_scales=A, dtype=pq2.PQ2_I8, pages=10, heads=2, page_size=16,
             dim=128, page_stride=4096, head_stride=2048, token_stride=128)
    return pq2.CKvCache(**(c | change))


CACHES = [(dict(k=None), NULL), (dict(v=None), NULL), (dict(k_scales=None), NULL),
          (dict(v_scales=None), NULL), (dict(dtype=pq2.PQ2_F32), DTYPE), (dict(dtype=9), DTYPE),
          (dict(pages=0), SHAPE), (dict(heads=0), SHAPE), (dict(heads=65537), SHAPE),
          (dict(page_size=0), SHAPE), (dict(page_size=24), SHAPE),
          (dict(page_size=(1 << 20) + 16), SHAPE), (dict(dim=96), SHAPE),
          (dict(page_stride=-16), SHAPE), (dict(token_stride=1 << 40), SHAPE),
          (dict(token_stride=136), ALIGN), (dict(head_stride=8), ALIGN), (dict(k=A + 8), ALIGN),
          (dict(v_scales=A + 4), ALIGN),
          (dict(dtype=pq2.PQ2_F16, k_scales=None, v_scales=None, token_stride=132), ALIGN)]


def test_the_cache_s_layout():
    cache = pq2.kv_cache(7, 3, 16, 64, device="cpu")
    packed, heads, dim = pq2._c_cache(cache)
    c = pq2.CKvCache.from_buffer_copy(packed)
    assert len(packed) == ctypes.sizeof(pq2.CKvCache) and (heads, dim) == (3, 64)
    assert (c.k, c.v, c.k_scales, c.v_scales) == tuple(t.data_ptr() for t in cache)
    assert (c.dtype, c.pages, c.heads, c.page_size, c.dim) == (pq2.PQ2_I8, 7, 3, 16, 64)
    assert (c.page_stride, c.head_stride, c.token_stride) == cache.k.stride()[:3]


def test_caches(L):
    decode = lambda c: L.pq2_attn_decode(  # noqa: E731
        A, pq2.PQ2_BF16, 512, 512, 128, 1, 1, 4, c, A, 4, 4, A, 1.0, A, None, A, 1 << 40, None, None)
    store = lambda c: L.pq2_kv_store(  # noqa: E731
        A, 256, 128, A, 256, 128, pq2.PQ2_BF16, 4, c, A, 4, 4, None, A, 2, None)
    load = lambda c: L.pq2_kv_load(  # noqa: E731
        c, A, 4, 4, None, A, 2, A, A, pq2.PQ2_BF16, 4, None)
    for call in (store, load, decode):
        assert call(None) == NULL
        for change, err in CACHES:
            c = c_cache(**change)
            want = DTYPE if call is decode and change.get("dtype") == pq2.PQ2_F32 else err
            assert call(ctypes.addressof(c)) == want, change
    other = c_cache(dtype=pq2.PQ2_F16, token_stride=128)
    assert decode(ctypes.addressof(other)) == DTYPE  # not q's type


def test_store_and_load_refusals(L):
    c = c_cache()
    a = ctypes.addressof(c)
    ok = [A, 256, 128, A, 256, 128, pq2.PQ2_BF16, 4, a, A, 4, 4, A, A, 2, None]
    refused(L.pq2_kv_store, ok, (0, None, NULL), (3, None, NULL), (9, None, NULL),
            (13, None, NULL), (6, 3, DTYPE), (7, -1, SHAPE), (7, (1 << 24) + 1, SHAPE),
            (1, -1, SHAPE), (5, 1 << 39, SHAPE), (10, 3, SHAPE), (11, 0, SHAPE), (14, 0, SHAPE),
            (0, A + 1, ALIGN), (9, A + 2, ALIGN), (12, A + 1, ALIGN), (13, A + 2, ALIGN))
    uneven = list(ok)
    uneven[7], uneven[12] = 5, None
    assert L.pq2_kv_store(*uneven) == SHAPE
    ok = [a, A, 4, 4, A, A, 2, A, A, pq2.PQ2_F32, 4, None]
    refused(L.pq2_kv_load, ok, (1, None, NULL), (5, None, NULL), (7, None, NULL), (8, None, NULL),
            (9, 3, DTYPE), (10, -1, SHAPE), (6, 0, SHAPE), (2, 3, SHAPE), (7, A + 8, ALIGN),
            (8, A + 4, ALIGN), (5, A + 1, ALIGN))


def test_decode_refusals(L):
    c = c_cache()
    ok = [A, pq2.PQ2_BF16, 512, 512, 128, 9, 1, 4, ctypes.addressof(c), A, 10000, 10000, A, 1.0, A, A, A,
          1 << 40, A, None]
    refused(L.pq2_attn_decode, ok, (0, None, NULL), (9, None, NULL), (12, None, NULL),
            (14, None, NULL), (16, None, NULL), (1, pq2.PQ2_F32, DTYPE), (1, 7, DTYPE),
            (5, 0, SHAPE), (5, 65537, SHAPE), (6, 0, SHAPE), (6, 65, SHAPE), (7, 3, SHAPE),
            (7, 1024, SHAPE), (7, 0, SHAPE), (13, float("inf"), SHAPE), (13, 2e6, SHAPE), (13, float("nan"), SHAPE),
            (2, -2, SHAPE), (4, 127, ALIGN), (10, 3, SHAPE), (11, 0, SHAPE), (17, 0, SHAPE),
            (0, A + 2, ALIGN), (14, A + 8, ALIGN), (15, A + 2, ALIGN), (16, A + 8, ALIGN),
            (18, A + 1, ALIGN))
    f = L.pq2_attn_decode_workspace_bytes
    for none in ((1, 1, 4, 2, 128, 4096), (16, 1, 8, 1, 128, 4096), (1, 5, 320, 8, 64, 16)):
        assert f(*none) == 0
    for some in ((1, 1, 4, 2, 128, 1 << 17), (300, 1, 8, 2, 128, 256), (64, 1, 32, 8, 64, 16384), (2, 8, 64, 8, 256, 40000)):
        assert f(*some) > 0
    for bad in ((0, 1, 4, 2, 128, 1 << 20), (1, 0, 4, 2, 128, 1 << 20), (1, 1, 3, 2, 128, 1 << 20),
                (1, 1, 4, 2, 80, 1 << 20), (1, 1, 514, 2, 64, 1 << 20), (99, 1, 4, 2, 128, -1)):
        assert f(*bad) == 0


def test_prefill_refusals(L):
    ok = [A, 512, 128, A, 256, 128, A, 256, 128, pq2.PQ2_F16, 10, 10, 4, 2, 128, A, A, 2, 1.0, 1, A,
          A, A, 1 << 40, A, None]
    refused(L.pq2_attn_prefill, ok, (0, None, NULL), (3, None, NULL), (6, None, NULL),
            (15, None, NULL), (16, None, NULL), (20, None, NULL), (9, pq2.PQ2_F32, DTYPE),
            (10, 0, SHAPE), (11, -1, SHAPE), (10, (1 << 24) + 1, SHAPE), (12, 5, SHAPE),
            (12, 258, SHAPE), (13, 0, SHAPE), (14, 32, SHAPE), (17, 0, SHAPE),
            (18, float("nan"), SHAPE), (18, -2e6, SHAPE), (1, -8, SHAPE), (5, 1 << 39, SHAPE), (1, 508, ALIGN),
            (8, 4, ALIGN), (0, A + 8, ALIGN), (3, A + 2, ALIGN), (20, A + 8, ALIGN),
            (21, A + 1, ALIGN), (15, A + 2, ALIGN))
    f = L.pq2_attn_prefill_workspace_bytes
    assert f(1, 8192, 8192, 40, 8, 128) == 0 and f(1, 64, 16000, 40, 8, 128) > 0
    parts = list(ok)
    parts[10], parts[11], parts[22] = 64, 16000, None
    assert L.pq2_attn_prefill(*parts) == NULL
    parts[22], parts[23] = A, 64
    assert L.pq2_attn_prefill(*parts) == SHAPE
    for bad in ((0, 1, 1, 4, 2, 128), (1, 0, 1, 4, 2, 128), (1, 1, -1, 4, 2, 128),
                (1, 1, 1, 3, 2, 128), (1, 1, 1, 4, 2, 96)):
        assert f(*bad) == 0


def tensors(dtype=torch.bfloat16):
    cache = pq2.kv_cache(4, 2, 16, 64, dtype, device="cpu")
    table = torch.zeros((2, 2), dtype=torch.int32)
    lens = torch.tensor([3, 5], dtype=torch.int32)
    return cache, table, lens


def test_python_refusals():
    cache, table, lens = tensors()
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 1, 4], dtype=torch.int32)
    store = lambda k=k, v=k, c=cache, t=table, n=lens, **kw: pq2.pq2_kv_store(  # noqa: E731
        k, v, c, t, n, **kw)
    decode = lambda q=q, c=cache, t=table, n=lens, **kw: pq2.pq2_attn_decode(  # noqa: E731
        q, c, t, n, **kw)
    prefill = lambda q=k, k=k, v=k, cu=cu, **kw: pq2.pq2_attn_prefill(q, k, v, cu, **kw)  # noqa: E731
    load = lambda c=cache, t=table, n=lens, **kw: pq2.pq2_kv_load(c, t, n, **kw)  # noqa: E731
    if not os.path.exists(pq2.LIB_PATH):
        build.build()
    eight = pq2.kv_cache(4, 2, 16, 64, device="cpu")
    bad_caches = [cache._replace(v=cache.v[:, :1]), cache._replace(k=cache.k.float()),
                  cache._replace(k=cache.k[..., ::2], v=cache.v[..., ::2]),
                  cache._replace(k=cache.k.transpose(1, 2).contiguous().transpose(1, 2)),
                  cache._replace(k_scales=eight.k_scales, v_scales=eight.v_scales),
                  eight._replace(k_scales=None, v_scales=None), eight._replace(v_scales=None),
                  eight._replace(k_scales=eight.k_scales.half()),
                  eight._replace(k_scales=eight.k_scales[:, :1])]
    for call in (store, decode, lambda c: load(c, tokens=2)):
        for bad in bad_caches:
            with pytest.raises(ValueError):
                call(c=bad)
        for bad in (table.long(), table[0], table.t().contiguous().t()):
            with pytest.raises(ValueError):
                call(**({"t": bad}), **({"c": cache}))if call in (store, decode) else \
                    load(t=bad, tokens=2)
    for call in (lambda: store(k=k[:, :1]), lambda: store(k=k[..., :32]), lambda: store(k=k.int()),
                 lambda: store(v=k.float()), lambda: store(n=lens.long()),
                 lambda: store(n=lens[:1]), lambda: store(cu=cu[:2]), lambda: store(cu=cu.long()),
                 lambda: store(k=torch.zeros((4, 2, 128), dtype=torch.bfloat16)[..., ::2]),
                 lambda: load(), lambda: load(out=(k.int(), k.int())),
                 lambda: load(out=(k, k[:3])), lambda: load(out=(k, k.float())),
                 lambda: decode(q=q.float()), lambda: decode(q=q.half()), lambda: decode(q=q[:1]),
                 lambda: decode(q=q[..., :32]), lambda: decode(q=q[0]),
                 lambda: decode(out=q[:, :3]), lambda: decode(out=q.float()),
                 lambda: decode(lse=torch.zeros((2, 4, 1))), lambda: decode(lse=q[..., 0]),
                 lambda: prefill(k=k[..., :32]), lambda: prefill(k=k[:3]),
                 lambda: prefill(q=k.half()), lambda: prefill(v=k.half()),
                 lambda: prefill(cu=cu.long()), lambda: prefill(cu_k=cu[:2]),
                 lambda: prefill(out=q), lambda: prefill(lse=torch.zeros(4)),
                 lambda: pq2.kv_cache(4, 2, 16, 64, torch.float32, device="cpu")):
        with pytest.raises(ValueError):
            call()
    # host tensors
    for call in (store, decode, prefill, lambda: load(tokens=2)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
