"""The argument checks of pq2_w4_*, pq2_token_logprobs and
pq2_norm_gate_residual on the host: every refusal comes before any CUDA call,
so fake addresses are never dereferenced."""
import os

import pytest

from ternary_weight_int8_gb300 import build, pq2

A = 1 << 20   # a 16-byte aligned fake address


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


NULL, SHAPE, ALIGN, DTYPE = (pq2.PQ2_ERR_NULL, pq2.PQ2_ERR_SHAPE, pq2.PQ2_ERR_ALIGN,
                             pq2.PQ2_ERR_DTYPE)


def test_plane_bytes(L):
    f = L.pq2_w4_plane_bytes
    # 16 rows x 128 columns: 1024 bytes of codes, 32 of scales per group, 8 of
    # zero points per group, to 16 bytes
    assert f(16, 128, 128, 0) == 1056 and f(16, 128, 64, 0) == 1088 and f(16, 128, 32, 0) == 1152
    assert f(16, 128, 128, 1) == 1072 and f(16, 128, 64, 1) == 1104 and f(16, 128, 32, 1) == 1184
    assert f(17, 160, 32, 0) == 4 * 1152
    for bad in ((0, 128, 128, 0), (16, 64, 128, 0), (16, 192, 128, 0), (16, 128, 16, 0),
                (16, 0, 32, 0)):
        assert f(*bad) == 0


def test_w4_prepare_refusals(L):
    ok = [A, 64, A, A, 10, 128, 64, A, None]
    refused(L.pq2_w4_prepare, ok, (0, None, NULL), (2, None, NULL), (7, None, NULL),
            (1, 63, SHAPE), (4, 0, SHAPE), (5, 96, SHAPE), (6, 48, SHAPE), (2, A + 1, ALIGN),
            (7, A + 8, ALIGN))


def test_w4_mmv_refusals(L):
    ok = [A, pq2.PQ2_BF16, 256, 4, 10, 256, 128, 0, A, A, pq2.PQ2_F32, 0, None]
    refused(L.pq2_w4_mmv, ok, (0, None, NULL), (8, None, NULL), (9, None, NULL), (1, 3, DTYPE),
            (10, -1, DTYPE), (11, 4, DTYPE), (3, 0, SHAPE), (3, 33, SHAPE), (4, 0, SHAPE),
            (2, 255, SHAPE), (5, 192, SHAPE), (6, 256, SHAPE), (0, A + 1, ALIGN),
            (8, A + 8, ALIGN), (9, A + 2, ALIGN))


def test_token_logprobs_refusals(L):
    ok = [A, pq2.PQ2_BF16, 100, 2, 100, 1.0, A, 1, A, A, 5, A, A, None]
    refused(L.pq2_token_logprobs, ok, (0, None, NULL), (6, None, NULL), (8, None, NULL),
            (11, None, NULL), (12, None, NULL), (1, 7, DTYPE), (2, 99, SHAPE), (3, 0, SHAPE),
            (3, (1 << 20) + 1, SHAPE), (4, 0, SHAPE), (4, 4, SHAPE), (5, 0.0, SHAPE),
            (5, float("inf"), SHAPE), (5, float("nan"), SHAPE), (7, -1, SHAPE), (10, 33, SHAPE),
            (10, -1, SHAPE), (0, A + 1, ALIGN), (6, A + 4, ALIGN), (8, A + 2, ALIGN),
            (9, A + 2, ALIGN), (11, A + 4, ALIGN), (12, A + 1, ALIGN))


def test_norm_refusals(L):
    ok = [A, 64, A, 64, pq2.PQ2_BF16, A, A, 64, 1, 1.0, A, 0.0, 1e-6, 3, 64, A, A, None]
    refused(L.pq2_norm_gate_residual, ok, (2, None, NULL), (0, None, NULL), (10, None, NULL),
            (4, 5, DTYPE), (1, 63, SHAPE), (3, 63, SHAPE), (7, 63, SHAPE), (8, 0, SHAPE),
            (12, -1e-6, SHAPE), (12, 2.0, SHAPE), (13, 0, SHAPE), (14, 0, SHAPE),
            (14, pq2.PQ2_PREP_MAX_K + 1, SHAPE), (0, A + 1, ALIGN), (5, A + 1, ALIGN),
            (15, A + 1, ALIGN))
    both = list(ok)
    both[15] = both[16] = None
    assert L.pq2_norm_gate_residual(*both) == NULL
    strided = list(ok)
    strided[3] = 72  # h_out over h needs h to be contiguous
    assert L.pq2_norm_gate_residual(*strided) == SHAPE
