"""pq2_norm_gate_residual on buffers of more than 2^31 elements, every row
another one, so that a row read or written elsewhere shows.  Tolerance: that of
the operator's other tests."""
import pytest
import torch

from ternary_weight_int8_gb300 import pq2

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_every_buffer_beyond_32_bits():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    M, K, alpha, eps = 140001, 16384, 0.5, 1e-6
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    z, h, gate = (torch.empty((M, K), dtype=BF16, device="cuda").normal_(0, s, generator=g)
                  for s in (3, 10, 1))
    w_post, w_pre = (torch.empty(K, dtype=BF16, device="cuda").normal_(1, 0.2, generator=g)
                     for _ in range(2))
    h_out, n_out = (torch.full((M, K), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    assert h.numel() > 1 << 31
    pq2.pq2_norm_gate_residual(z, h, w_pre, w_post=w_post, gate=gate, alpha=alpha, eps=eps,
                               h_out=h_out, n_out=n_out)
    torch.cuda.synchronize()
    # the ends, 2^30 and 2^31 elements, and places between
    rows = torch.tensor([0, 1, 8929, 8930, 65535, 65536, 100003, 131071, 131072, 131073, M - 2,
                         M - 1], device="cuda")
    p = z[rows].double()
    p = p * torch.rsqrt(p.square().mean(1, keepdim=True) + eps) * w_post.double()
    add = alpha * p * gate[rows].double()
    h64 = h[rows].double() + add
    inv = torch.rsqrt(h64.square().mean(1, keepdim=True) + eps)
    n64 = h64 * inv * w_pre.double()
    e, half = (K / 256 + 64) * 2.0 ** -24, 2.0 ** -8
    mag = h[rows].double().abs() + add.abs()
    off_h = (h_out[rows].double() - h64).abs() - (e * mag * (1 + half) + half * h64.abs() * 1.01)
    off_n = (n_out[rows].double() - n64).abs() - (
        (e * mag * (inv * w_pre.double()).abs() + e * n64.abs()) * (1 + half)
        + half * n64.abs() * 1.01)
    assert bool((off_h <= 0).all()) and bool((off_n <= 0).all())
    # every row was written
    for a in range(0, M, 10000):
        assert bool(h_out[a:a + 10000].isfinite().all())
        assert bool(n_out[a:a + 10000].isfinite().all())
