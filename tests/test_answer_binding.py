"""What the Python calls of pq2_w4_*, pq2_token_logprobs and
pq2_norm_gate_residual refuse by themselves, before a kernel could read or
write past a buffer: shown on host tensors, as the checks look at shapes,
strides and types only."""
import os

import pytest
import torch

from ternary_weight_int8_gb300 import build, pq2

N, K, G = 32, 256, 128
BYTES = 2 * 2 * 1056  # two tiles of two units


def codes_and_scales():
    return torch.zeros((N, K // 2), dtype=torch.uint8), torch.ones((N, K // G)).half()


@pytest.mark.parametrize("plane", [
    torch.zeros(1, dtype=torch.uint8).expand(BYTES),          # one byte in store
    torch.zeros(2 * BYTES, dtype=torch.uint8)[::2],           # every other byte
    torch.zeros((64, BYTES // 64 + 8), dtype=torch.uint8)[:, :-8]])
def test_planes_with_gaps(plane):
    assert plane.numel() >= BYTES and not plane.is_contiguous()
    with pytest.raises(ValueError, match="plane"):
        pq2.pq2_w4_mmv(torch.zeros((1, K)), plane, N, G)
    with pytest.raises(ValueError, match="plane"):
        pq2.pq2_w4_prepare(*codes_and_scales(), group=G, plane=plane)


@pytest.mark.parametrize("dtype", [torch.float32, torch.int8, torch.int64])
def test_planes_of_another_type(dtype):
    plane = torch.zeros(BYTES, dtype=dtype)
    with pytest.raises(ValueError, match="plane"):
        pq2.pq2_w4_mmv(torch.zeros((1, K)), plane, N, G)
    with pytest.raises(ValueError, match="plane"):
        pq2.pq2_w4_prepare(*codes_and_scales(), group=G, plane=plane)


def test_types_outside_the_three():
    """A ValueError that names the types, as for the other arguments."""
    f64 = torch.zeros((2, K), dtype=torch.float64)
    f32 = torch.zeros((2, K))
    plane = torch.zeros(BYTES, dtype=torch.uint8)
    for call in (lambda: pq2.pq2_w4_mmv(f64, plane, N, G),
                 lambda: pq2.pq2_w4_mmv(f32, plane, N, G, out_dtype=torch.float64),
                 lambda: pq2.pq2_w4_mmv(f32, plane, N, G,
                                        y=torch.zeros((2, N), dtype=torch.int32)),
                 lambda: pq2.pq2_token_logprobs(f64),
                 lambda: pq2.pq2_norm_gate_residual(None, f64, f64[0])):
        with pytest.raises(ValueError, match="bfloat16, float16 or float32"):
            call()


@pytest.mark.parametrize("group", [0, -32])
def test_groups_below_one(group):
    if not os.path.exists(pq2.LIB_PATH):
        build.build()
    with pytest.raises(pq2.Pq2Error):
        pq2.pq2_w4_prepare(*codes_and_scales(), group=group)
