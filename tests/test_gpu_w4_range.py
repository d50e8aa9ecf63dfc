"""pq2_w4_mmv with elements of x far below the largest of their 256 columns.

A 32-bit x is the sum of two fp16 parts, the second with a scale 2^12 times the
first's.  With L the largest |x| of a column's aligned 256 elements, an element
is off by at most max(2^-23 |x|, 2^-51 L): of 24 bits the first part takes 11
and the second 11 of at most 12 left (2^-23); below that the second part's
smallest step is 2^-24, half of it undone by 2^12 and by the scale that brings
L to at least 2^14 (2^-25-12-14).  A bf16 x is one part: exact down to 2^-28 L,
within 2^-39 L below.

The largest elements meet weights of zero (the code equal to the zero point, or
a scale of zero), so that they do not hide what the others lose.  Tolerance
(fixed before the first run): with B = sum |s (c - z) x|, in which they have no
share, 1e-5 B as for ordinary x (the arithmetic after the parts is the same, and
2^-23 of each element is within it), and sum |s (c - z)| 2^-51 L (bf16: 2^-39
L)."""
import pytest
import torch

from ternary_weight_int8_gb300 import pq2

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pq2.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [1, 3, 20])
@pytest.mark.parametrize("N,K,G", [(40, 512, 32), (70, 1280, 128), (200, 5120, 64)])
@pytest.mark.parametrize("dtype,power", [(F32, 20), (F32, 24), (F32, 28), (F32, 31), (F32, 42),
                                         (BF16, 20), (BF16, 28), (BF16, 34)])
def test_small_elements_beside_large_ones(M, N, K, G, dtype, power):
    g = torch.Generator(device="cuda")
    g.manual_seed(K + power)
    code = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    zero = torch.randint(0, 16, (N, K // G), generator=g, device="cuda", dtype=torch.uint8)
    scale = (torch.rand((N, K // G), generator=g, device="cuda") * 0.045 + 0.005).half()
    x = torch.randn((M, K), generator=g, device="cuda")
    # one large channel in each 256 columns, 2^power above the others
    large = torch.arange(0, K, 256, device="cuda") + torch.randint(
        0, min(256, K % 256 or 256), (-(-K // 256),), generator=g, device="cuda")
    x[:, large] = 1.5 * 2.0 ** power
    x = x.to(dtype)
    code[:, large] = zero[:, large // G]
    scale[1::4, large // G] = 0
    code[1::4, large] = 15
    packed = (code[:, 0::2] | code[:, 1::2] << 4).contiguous()
    w = (code.double() - zero.double().repeat_interleave(G, 1)) * \
        scale.double().repeat_interleave(G, 1)
    assert not w[:, large].any()
    plane = pq2.pq2_w4_prepare(packed, scale, zero, group=G)
    y = pq2.pq2_w4_mmv(x, plane, N, G, zeros=True)
    y64 = x.double() @ w.t()
    most = torch.full((M, K), 1.5 * 2.0 ** power, dtype=torch.float64, device="cuda")
    least = 2.0 ** (-51 if dtype == F32 else -39)
    tol = 1e-5 * (x.double().abs() @ w.abs().t()) + least * (most @ w.abs().t())
    off = (y.double() - y64).abs() - tol
    assert bool((off <= 0).all()), float(((y.double() - y64).abs() / tol).max())
    assert torch.equal(pq2.pq2_w4_mmv(x[M - 1:], plane, N, G, zeros=True), y[M - 1:])


def test_tiny_and_huge_32_bit_x():
    """The second part's factor undone where the first's is the smallest or
    the largest: subnormal, tiny and huge x keep 23 bits."""
    N, K, G = 48, 256, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    code = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.full((N, K // G), 1.0, device="cuda").half()
    plane = pq2.pq2_w4_prepare(code, scale, group=G)
    c = torch.stack((code % 16, code // 16), -1).view(N, K).double() - 8
    for power in (-140, -127, -126, -113, -40, 0, 60, 112, 117):
        x = ((1 + torch.rand((2, K), generator=g, device="cuda").double()) * 2.0 ** power).float()
        y = pq2.pq2_w4_mmv(x, plane, N, G)
        y64 = x.double() @ c.t()
        # and one rounding to a subnormal y for each of the two parts' pair sums
        tol = 1e-5 * (x.double().abs() @ c.abs().t()) + 4 * 2.0 ** -149
        assert bool(((y.double() - y64).abs() <= tol).all()), power
