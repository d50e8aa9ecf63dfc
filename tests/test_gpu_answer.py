"""examples/answer_step.py: the projection, the gated residual norms, the 4-bit
head and the log-probabilities in one chain, each step against 64 bits on the
inputs that it had."""
import os
import sys

import pytest
import torch

from ternary_weight_int8_gb300 import pq2, synth

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.mark.parametrize("M", [1, 5, 24])
@pytest.mark.parametrize("hidden,vocabulary,group", [(1280, 5003, 64), (2048, 20000, 128)])
def test_answer_step(M, hidden, vocabulary, group):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from answer_step import AnswerStep
    step = AnswerStep(hidden, vocabulary, group, seed=M)
    x = synth.activations(M, hidden, seed=2, device="cuda", outlier_frac=0.01)
    h0 = synth.activations(M, hidden, seed=3, device="cuda")
    tokens = torch.randint(0, vocabulary, (M, 2), device="cuda",
                           generator=torch.Generator("cuda").manual_seed(4))
    # Several steps in a row, nothing waited for between them.
    for _ in range(3):
        h, logits, lp, entropy, ids, top = step(x, h0, tokens, 4, temperature=0.8)
    torch.cuda.synchronize()

    z = pq2.pq2_linear(x, step.codes, step.scales, out_dtype=torch.bfloat16).double()
    z = z * torch.rsqrt(z.square().mean(1, keepdim=True) + 1e-6) * step.w_post.double()
    h64 = h0.double() + 0.5 * z * step.gate.double()
    # bf16 of an fp32 result: half a unit in the last place, and fp32 steps
    assert bool(((h.double() - h64).abs() <= 2.0 ** -8 * h64.abs() + 1e-5).all())

    n64 = h64 * torch.rsqrt(h64.square().mean(1, keepdim=True) + 1e-6) * step.w_pre.double()
    _, n = pq2.pq2_norm_gate_residual(
        pq2.pq2_linear(x, step.codes, step.scales, out_dtype=torch.bfloat16), h0, step.w_pre,
        w_post=step.w_post, gate=step.gate, rows_per_gate=M, alpha=0.5)
    assert bool(((n.double() - n64).abs() <= 2.0 ** -8 * n64.abs() + 1e-5).all())

    c = torch.stack((step.head_codes % 16, step.head_codes // 16), -1).view(vocabulary, hidden)
    w = (c.double() - step.head_zeros.double().repeat_interleave(group, 1)) * \
        step.head_scales.double().repeat_interleave(group, 1)
    y64 = n.double() @ w.t()
    # the tolerance of the head's own tests
    assert bool(((logits.double() - y64).abs() <= 1e-5 * (n.double().abs() @ w.abs().t())).all())

    logp = torch.log_softmax(logits.double() / 0.8, 1)
    assert torch.equal(ids, torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :4])
    assert float((lp.double() - logp.gather(1, tokens)).abs().max()) < 1e-4
    assert float((top.double() - logp.gather(1, ids)).abs().max()) < 1e-4
    assert float((entropy.double() + (logp.exp() * logp).sum(1)).abs().max()) < 1e-3
