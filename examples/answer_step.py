"""The end of a decode step of a ternary model on one GPU: a block's ternary
projection, the norms around it with its gate and residual scale, the 4-bit
output head, and the log-probabilities of the tokens it may answer with.

    python examples/answer_step.py [--tokens M] [--hidden K] [--vocabulary V]

Weights are random; every step is a call of the library on the current stream.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from ternary_weight_int8_gb300 import pq2, synth  # noqa: E402


class AnswerStep:
    """The weights of the last block's output projection and of the head, laid
    out once, and one call per step."""

    def __init__(self, hidden: int, vocabulary: int, group: int = 128, seed: int = 0,
                 device="cuda"):
        self.hidden, self.vocabulary, self.group = hidden, vocabulary, group
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def rand(*shape):
            return torch.rand(shape, generator=g, device=device)
        self.raw = synth.raw_weights(hidden, hidden, seed=seed + 1, device=device)
        self.codes, self.scales = pq2.pq2_prepare(self.raw, hidden)
        self.w_post = (0.8 + 0.4 * rand(hidden)).bfloat16()
        self.w_pre = (0.8 + 0.4 * rand(hidden)).bfloat16()
        self.gate = (rand(1, hidden) * 2 - 1).bfloat16()
        self.head_codes = torch.randint(0, 256, (vocabulary, hidden // 2), generator=g,
                                        device=device, dtype=torch.uint8)
        self.head_scales = (rand(vocabulary, hidden // group) * 0.01 + 0.002).half()
        self.head_zeros = torch.randint(6, 10, (vocabulary, hidden // group), generator=g,
                                        device=device, dtype=torch.uint8)
        self.plane = pq2.pq2_w4_prepare(self.head_codes, self.head_scales, self.head_zeros,
                                        group=group)
        # The planes are complete before a call may stream them early.
        torch.cuda.synchronize()

    def __call__(self, x, h, tokens, k: int, temperature: float = 1.0, alpha: float = 0.5):
        """x bf16 [M][hidden]: the projection's input; h bf16 [M][hidden]: the
        residual stream -> (h after the block, logits, log-probabilities of
        `tokens`, entropy, the k best ids and their log-probabilities)."""
        z = pq2.pq2_linear(x, self.codes, self.scales, out_dtype=torch.bfloat16)
        h, n = pq2.pq2_norm_gate_residual(z, h, self.w_pre, w_post=self.w_post, gate=self.gate,
                                          rows_per_gate=x.shape[0], alpha=alpha)
        logits = pq2.pq2_w4_mmv(n, self.plane, self.vocabulary, self.group, zeros=True,
                                flags=pq2.PQ2_MMV_OVERLAP_WEIGHTS)
        return (h, logits, *pq2.pq2_token_logprobs(logits, tokens, k, scale=1.0 / temperature))


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--vocabulary", type=int, default=131072)
    a = ap.parse_args()
    step = AnswerStep(a.hidden, a.vocabulary)
    x = synth.activations(a.tokens, a.hidden, seed=2, device="cuda", outlier_frac=0.01)
    h = synth.activations(a.tokens, a.hidden, seed=3, device="cuda")
    tokens = torch.arange(a.tokens, device="cuda")[:, None]
    _, _, lp, entropy, ids, top = step(x, h, tokens, 5)
    for m in range(a.tokens):
        best = ", ".join(f"{i} ({v:.3f})" for i, v in zip(ids[m].tolist(), top[m].tolist()))
        print(f"row {m}: entropy {entropy[m]:.3f}, log p of token {m} {lp[m, 0]:.3f}; best {best}")


if __name__ == "__main__":
    main()
