"""Scoring given tokens with an 8-bit output projection.

A language model's last hidden states [M, K] go through the output projection
(lm_head) [V, K] and the log probabilities of the tokens that follow are
wanted, with the entropy and the most probable alternatives: what evaluation,
reranking and distillation ask of a served model.  The weights are quantised
once to 8-bit integers with one scale per channel; per call the activations
are quantised per token, the projection runs in 8-bit integers into 32-bit
logits, and one pass over the logits gives the scores.

    python examples/score_tokens.py [--rows 64] [--vocab 32768] [--hidden 5120]

prints a few scores and the largest difference from the same chain in 64 bits
on the unquantised weights (the difference is the quantisation's)."""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def quantize_weight(W):
    """Codes int8 [V, K] and one float32 scale per row of a float weight."""
    import torch
    scale = W.abs().amax(dim=1).clamp_min(1e-12) / 127.0
    return torch.round(W / scale[:, None]).to(torch.int8).contiguous(), scale


class Scorer:
    """An 8-bit output projection and the scores of given tokens under it."""

    def __init__(self, W):
        import weight_only_quantized_qgemm_gb300 as qg
        self.qg = qg
        self.W, self.scale = quantize_weight(W.float())
        self.workspace = qg.Workspace()

    def __call__(self, hidden, tokens, top_k=5):
        """hidden: bf16 or fp16 [M, K]; tokens: int64 [M] or [M, T]."""
        import torch
        Xq, sx = self.qg.quantize_act_int8(hidden)
        logits = self.qg.qgemm_w8a8_int8(Xq, sx, self.W, self.scale, out_dtype=torch.float32,
                                         workspace=self.workspace)
        return self.qg.logprobs(logits, tokens, top_k=top_k, entropy=True)


def main() -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=64)
    ap.add_argument("--vocab", type=int, default=32768)
    ap.add_argument("--hidden", type=int, default=5120)
    a = ap.parse_args()
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)
    W = torch.randn(a.vocab, a.hidden, generator=g, device="cuda") * 0.02
    hidden = torch.randn(a.rows, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    tokens = torch.randint(0, a.vocab, (a.rows,), generator=g, device="cuda")
    r = Scorer(W)(hidden, tokens)
    exact = torch.log_softmax(hidden.double() @ W.double().t(), dim=1)
    off = (r.token_logprobs.double() - exact.gather(1, tokens[:, None])[:, 0]).abs().max().item()
    for m in range(min(3, a.rows)):
        top = ", ".join(f"{i}: {p:.3f}" for i, p in zip(r.top_ids[m].tolist(), r.top_logprobs[m].tolist()))
        print(f"row {m}: token {int(tokens[m])} ln p {float(r.token_logprobs[m]):.3f}, "
              f"entropy {float(r.entropy[m]):.3f}, top {top}")
    print(f"largest difference from 64 bits on unquantised weights: {off:.4f}")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
