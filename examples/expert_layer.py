"""A feed-forward layer of experts in 8 bits, and drafted tokens checked behind it.

A router sends every token to a few of many experts; each expert is a gated
feed-forward layer (silu(x Wg) * (x Wu)) Wd.  The weights are quantised once to
E4M3 with a scale for each block of 128 x 128; per call the activations are
quantised onto the rows of the experts that they go to, the two products run
grouped by expert, and the results come back weighted.  Nothing of the routing
reaches the host, so that a captured call serves any batch.

    python examples/expert_layer.py [--tokens 64] [--hidden 1024] [--inner 512] [--experts 16] [--top 4]

runs the layer on a batch of sequences with drafted tokens, projects the last
states to logits, checks the drafts, and prints how many are kept and the
layer's difference from the same chain in 64 bits on the unquantised weights
(the difference is the quantisation's)."""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def quantize_blocks(W):
    """E4M3 codes (uint8) of float weights [E, N, K] and a float32 scale for each
    block of 128 x 128: [E, ceil(N/128), ceil(K/128)]."""
    import torch
    E, N, K = W.shape
    NB, KB = -(-N // 128), -(-K // 128)
    padded = torch.zeros((E, NB * 128, KB * 128), device=W.device)
    padded[:, :N, :K] = W
    amax = padded.view(E, NB, 128, KB, 128).abs().amax(dim=(2, 4))
    scale = torch.where(amax > 0, amax / 448.0, 1.0)
    spread = scale.repeat_interleave(128, dim=1)[:, :N].repeat_interleave(128, dim=2)[:, :, :K]
    codes = (W / spread).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).contiguous(), scale.contiguous()


class ExpertLayer:
    """router [E, H]; gate, up [E, F, H] and down [E, H, F] of every expert."""

    def __init__(self, router, gate, up, down, top_k, bias=None, score="softmax", scale=1.0):
        import torch
        import weight_only_quantized_qgemm_gb300 as qg
        self.qg, self.router, self.top_k = qg, router, top_k
        self.how = dict(score=score, bias=bias, scale=scale)
        self.gate_up = quantize_blocks(torch.cat([gate, up], dim=1))
        self.down = quantize_blocks(down)

    def __call__(self, x, residual=None):
        """x: bf16 [M, H] -> bf16 [M, H]."""
        qg = self.qg
        r = qg.moe_route(x @ self.router.t(), self.top_k, **self.how)
        codes, scales = qg.quantize_rows_e4m3(x, rows=r.rows)
        h = qg.qgemm_w8a8_grouped(codes, scales, *self.gate_up, r.offsets)
        codes, scales = qg.quantize_rows_e4m3(h, gated=True, num_rows=r.offsets[-1:])
        y = qg.qgemm_w8a8_grouped(codes, scales, *self.down, r.offsets)
        return qg.moe_combine(y, r.rows, r.weights, residual=residual)


def main() -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=512)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top", type=int, default=4)
    ap.add_argument("--vocab", type=int, default=8192)
    ap.add_argument("--drafts", type=int, default=3)
    a = ap.parse_args()
    import torch
    import weight_only_quantized_qgemm_gb300 as qg
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*size, std=1.0):
        return torch.randn(*size, generator=g, device="cuda") * std

    E, H, F = a.experts, a.hidden, a.inner
    gate, up, down = normal(E, F, H, std=H ** -0.5), normal(E, F, H, std=H ** -0.5), normal(E, H, F, std=F ** -0.5)
    router = normal(E, H, std=H ** -0.5).to(torch.bfloat16)
    layer = ExpertLayer(router, gate, up, down, a.top)
    sequences = max(1, a.tokens // (a.drafts + 1))
    x = normal(sequences * (a.drafts + 1), H).to(torch.bfloat16)
    y = layer(x)

    # the same in 64 bits, with every expert on every token
    r = qg.moe_route(x @ router.t(), a.top)
    xd = x.double()
    exact = torch.zeros_like(xd)
    for e in range(E):
        w = (r.weights.double() * (r.experts == e)).sum(dim=1, keepdim=True)
        h = torch.nn.functional.silu(xd @ gate[e].double().t()) * (xd @ up[e].double().t())
        exact += w * (h @ down[e].double().t())
    off = float((y.double() - exact).norm() / exact.norm())

    head = normal(a.vocab, H, std=2.0 * H ** -0.5).to(torch.bfloat16)
    logits = ((x.float() + y.float()).to(torch.bfloat16) @ head.t()).view(sequences, a.drafts + 1, a.vocab)
    draft = (logits[:, :-1].float() + 0.5 * normal(sequences, a.drafts, a.vocab)).to(torch.bfloat16)
    drafted = (torch.softmax(draft.float(), dim=2) /
               torch.empty(draft.shape, device="cuda").exponential_(generator=g)).argmax(dim=2)
    check = qg.verify_drafts(logits, drafted, draft, torch.rand(sequences, a.drafts, generator=g, device="cuda"),
                             torch.empty(sequences, a.vocab, device="cuda").exponential_(generator=g))
    kept = check.accepted.float().mean().item()
    print(f"{x.shape[0]} tokens, {a.top} of {E} experts: difference from 64 bits on unquantised weights {off:.4f}")
    print(f"{sequences} sequences: {kept:.2f} of {a.drafts} drafts kept, first tokens {check.tokens[0].tolist()}")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
