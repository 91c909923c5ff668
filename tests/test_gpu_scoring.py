"""The scoring path end to end (examples/score_tokens.py): quantiser, 8-bit
output projection and log probabilities in a row, against 64-bit arithmetic on
the same codes."""
import importlib.util
import os

import pytest
import torch

from gpu_util import qg

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("score_tokens", os.path.join(ROOT, "examples", "score_tokens.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("M,V,K", [(1, 1000, 256), (7, 5003, 512), (40, 8192, 1024), (300, 2051, 272)])
def test_scores_match_64_bits_on_the_codes(M, V, K):
    q = qg()
    ex = _example()
    g = torch.Generator(device="cuda").manual_seed(M)
    W = torch.randn(V, K, generator=g, device="cuda") * 0.2
    hidden = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    tokens = torch.randint(0, V, (M, 2), generator=g, device="cuda")
    scorer = ex.Scorer(W)
    r = scorer(hidden, tokens, top_k=4)
    assert q.last_device_status() == 0
    Xq, sx = q.quantize_act_int8(hidden)
    logits = (Xq.double() * sx.double()[:, None]) @ (scorer.W.double() * scorer.scale.double()[:, None]).t()
    lp = torch.log_softmax(logits, dim=1)
    # a logit is off by 3 roundings of 2^-24 of its size; scores by that of the
    # largest logits and by the sums' own error (64 u and the terms' arguments)
    big = logits.abs().amax().item()
    tol = 2.0 ** -24 * (8 * big + 2 * (logits.amax() - logits.amin()).item() + V / 128 + 64)
    assert (r.token_logprobs.double() - lp.gather(1, tokens)).abs().max().item() <= tol
    assert (r.top_logprobs.double() - lp.topk(4, dim=1).values).abs().max().item() <= tol
    entropy = torch.special.entr(lp.exp()).sum(dim=1)
    assert (r.entropy.double() - entropy).abs().max().item() <= tol * (2 + 4 * float(entropy.max()))


def test_example_runs(capsys, monkeypatch):
    ex = _example()
    monkeypatch.setattr("sys.argv", ["score_tokens.py", "--rows", "5", "--vocab", "2000", "--hidden", "512"])
    assert ex.main() == 0
    out = capsys.readouterr().out
    assert "row 0: token" in out and "largest difference" in out
