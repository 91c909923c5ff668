"""Paths of the router, the grouped GEMM and the draft verification that only some
sizes reach, each held to a plain implementation in 64 bits (tolerances as in
test_gpu_experts.py and test_gpu_verify.py)."""
import math

import pytest
import torch

from gpu_util import qg
from test_gpu_experts import DTYPES, check_grouped, check_route, gen, grouped_problem
from test_gpu_verify import SHAPES, check, problem, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    return qg()


# ----------------------------------------------------------------- router
# With more than four tokens a warp (of 32 on each SM; of 16 from 513 experts on) their
# places wait in `rows`, not in shared memory.
@pytest.mark.parametrize("M,E,k,score,biased", [(19456, 40, 3, "softmax", False), (19457, 40, 3, "softmax", False),
                                                (20000, 256, 8, "sigmoid", True), (40001, 64, 6, "softmax", True),
                                                (24000, 513, 4, "sigmoid", False), (65537, 16, 2, "softmax", False)])
def test_route_many_tokens_a_warp(q, M, E, k, score, biased):
    g = gen(M + E)
    logits = (torch.randn(M, E, generator=g, device="cuda") * 2).to(torch.bfloat16)
    logits[::1001] = -math.inf                       # padding
    logits[5::997, : E // 2] = -math.inf
    logits[7, 1] = math.nan
    bias = torch.randn(E, generator=g, device="cuda") * 0.1 if biased else None
    check_route(q, logits, k, score=score, bias=bias, scale=2.5)


@pytest.mark.parametrize("E", [40, 64, 200])
@pytest.mark.parametrize("k", [1, 5, 32])
def test_route_softmax_scores_nearer_than_32_bits(q, E, k):
    """Sums of softmax and bias that differ by less than an FP32 step."""
    x = torch.linspace(-3, 3, E, device="cuda", dtype=torch.float32).repeat(40, 1)
    x[20:] = x[20:].flip(1)
    bias = (0.9 - torch.softmax(x[0].double(), dim=0)).float()
    check_route(q, x, k, score="softmax", bias=bias)
    check_route(q, x[:, torch.randperm(E, generator=gen(E), device="cuda")], k, score="softmax", bias=bias, renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [math.inf, 3e38, -3e38, 1e8])
def test_route_biases_beyond_the_scores(q, score, value):
    """A bias in which a score is lost, in FP32 or altogether: the order of 64 bits, ties
    to the lower index."""
    E, M = 50, 70
    logits = torch.randn(M, E, generator=gen(5), device="cuda") * 2
    logits[3, 10:] = -math.inf
    bias = torch.zeros(E, device="cuda")
    bias[5:E:5] = value
    for k in (1, 4, 12):
        check_route(q, logits, k, score=score, bias=bias)
        check_route(q, logits, k, score=score, bias=bias, renormalize=False)


# ----------------------------------------------------------------- row quantiser
def test_a_place_named_twice_by_its_token(q):
    X = torch.randn(3, 272, generator=gen(1), device="cuda").to(torch.bfloat16)
    rows = torch.tensor([[4, 4, 4], [1, 0, 1], [-1, 7, 7]], dtype=torch.int32, device="cuda")
    Xq, Xs = torch.full((9, 272), 0x55, dtype=torch.uint8, device="cuda"), torch.full((3, 12), -7.0, device="cuda")
    q.quantize_rows_e4m3(X, rows=rows, Xq=Xq, X_scale=Xs)
    want_q, want_s = q.quantize_act_e4m3(X)
    for row, m in ((4, 0), (0, 1), (1, 1), (7, 2)):
        assert torch.equal(Xq[row], want_q[m]) and torch.equal(Xs[:, row], want_s[:, m])
    assert bool((Xq[[2, 3, 5, 6, 8]] == 0x55).all()) and bool((Xs[:, [2, 3, 5, 6, 8, 9, 10, 11]] == -7.0).all())


# ----------------------------------------------------------------- grouped GEMM
CANDIDATES = [[5, 2], [3] * 40, [30, 31] * 20, [40, 33, 1, 0, 32, 31] * 4, [64, 60] * 40, [64] * 60, [700, 300] * 10,
              [1500, 3000, 1]]


@pytest.mark.parametrize("rows", [16, 32, 64, 256])
def test_a_wait_that_runs_out_in_the_form_of_this_device(q, rows):
    """As the form goes by the device's own number of SMs."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    sizes = [s for s in CANDIDATES if q.grouped_tile_rows(sum(s), len(s), 512, 2048, sms) == rows]
    assert sizes, "no candidate takes this form"
    Xq, Xs, W, Ws, off = grouped_problem(sizes[0], 512, 2048, 3)
    assert q.last_device_status() == 0
    q.set_wait_timeout_ns(20_000_000)
    q.set_fault_injection(3)
    try:
        q.qgemm_w8a8_grouped(Xq, Xs, W, Ws, off)
        assert q.last_device_status() == 5
    finally:
        q.set_fault_injection(-1)
        q.set_wait_timeout_ns(1_000_000_000)
    for s in sizes:
        check_grouped(q, s, 512, 2048, "bf16")


# ----------------------------------------------------------------- drafts
@pytest.mark.parametrize("B,G,V", [(20, 2, 65537), (24, 3, 70001), (20, 1, 131072), (40, 2, 140001)])
@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("fp32", 3)])
def test_many_sequences_of_a_large_vocabulary(q, B, G, V, dtype, pad):
    """More stretches of a row than a warp has lanes, and rows that are done again
    about their maximum."""
    t, d, tok, u, e = problem(B, G, V, dtype, B + V, pad)
    lengths = torch.randint(0, G + 1, (B,), generator=gen(V), device="cuda", dtype=torch.int32)
    check(q, t, tok, draft=d, uniform=u, noise=e)
    check(q, t, tok, draft=d, uniform=u, noise=e, lengths=lengths)
    keep = torch.rand(V, generator=gen(B), device="cuda") < 0.01
    keep[:4] = True
    t[1] = torch.where(keep, t[1], torch.finfo(DTYPES[dtype]).min)
    d[2] = torch.where(keep, d[2], -math.inf)
    t[3, 0] = torch.finfo(DTYPES[dtype]).min
    t[4, 0, V - 1] = math.nan
    t[5, 0] = -math.inf
    t[6, 0, 66000 % V] = math.inf
    tok[7:, 0] = t[7:, 0].float().argmax(dim=1)
    check(q, t, tok, uniform=u, noise=e, most_unsure=0.1)
    check(q, t, tok, lengths=lengths, most_unsure=0.1)


@pytest.mark.parametrize("B,G,V", [s for s in SHAPES if s[0] <= 3])
@pytest.mark.parametrize("kind", ["sampled", "certain", "greedy"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_lone_sequences_that_are_decided(q, B, G, V, kind, dtype):
    """Of few sequences every one may be too near to call: seeds until some are not,
    and those are compared."""
    compared = 0
    for seed in range(12):
        t, d, tok, u, e = problem(B, G, V, dtype, 1000 + seed)
        kw = {} if kind == "greedy" else dict(uniform=u, noise=e)
        if kind == "sampled":
            kw["draft"] = d
        elif seed % 2:
            tok = t[:, :G].float().argmax(dim=2)
        sure = sum(r[2] for r in reference(t, tok, **kw))
        check(q, t, tok, most_unsure=1.0, **kw)
        compared += sure
        if compared >= 3:
            return
    assert compared >= 3


@pytest.mark.parametrize("B", [5, 25])
def test_draft_rows_that_say_nothing(q, B):
    """A draft's row with a NaN or +inf, or with nothing but -inf, keeps no draft, and the
    token is drawn from the target's row alone."""
    t, d, tok, u, e = problem(B, 2, 9000, "fp32", 3)
    tok[:, 0] = t[:, 0].argmax(dim=1)
    u[:, 0] = 0.0
    d[0, 0, 8999] = math.nan
    d[1, 0] = -math.inf
    d[2, 0, 5] = math.inf
    d[3, 0] = math.nan
    got = q.verify_drafts(t, tok, d, u, e)
    p = torch.softmax(t[:, 0].double(), dim=1) / e.double()
    top = p.topk(2, dim=1)
    for b in range(4):
        assert int(got.accepted[b]) == 0
        if float(top.values[b, 0]) * (1 - 2.0 ** -18) > float(top.values[b, 1]):
            assert int(got.tokens[b, 0]) == int(top.indices[b, 0])
    assert bool((got.accepted[4:] >= 1).all())
