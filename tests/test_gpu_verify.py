"""Verification of drafted tokens on the GPU against a plain implementation in
64 bits.  Kept counts and tokens are whole numbers and have to be equal, except
where the decision in 64 bits is nearer than the FP32 probabilities' error (their
exponentials and sums are good to 2^-20; the difference max(p - q, 0) to that of
p and q): those sequences are left out, and counted."""
import math

import pytest
import torch

from gpu_util import qg

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NEAR = 2.0 ** -19


@pytest.fixture(scope="module")
def q():
    return qg()


def reference(target, tokens, draft=None, uniform=None, noise=None, lengths=None):
    """[(accepted, tokens, decided)] per sequence."""
    B, G1, V = target.shape
    G = G1 - 1
    out = []
    for b in range(B):
        length = G if lengths is None else max(0, min(G, int(lengths[b])))
        n, sure = 0, True
        if uniform is None:
            def largest(row):
                row = torch.where(row.isnan(), -math.inf, row)
                m = row.max()
                return -1 if m == -math.inf else int(torch.nonzero(row == m)[0])
            while n < length and largest(target[b, n].double()) == int(tokens[b, n]):
                n += 1
            last = largest(target[b, n].double())
        else:
            def probs(row):
                row = row.double()
                return torch.softmax(row, dim=0) if bool((row < math.inf).all()) and bool((row > -math.inf).any()) \
                    else torch.full_like(row, math.nan)

            def other(i):
                if draft is not None:
                    return probs(draft[b, i])
                one = torch.zeros(V, dtype=torch.float64, device=target.device)
                if 0 <= int(tokens[b, i]) < V:
                    one[int(tokens[b, i])] = 1.0
                return one
            while n < length:
                d = int(tokens[b, n])
                if not 0 <= d < V:
                    break
                p, qd = float(probs(target[b, n])[d]), float(uniform[b, n]) * float(other(n)[d])
                if math.isfinite(p) and math.isfinite(qd) and p != qd:
                    sure &= abs(p - qd) > NEAR * max(p, qd)
                if not qd < p:
                    break
                n += 1
            p = probs(target[b, n])
            err = NEAR * p
            w = p
            if n < length:
                o = other(n)
                diff = (p - o).clamp_min(0)
                diff = torch.where((p - o).isnan(), math.nan, diff)
                if bool((diff > 0).any()):
                    w, err = diff, NEAR * (p + o)
            # a noise of 0 makes a ratio of infinity
            ratio = torch.where((w > 0) & (noise[b] >= 0), w / noise[b].double(), 0.0)
            wrong = torch.where((w > 0) & (noise[b] >= 0), err / noise[b].double(), 0.0)
            if bool((ratio > 0).any()):
                last = int(ratio.argmax())
                rest = ratio + wrong
                rest[last] = 0
                sure &= bool(ratio[last] - wrong[last] > rest.max())
            else:
                last = -1
        out.append((n, tokens[b, :n].tolist() + [last] + [-1] * (G - n), sure))
    return out


def check(q, target, tokens, most_unsure=0.05, **kw):
    got = q.verify_drafts(target, tokens, draft_logits=kw.get("draft"), uniform=kw.get("uniform"),
                          noise=kw.get("noise"), lengths=kw.get("lengths"))
    ref = reference(target, tokens, **kw)
    sure = [r[2] for r in ref]
    assert sum(sure) >= (1 - most_unsure) * len(sure) - 1
    for b, (n, toks, ok) in enumerate(ref):
        if ok:
            assert int(got.accepted[b]) == n, b
            assert got.tokens[b].tolist() == toks, b
    return got


def problem(B, G, V, dtype, seed, pad=0, noise=0.6):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(B, G + 1, V, generator=g, device="cuda") * 2.5
    d = t[:, :G] + noise * torch.randn(B, G, V, generator=g, device="cuda")
    wide_t = torch.zeros((B, G + 1, V + pad), dtype=DTYPES[dtype], device="cuda")
    wide_d = torch.zeros((B, G, V + pad), dtype=DTYPES[dtype], device="cuda")
    wide_t[:, :, :V] = t
    wide_d[:, :, :V] = d
    target, draft = wide_t[:, :, :V], wide_d[:, :, :V]
    if G:
        race = torch.empty(B, G, V, device="cuda").exponential_(generator=g)
        tokens = (torch.softmax(draft.float(), dim=2) / race).argmax(dim=2)
    else:
        tokens = torch.empty((B, 0), dtype=torch.int64, device="cuda")
    uniform = torch.rand(B, G, generator=g, device="cuda")
    exp = torch.empty(B, V, device="cuda").exponential_(generator=g)
    return target, draft, tokens, uniform, exp


SHAPES = [(1, 1, 1), (1, 1, 7), (3, 2, 100), (2, 4, 2048), (1, 4, 32768), (5, 3, 50021), (40, 5, 4099), (160, 1, 3001),
          (2, 31, 5000), (4, 0, 9000), (1, 8, 131072), (300, 2, 257)]


@pytest.mark.parametrize("B,G,V", SHAPES)
@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("bf16", 5), ("fp16", 64), ("fp32", 1)])
def test_sampled_drafts(q, B, G, V, dtype, pad):
    t, d, tok, u, e = problem(B, G, V, dtype, B * 31 + G * 7 + V, pad)
    check(q, t, tok, draft=d, uniform=u, noise=e)


@pytest.mark.parametrize("B,G,V", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_certain_drafts(q, B, G, V, dtype):
    t, d, tok, u, e = problem(B, G, V, dtype, B + G + V, 3)
    if G:
        tok = torch.where(torch.rand(B, G, device="cuda") < 0.7, t[:, :G].float().argmax(dim=2), tok)
    check(q, t, tok, uniform=u, noise=e)


@pytest.mark.parametrize("B,G,V", SHAPES)
@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("fp16", 3), ("fp32", 0)])
def test_greedy(q, B, G, V, dtype, pad):
    t, d, tok, u, e = problem(B, G, V, dtype, B * 3 + G + V, pad)
    if G:
        # the first of the largest, mostly
        first = torch.where(t[:, :G] == t[:, :G].amax(dim=2, keepdim=True),
                            torch.arange(V, device="cuda"), V).amin(dim=2)
        tok = torch.where(torch.rand(B, G, device="cuda") < 0.8, first, tok)
    check(q, t, tok)


def test_lengths_and_odd_tokens(q):
    B, G, V = 24, 6, 3000
    t, d, tok, u, e = problem(B, G, V, "bf16", 77)
    lengths = torch.tensor([0, 1, 2, 3, 4, 5, 6, 9, -2] * 3, dtype=torch.int32, device="cuda")[:B]
    tok[3, 0] = -1
    tok[4, 1] = V
    tok[5, 0] = 2 ** 40
    check(q, t, tok, draft=d, uniform=u, noise=e, lengths=lengths)
    check(q, t, tok, uniform=u, noise=e, lengths=lengths)
    check(q, t, tok, lengths=lengths)


def test_rows_behind_a_length_are_not_looked_at(q):
    B, G, V = 4, 5, 2500
    t, d, tok, u, e = problem(B, G, V, "fp32", 78)
    lengths = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    a = q.verify_drafts(t, tok, d, u, e, lengths)
    t[:, 3:] = math.nan
    d[:, 2:] = math.nan
    b = q.verify_drafts(t, tok, d, u, e, lengths)
    assert torch.equal(a.accepted, b.accepted) and torch.equal(a.tokens, b.tokens)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masks_infinities_and_nan(q, dtype):
    B, G, V = 14, 3, 5000
    t, d, tok, u, e = problem(B, G, V, dtype, 79)
    lowest = torch.finfo(DTYPES[dtype]).min
    keep = torch.rand(V, device="cuda") < 0.01
    keep[:4] = True
    t[0] = torch.where(keep, t[0], -math.inf)               # a filter of the target
    d[1] = torch.where(keep, d[1], -math.inf)
    t[2, 0] = -math.inf                                      # nothing left
    t[3, 1, 17] = math.nan
    t[4, 0, V - 1] = math.inf
    d[5, 0] = -math.inf
    d[6, 1, 3] = math.nan
    t[7] = torch.where(keep, t[7], lowest)                   # masked with the type's lowest value
    d[7] = torch.where(keep, d[7], lowest)
    t[8, 0] = lowest                                         # all equal, as low as can be
    t[9, 0, :] = -math.inf
    t[9, 0, 123] = 2.0                                       # one token left
    tok[9, 0] = 123
    tok[10, 0] = 7
    t[10, 0, 7] = -math.inf                                  # the draft is masked by both
    d[10, 0, 7] = -math.inf
    d[11] = t[11, :G]                                        # the same distribution: all are kept
    e[12] = 0.0                                              # every ratio is infinite
    t[13] = t[13] * 0 + 3e4 * (torch.arange(V, device="cuda") == 11)   # a token beyond all others
    check(q, t, tok, draft=d, uniform=u, noise=e, most_unsure=0.5)
    check(q, t, tok, uniform=u, noise=e, most_unsure=0.5)
    check(q, t, tok, most_unsure=0.5)
    got = q.verify_drafts(t, tok, d, u, e)
    assert int(got.accepted[11]) == G
    assert int(got.tokens[2, 0]) == -1 and int(got.tokens[4, 0]) == -1


def test_distribution_is_the_targets(q):
    """Over many sequences with the same rows, the first token is distributed as
    the target's (chi-squared with 15 degrees of freedom: below 60 with 1 - 2e-7)."""
    V, B = 16, 20000
    g = torch.Generator(device="cuda").manual_seed(3)
    t = torch.randn(1, 2, V, generator=g, device="cuda").expand(B, 2, V).contiguous()
    d = torch.randn(1, 1, V, generator=g, device="cuda").expand(B, 1, V).contiguous()
    race = torch.empty(B, V, device="cuda").exponential_(generator=g)
    tok = (torch.softmax(d[:, 0], dim=1) / race).argmax(dim=1, keepdim=True)
    u = torch.rand(B, 1, generator=g, device="cuda")
    e = torch.empty(B, V, device="cuda").exponential_(generator=g)
    got = q.verify_drafts(t, tok, d, u, e)
    want = torch.softmax(t[0, 0].double(), dim=0) * B
    seen = torch.bincount(got.tokens[:, 0], minlength=V).double()
    assert float(((seen - want) ** 2 / want).sum()) < 60


# sequences enough that the rows' sums come from a kernel of their own
MANY = [(24, 3, 20011), (64, 5, 9000), (20, 31, 8192), (130, 1, 8193), (40, 0, 12000)]


@pytest.mark.parametrize("B,G,V", MANY)
@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("bf16", 3), ("fp16", 8), ("fp32", 1), ("fp32", 4)])
def test_many_sequences(q, B, G, V, dtype, pad):
    t, d, tok, u, e = problem(B, G, V, dtype, B + G * 5 + V, pad)
    lengths = torch.randint(-1, G + 2, (B,), device="cuda", dtype=torch.int32)
    check(q, t, tok, draft=d, uniform=u, noise=e)
    check(q, t, tok, draft=d, uniform=u, noise=e, lengths=lengths)
    if G:
        tok = torch.where(torch.rand(B, G, device="cuda") < 0.7, t[:, :G].float().argmax(dim=2), tok)
    check(q, t, tok, uniform=u, noise=e, lengths=lengths)
    check(q, t, tok, lengths=lengths)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_odd_rows_of_many_sequences(q, dtype):
    B, G, V = 30, 2, 9001
    t, d, tok, u, e = problem(B, G, V, dtype, 5, 7)
    keep = torch.rand(V, device="cuda") < 0.01
    keep[:4] = True
    t[0] = torch.where(keep, t[0], -math.inf)
    d[1] = torch.where(keep, d[1], -math.inf)
    t[2, 0] = -math.inf
    t[3, 1, 17] = math.nan
    t[4, 0, V - 1] = math.inf
    d[5, 0] = -math.inf
    d[6, 1, 3] = math.nan
    t[7] = torch.where(keep, t[7], torch.finfo(DTYPES[dtype]).min)
    tok[8, 0], tok[9, 1] = -5, V
    tok[10, 0] = 7
    t[10, 0, 7] = -math.inf
    d[10, 0, 7] = -math.inf
    t[11, 2] = math.nan
    check(q, t, tok, draft=d, uniform=u, noise=e, most_unsure=0.2)
    check(q, t, tok, uniform=u, noise=e, most_unsure=0.2)
    check(q, t, tok, most_unsure=0.2)
    # the same sequences a few at a time, which one kernel does alone
    whole = q.verify_drafts(t, tok, d, u, e)
    for a in range(0, B, 5):
        part = q.verify_drafts(t[a:a + 5], tok[a:a + 5], d[a:a + 5], u[a:a + 5], e[a:a + 5])
        assert torch.equal(part.accepted, whole.accepted[a:a + 5])


@pytest.mark.parametrize("B", [2, 40])
@pytest.mark.parametrize("V", [257, 9000])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_rows_of_the_lowest_value(q, B, V, dtype):
    """All logits equal, as low (or as high) as the type goes: every token is as
    likely, so that the race goes to the least noise."""
    g = torch.Generator(device="cuda").manual_seed(V)
    e = torch.empty(B, V, device="cuda").exponential_(generator=g)
    tok = torch.zeros((B, 1), dtype=torch.int64, device="cuda")
    u = torch.full((B, 1), 0.5, device="cuda")
    for value in (torch.finfo(DTYPES[dtype]).min, torch.finfo(DTYPES[dtype]).max):
        t = torch.full((B, 2, V), value, dtype=DTYPES[dtype], device="cuda")
        got = q.verify_drafts(t[:, :1], tok[:, :0], None, u[:, :0], e)
        assert got.tokens[:, 0].tolist() == e.argmin(dim=1).tolist()
        # a draft of the same rows is kept, a certain one at 1 / V is not
        got = q.verify_drafts(t, tok, t[:, :1], u, e)
        assert got.accepted.tolist() == [1] * B and got.tokens[:, 1].tolist() == e.argmin(dim=1).tolist()
        got = q.verify_drafts(t, tok, None, u, e)
        assert got.accepted.tolist() == [0] * B
        assert got.tokens[:, 0].tolist() == (e[:, 1:].argmin(dim=1) + 1).tolist()


@pytest.mark.parametrize("B", [3, 24])
def test_far_logits(q, B):
    """Rows whose largest logit lies far from 0, where a logit's neighbours are
    whole numbers apart."""
    V = 9000
    t, d, tok, u, e = problem(B, 2, V, "fp32", B)
    shift = torch.tensor([8e6, -7e6, 1e3], device="cuda").repeat(B // 3)[:, None, None]
    t, d = (t * 4).round() + shift, (d * 4).round() - shift
    check(q, t, tok, draft=d, uniform=u, noise=e)
    check(q, t, tok, uniform=u, noise=e)
    check(q, t, tok)


@pytest.mark.parametrize("B", [8, 24])
@pytest.mark.parametrize("V,pad", [(8200, 0), (9001, 3), (100, 0)])
def test_noise_at_its_ends(q, B, V, pad):
    t, d, tok, u, e = problem(B, 2, V, "bf16", V + B, pad)
    for b in range(0, B, 8):
        e[b, [17, 90, V - 1]] = 0.0           # ratios of infinity: the lowest index
        e[b + 1, 55] = 1e-42                  # a subnormal one
        e[b + 2, ::2] = math.inf              # a ratio of 0: never drawn
        e[b + 3, 1::2] = math.nan
        e[b + 4, ::3] *= -1.0
        e[b + 5] = math.inf
        e[b + 6] *= 1e30
        e[b + 7] *= 1e-30
    check(q, t, tok, draft=d, uniform=u, noise=e, most_unsure=0.2)
    check(q, t, tok, uniform=u, noise=e, most_unsure=0.2)
    none = q.verify_drafts(t, tok, d, u, e).tokens[5::8]
    assert all(-1 in row for row in none.tolist())
