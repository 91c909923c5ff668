"""Log probabilities, entropy and top alternatives against 64-bit arithmetic.

Bounds (u = 2^-24, D = the row's range of finite logits, at most 104 where a
term still counts): each exponential is off by 4 u from the instruction and by
at most D u from its argument, a thread's running sums by one u per term and
the joining trees by 32 u, so the sums are off by
    R = (4 + 2 min(D, 104) + V / 128 + 32) u
relatively; a log probability by R plus 4 u of its size (and of D), the
entropy by R (2 + 2 ln V + 2 H)."""
import math

import numpy as np
import pytest
import torch

from gpu_util import qg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
INF = float("inf")


def _reference(x, tokens, k):
    """x: float64 [M, V] on the CPU."""
    M, V = x.shape
    lp = np.full((M, V), -np.inf)
    H = np.zeros(M)
    for m in range(M):
        r = x[m]
        if np.isnan(r).any() or (r == np.inf).any():
            lp[m] = np.nan
            H[m] = np.nan
            continue
        mx = r.max()
        if mx == -np.inf:
            continue
        d = r - mx
        s = np.exp(d).sum()
        lp[m] = d - math.log(s)
        p = np.exp(lp[m])
        H[m] = -(p[p > 0] * lp[m][p > 0]).sum()
    key = np.where(np.isnan(x), np.inf, x)
    ids = np.empty((M, k), np.int64)
    for m in range(M):
        order = np.lexsort((np.arange(V), -key[m], ~np.isnan(x[m])))
        ids[m] = order[:k]
    tok = np.array([[lp[m, t] if 0 <= t < V else -np.inf for t in tokens[m]] for m in range(M)])
    return lp, tok.reshape(M, -1), H, ids


def _check(logits, tokens, k):
    q = qg()
    M, V = logits.shape
    r = q.logprobs(logits, torch.from_numpy(tokens).cuda(), top_k=k, entropy=True)
    assert q.last_device_status() == 0
    x = logits.double().cpu().numpy()
    lp, tok, H, ids = _reference(x, tokens, k)
    fin = np.where(np.isfinite(x), x, np.nan)
    with np.errstate(all="ignore"):
        D = np.nan_to_num(np.nanmax(np.where(np.isfinite(fin), fin, -1e300), axis=1) -
                          np.nanmin(np.where(np.isfinite(fin), fin, 1e300), axis=1), nan=0.0)
    R = (4 + 2 * np.minimum(np.maximum(D, 0), 104) + V / 128 + 32) * U

    def close(got, want, tol):
        same = (got == want) | (np.isnan(got) & np.isnan(want))
        with np.errstate(all="ignore"):
            ok = same | (np.isfinite(want) & (np.abs(got - want) <= tol))
        assert ok.all(), (np.argwhere(~ok)[:4].tolist(), got[~ok][:4], want[~ok][:4])

    with np.errstate(all="ignore"):
        got = r.token_logprobs.double().cpu().numpy().reshape(M, -1)
        close(got, tok, R[:, None] + 4 * U * np.abs(tok))
        close(r.entropy.double().cpu().numpy(), H, R * (2 + 2 * math.log(max(V, 2)) + 2 * np.abs(H)))
        if k:
            assert np.array_equal(r.top_ids.cpu().numpy(), ids)
            want = np.take_along_axis(lp, ids, axis=1)
            close(r.top_logprobs.double().cpu().numpy(), want, R[:, None] + 4 * U * np.abs(want))
    return r


def _logits(M, V, dtype, seed, pad=0, offset=0, scale=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((M * (V + pad) + offset,), 1e4, dtype=DT[dtype], device="cuda")   # a large value if read by mistake
    rows = buf[offset:].view(M, V + pad)[:, :V]
    rows.copy_(torch.randn(M, V, generator=g, device="cuda") * scale)
    return rows


def _tokens(M, T, V, seed=1):
    return np.random.default_rng(seed).integers(0, V, size=(M, T))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,V,T,k,pad,offset", [
    (1, 1, 1, 1, 0, 0), (1, 2, 1, 2, 0, 1), (3, 7, 2, 7, 3, 1), (2, 31, 1, 31, 0, 3), (5, 33, 1, 32, 0, 1),
    (1, 1000, 1, 5, 0, 0), (7, 1003, 3, 20, 0, 1), (4, 4099, 1, 8, 13, 5), (33, 32768, 1, 5, 0, 0),
    (2, 50021, 4, 20, 27, 7), (1, 131072, 1, 20, 0, 0), (9, 100003, 1, 32, 0, 3), (300, 2050, 1, 1, 2, 1),
    (700, 517, 1, 3, 0, 0),
])
def test_matches_64_bits(dtype, M, V, T, k, pad, offset):
    _check(_logits(M, V, dtype, M + V, pad, offset), _tokens(M, T, V), k)


@pytest.mark.parametrize("dtype", list(DT))
def test_masked_and_empty_rows(dtype):
    """Masks as -inf: all but one token, fewer tokens than alternatives asked,
    scattered, one contiguous run, and nothing left."""
    V = 20011
    x = _logits(8, V, dtype, 5)
    keep = torch.zeros(8, V, dtype=torch.bool, device="cuda")
    keep[0, 777] = True
    keep[1, [3, 9000, 20010]] = True
    keep[2, ::97] = True
    keep[3, 4096:4200] = True
    keep[5] = True
    keep[5, :8192] = False
    keep[6, :5] = True
    keep[7] = torch.rand(V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) < 0.5
    x.masked_fill_(~keep, -INF)
    tokens = _tokens(8, 3, V)
    tokens[0, 0], tokens[1, 1], tokens[4, 0] = 777, 9000, 0
    r = _check(x, tokens, 20)
    assert r.top_ids[4].tolist() == list(range(20)) and float(r.entropy[4]) == 0.0
    assert r.top_ids[0, :3].tolist() == [777, 0, 1]


@pytest.mark.parametrize("dtype", list(DT))
def test_lowest_value_masks(dtype):
    """Masks as the type's lowest value; a row of nothing else is uniform."""
    V = 5003
    low = torch.finfo(DT[dtype]).min
    x = _logits(4, V, dtype, 6)
    x[0] = low
    x[1, 10:] = low
    x[2, ::2] = low
    x[3] = low
    x[3, 5:4000] = -INF
    r = _check(x, _tokens(4, 2, V), 12)
    assert abs(float(r.entropy[0]) - math.log(V)) < 1e-4
    assert r.top_ids[3].tolist()[:6] == [0, 1, 2, 3, 4, 4000]


@pytest.mark.parametrize("dtype", list(DT))
def test_ties_go_to_the_lower_index(dtype):
    V = 30011
    x = _logits(5, V, dtype, 8)
    x[0] = 1.5
    x[1] = torch.arange(V, device="cuda") % 3
    x[2, 100::64] = 30.0
    x[3] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0)
    x[4] = (x[4] * 2).round() / 2
    _check(x, _tokens(5, 1, V), 32)


@pytest.mark.parametrize("dtype", list(DT))
def test_nan_and_infinity(dtype):
    V = 9001
    x = _logits(5, V, dtype, 9)
    x[0, 17] = float("nan")
    x[1, 8000] = INF
    x[2, 3] = INF
    x[2, 4000] = float("nan")
    x[2, 9000] = -float("nan")
    x[3, 0] = -INF
    tokens = _tokens(5, 2, V)
    tokens[0, 0] = -1
    tokens[4] = (V, -100)
    r = _check(x, tokens, 4)
    assert r.top_ids[2].tolist()[:3] == [4000, 9000, 3]
    assert r.token_logprobs[4].tolist() == [-INF, -INF]
    assert float(r.token_logprobs[0, 0]) == -INF


@pytest.mark.parametrize("shift", [3e3, -4e4, 1e9, -3e12, 1e30])
def test_large_offsets(shift):
    """A row far from zero: its differences are what 32 bits hold of them."""
    V = 4001
    x = _logits(3, V, "fp32", 10) + shift
    _check(x, _tokens(3, 1, V), 10)


def test_peaked_and_rising_rows():
    """A maximum that keeps moving (ascending logits), and one token that
    holds all the probability."""
    V = 70000
    x = torch.empty(3, V, device="cuda")
    x[0] = torch.linspace(-50, 50, V, device="cuda")
    x[1] = torch.linspace(50, -50, V, device="cuda")
    x[2] = 0.0
    x[2, 61234] = 90.0
    _check(x, np.array([[V - 1, 0], [0, 5], [61234, 1]]), 20)


def test_more_rows_than_64_thousand():
    V = 40
    x = _logits(70001, V, "bf16", 12)
    q = qg()
    r = q.logprobs(x, top_k=2)
    ref = torch.log_softmax(x.double(), dim=1)
    top = ref.max(dim=1).values
    assert float((r.top_logprobs[:, 0].double() - top).abs().max()) < 1e-5
    assert r.entropy is None and r.token_logprobs is None


def test_offsets_past_32_bits():
    """Rows whose elements lie beyond 2^32 bytes and 2^31 elements."""
    V = 131075
    M = (1 << 31) // V + 3
    x = torch.zeros(M, V, dtype=torch.bfloat16, device="cuda")
    x[M - 1, V - 1] = 3.0
    x[M - 2, 5] = 2.0
    q = qg()
    r = q.logprobs(x, torch.full((M,), V - 1, dtype=torch.int64, device="cuda"), top_k=1, entropy=True)
    assert r.top_ids[M - 1, 0].item() == V - 1 and r.top_ids[M - 2, 0].item() == 5 and r.top_ids[0, 0].item() == 0
    want = 3.0 - math.log(V - 1 + math.exp(3.0))
    assert abs(r.token_logprobs[M - 1].item() - want) < 1e-4
    del x
    torch.cuda.empty_cache()


def test_parts_on_their_own_and_other_streams():
    q = qg()
    V = 33333
    x = _logits(6, V, "bf16", 13)
    tok = torch.from_numpy(_tokens(6, 1, V)).cuda()
    full = q.logprobs(x, tok, top_k=7, entropy=True)
    assert torch.equal(q.logprobs(x, tok[:, 0]).token_logprobs, full.token_logprobs[:, 0])
    assert torch.equal(q.logprobs(x, entropy=True).entropy, full.entropy)
    part = q.logprobs(x, top_k=7)
    assert torch.equal(part.top_ids, full.top_ids) and torch.equal(part.top_logprobs, full.top_logprobs)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = q.logprobs(x, tok, top_k=7, entropy=True)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, full))
    # strided tokens and an expanded column of them
    wide = torch.zeros(6, 5, dtype=torch.int64, device="cuda")
    wide[:, 2] = tok[:, 0]
    assert torch.equal(q.logprobs(x, wide[:, 2]).token_logprobs, full.token_logprobs[:, 0])
    same = torch.full((1, 1), 9, dtype=torch.int64, device="cuda").expand(6, 3)
    one = q.logprobs(x, torch.full((6,), 9, dtype=torch.int64, device="cuda")).token_logprobs
    assert torch.equal(q.logprobs(x, same).token_logprobs, one[:, None].expand(6, 3))


def test_results_do_not_depend_on_the_batch():
    """The same row gives the same bits alone and among others."""
    q = qg()
    x = _logits(40, 32768, "bf16", 14)
    a = q.logprobs(x, top_k=5, entropy=True)
    again = q.logprobs(x, top_k=5, entropy=True)
    assert all(torch.equal(u, v) for u, v in zip(a[1:], again[1:]))
    ids = q.logprobs(x[7:8], top_k=5).top_ids
    assert torch.equal(ids, a.top_ids[7:8])


def test_refusals():
    q = qg()
    x = torch.zeros(3, 16, device="cuda")
    for bad in (lambda: q.logprobs(x.double()), lambda: q.logprobs(x.t()), lambda: q.logprobs(x.cpu(), entropy=True),
                lambda: q.logprobs(x, torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: q.logprobs(x, torch.zeros(4, dtype=torch.int64, device="cuda")),
                lambda: q.logprobs(x, torch.zeros(3, dtype=torch.int64))):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for k in (17, 33):
        with pytest.raises(q.QgemmError) as e:
            q.logprobs(torch.zeros(3, 40 if k == 33 else 16, device="cuda"), top_k=k)
        assert e.value.code == 2
    with pytest.raises(q.QgemmError):
        q.logprobs(x, top_k=-1)
    assert q.logprobs(torch.zeros(0, 16, device="cuda"), top_k=2).top_ids.shape == (0, 2)


@pytest.mark.parametrize("dtype", list(DT))
def test_entropy_of_a_certain_token(dtype):
    """One logit far above the others: the entropy is 0 within its bound
    (R (2 + 2 ln V), D counted as 104) and never negative."""
    q = qg()
    V = 5003
    rng = np.random.default_rng(17)
    x = rng.uniform(-2, 2, (64, V)) + rng.uniform(-300, 300, (64, 1))
    x[np.arange(64), rng.integers(0, V, 64)] += rng.uniform(110, 400, 64)
    H = q.logprobs(torch.from_numpy(x).to(DT[dtype]).cuda(), entropy=True).entropy.double().cpu().numpy()
    R = (4 + 2 * 104 + V / 128 + 32) * U
    assert (H >= 0).all() and (H <= R * (2 + 2 * math.log(V))).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,V,T,k,pad", [
    (1700, 9001, 2, 7, 3), (800, 20011, 1, 32, 0), (2300, 2003, 1, 20, 5), (4000, 517, 3, 1, 0),   # several rows a CTA
    (160, 131075, 1, 20, 0), (153, 200000, 1, 32, 8), (460, 70001, 1, 8, 1),                       # many turns a row
    (150, 40009, 1, 20, 0), (70, 40009, 1, 32, 1), (30, 65539, 1, 20, 0), (12, 131072, 1, 32, 0),  # rows in 2 to 16 parts
    (17, 2003, 130, 5, 0), (900, 1003, 129, 2, 1),                                                 # more tokens than threads
])
def test_many_rows_turns_and_parts(dtype, M, V, T, k, pad):
    """Against 64 bits on the device, with the bounds above; logits on a coarse
    grid in every other row, so that the alternatives tie across threads and parts."""
    x = _logits(M, V, dtype, 3 * M + V, pad)
    x[::2] = torch.round(x[::2].float() * 2).to(DT[dtype]) / 2
    x[1::7, :: 3] = -INF
    g = torch.Generator(device="cuda").manual_seed(M)
    tok = torch.randint(-1, V + 1, (M, T), generator=g, device="cuda")
    q = qg()
    r = q.logprobs(x, tok, top_k=k, entropy=True)
    assert q.last_device_status() == 0
    for m0 in range(0, M, 200):
        d = x[m0:m0 + 200].double()
        lp = torch.log_softmax(d, dim=1)
        H = torch.special.entr(lp.exp()).sum(dim=1)
        low = torch.where(d == -INF, d.amax(dim=1, keepdim=True), d).amin(dim=1)
        R = ((4 + 2 * (d.amax(dim=1) - low).clamp(max=104) + V / 128 + 32) * U)[:, None]
        order = torch.sort(d, dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(r.top_ids[m0:m0 + 200], order)
        t = tok[m0:m0 + 200]
        ref = lp.gather(1, t.clamp(0, V - 1)).masked_fill((t < 0) | (t >= V), -INF)
        for got, want in ((r.top_logprobs[m0:m0 + 200], lp.gather(1, order)), (r.token_logprobs[m0:m0 + 200], ref)):
            none = want == -INF
            assert torch.equal(got.double() == -INF, none)
            err = (got.double() - want).masked_fill(none, 0).abs()
            assert bool((err <= R + 4 * U * (want.masked_fill(none, 0).abs() + (d.amax(dim=1) - low)[:, None])).all())
        err = (r.entropy[m0:m0 + 200].double() - H).abs()
        assert bool((err <= R[:, 0] * (2 + 2 * math.log(V) + 2 * H)).all())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("mask", [-INF, -1e9, "lowest", 0.5], ids=["inf", "1e9", "lowest", "tied"])
@pytest.mark.parametrize("M,V,k", [(3, 131072, 8), (1, 20011, 32), (40, 40009, 20), (200, 9001, 5), (900, 5003, 7)])
def test_few_tokens_left(dtype, mask, M, V, k):
    """Masks that leave 0 to 40 tokens of a row, fewer than the alternatives
    asked for in most: the rest are masked ones, lower index first (rows with
    nothing left among them).  Bounds as above, D over the tokens left."""
    if mask == "lowest":
        mask = torch.finfo(DT[dtype]).min
    if mask == -1e9 and dtype == "fp16":
        mask = -6e4
    g = torch.Generator(device="cuda").manual_seed(M + V + k)
    x = torch.full((M, V), mask, dtype=DT[dtype], device="cuda")
    left = torch.zeros((M, V), dtype=torch.bool, device="cuda")
    for m in range(M):
        n = m % 41
        left[m, torch.randperm(V, generator=g, device="cuda")[:n]] = True
    x[left] = torch.randn(int(left.sum()), generator=g, device="cuda").to(DT[dtype])
    if V % 2:
        x[:, V - 1] = x[:, 0]   # the last logit ties with the first
    tok = torch.randint(0, V, (M, 2), generator=g, device="cuda")
    q = qg()
    r = q.logprobs(x, tok, top_k=k, entropy=True)
    assert q.last_device_status() == 0
    d = x.double()
    lp = torch.where((d.amax(dim=1) == -INF)[:, None], torch.full_like(d, -INF), torch.log_softmax(d, dim=1))
    order = torch.sort(d, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.top_ids, order)
    R = (4 + 2 * 16 + V / 128 + 32) * U   # the tokens left and 0.5 lie within 16 of each other
    for got, want in ((r.top_logprobs, lp.gather(1, order)), (r.token_logprobs, lp.gather(1, tok))):
        none = want == -INF
        assert torch.equal(got.double() == -INF, none)
        err = (got.double() - want).masked_fill(none, 0).abs()
        assert bool((err <= R + 4 * U * want.masked_fill(none, 0).abs()).all())
    H = torch.where(d.amax(dim=1) == -INF, 0.0, torch.special.entr(lp.exp()).sum(dim=1))
    assert bool(((r.entropy.double() - H).abs() <= R * (2 + 2 * math.log(V) + 2 * H)).all())


@pytest.mark.parametrize("dtype", list(DT))
def test_nan_among_ties(dtype):
    """Rows of ties with a NaN somewhere: NaN throughout, and first in order."""
    V, k = 40009, 9
    x = torch.zeros((6, V), dtype=DT[dtype], device="cuda")
    x[:, 7] = 1.0
    at = [0, 5, 20000, 39999, 40008, 12345]
    for m, v in enumerate(at):
        x[m, v] = float("nan")
    r = qg().logprobs(x, torch.zeros((6, 1), dtype=torch.int64, device="cuda"), top_k=k, entropy=True)
    assert bool(torch.isnan(r.entropy).all()) and bool(torch.isnan(r.token_logprobs).all())
    for m, v in enumerate(at):
        rest = [i for i in range(k + 2) if i not in (7, v)]
        assert r.top_ids[m].tolist() == ([v] + [7] + rest)[:k]


def test_strided_tokens_on_another_stream():
    """Expanded, transposed and sliced tokens with stream=: their copy is made
    on that stream.  The current stream is kept busy, so that work left to it
    would come too late; the tokens' memory was used for other tokens before."""
    q = qg()
    V, M = 33333, 6
    x = _logits(M, V, "bf16", 15)
    tok = torch.from_numpy(_tokens(M, 3, V)).cuda()
    forms = [tok[:, :1].expand(M, 3), tok.t().contiguous().t(), tok[:1].expand(M, 3), tok[:, 0]]
    expect = [q.logprobs(x, f.contiguous(), top_k=7, entropy=True) for f in forms]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    busy = torch.zeros(1 << 28, device="cuda")
    for stream in (st, st.cuda_stream):
        for f, want in zip(forms, expect):
            for _ in range(8):
                busy.add_(1.0)
            got = q.logprobs(x, f, top_k=7, entropy=True, stream=stream)
            st.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    assert q.last_device_status() == 0


@pytest.mark.parametrize("dtype", list(DT))
def test_no_log_probability_is_above_zero(dtype):
    """Rows held by one token, at offsets of every kind, whole and split over
    CTAs: its log probability is 0 within the bound and not above it, so that
    exp gives no more than 1 and log1p(-exp) no NaN."""
    q = qg()
    rng = np.random.default_rng(23)
    for M, V in ((64, 5003), (500, 700), (3, 70001), (1, 131072)):
        x = rng.uniform(-2, 2, (M, V)) + rng.uniform(-300, 300, (M, 1))
        ids = rng.integers(0, V, M)
        x[np.arange(M), ids] += rng.uniform(30, 400, M)
        tok = torch.from_numpy(ids).cuda()
        r = q.logprobs(torch.from_numpy(x).to(DT[dtype]).cuda(), tok, top_k=2, entropy=True)
        R = (4 + 2 * 104 + V / 128 + 32) * U
        for lp in (r.token_logprobs, r.top_logprobs[:, 0]):
            assert bool((lp <= 0).all()) and bool((lp >= -R).all())
        assert torch.equal(r.top_ids[:, 0], tok) and bool((r.top_logprobs[:, 1] <= 0).all())


def test_a_row_alone_and_among_others():
    """The rows of a batch that is split over more or fewer CTAs a row give the
    same alternatives, and values within the sums' bound of one another (their
    order, and so their last bits, depend on the number of rows)."""
    q = qg()
    V = 32768
    x = _logits(400, V, "bf16", 14)
    tok = torch.from_numpy(_tokens(400, 1, V)).cuda()
    whole = q.logprobs(x, tok, top_k=5, entropy=True)
    R = (4 + 2 * 104 + V / 128 + 32) * U
    for m, n in ((0, 1), (7, 8), (100, 140), (0, 160)):
        part = q.logprobs(x[m:n], tok[m:n], top_k=5, entropy=True)
        assert torch.equal(part.top_ids, whole.top_ids[m:n])
        for a, b in ((part.token_logprobs, whole.token_logprobs[m:n]), (part.top_logprobs, whole.top_logprobs[m:n])):
            assert bool(((a - b).abs() <= 2 * (R + 4 * U * b.abs())).all())
        H = whole.entropy[m:n]
        assert bool(((part.entropy - H).abs() <= 2 * R * (2 + 2 * math.log(V) + 2 * H)).all())
