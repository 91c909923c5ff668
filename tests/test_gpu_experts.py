"""The operators of a layer of experts on the GPU against plain implementations
in 64 bits: router, row quantiser, grouped W8A8 GEMM, combination.

Tolerances.  A rounding to a type is off by at most half a step (bf16 2^-8,
fp16 2^-11, e4m3 2^-4 of the value, or half the smallest step).  FP32 sums of n
terms: n roundings of at most 2^-24 of the sum of magnitudes; for the GEMM the
library's rule, 32 2^-24 of it, counts them (the tensor core adds 32 products at a
time, 4 times a block, and the fold has two roundings a block whose errors
are of both signs)."""
import math

import numpy as np
import pytest
import torch

from gpu_util import qg

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module")
def q():
    return qg()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ----------------------------------------------------------------- router
def route_reference(x, k, score, bias, renormalize, scale):
    """In numpy and 64 bits, token by token."""
    M, E = x.shape
    experts = np.full((M, k), -1, dtype=np.int64)
    weights = np.zeros((M, k))
    for m in range(M):
        row = x[m]
        if np.isnan(row).any() or np.isposinf(row).any():
            weights[m] = np.nan
            continue
        live = ~np.isneginf(row)
        if not live.any():
            continue
        s = np.zeros(E)
        if score == "softmax":
            s[live] = np.exp(row[live] - row[live].max())
            s /= s.sum()
        else:
            s[live] = 1 / (1 + np.exp(-row[live]))
        by = row.copy() if bias is None else s + bias
        by[~live] = -np.inf
        by[np.isnan(by)] = -np.inf
        order = np.lexsort((np.arange(E), -by))
        order = [e for e in order if by[e] > -np.inf][:k]
        experts[m, :len(order)] = order
        w = s[order]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else w * 0
        weights[m, :len(order)] = w * scale
    return experts, weights


def order_reference(experts, E):
    flat = experts.reshape(-1)
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    rows = np.full(flat.shape, -1, dtype=np.int64)
    at = offsets[:-1].copy()
    for i, e in enumerate(flat):
        if e >= 0:
            rows[i] = at[e]
            at[e] += 1
    return offsets, rows.reshape(experts.shape)


def check_route(q, logits, k, **kw):
    r = q.moe_route(logits, k, **kw)
    bias = kw.get("bias")
    E = logits.shape[1]
    experts, weights = route_reference(logits.double().cpu().numpy(), k, kw.get("score", "softmax"),
                                       None if bias is None else bias.double().cpu().numpy(),
                                       kw.get("renormalize", True), kw.get("scale", 1.0))
    assert np.array_equal(r.experts.cpu().numpy(), experts)
    got = r.weights.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(weights))
    # an exponential and a reciprocal of 2 units each, a sum of up to 1024 terms
    # of one sign (32 a lane, then 5 steps), a division and a product
    tol = 48 * 2.0 ** -24
    assert np.all(np.abs(np.nan_to_num(got - weights)) <= tol * np.abs(np.nan_to_num(weights)) + 1e-37)
    offsets, rows = order_reference(experts, E)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)


@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 8, 2), (3, 33, 8), (16, 128, 8), (64, 64, 6), (65, 256, 8),
                                   (257, 300, 5), (1000, 160, 6), (2433, 256, 8), (4099, 60, 4), (33, 1024, 32),
                                   (7, 32, 32), (6000, 2, 1)])
@pytest.mark.parametrize("score,biased,dtype", [("softmax", False, "fp32"), ("sigmoid", True, "bf16"),
                                                ("softmax", True, "fp16"), ("sigmoid", False, "bf16")])
def test_route(q, M, E, k, score, biased, dtype):
    g = gen(M * 7 + E)
    logits = (torch.randn(M, E, generator=g, device="cuda") * 2).to(DTYPES[dtype])
    bias = torch.randn(E, generator=g, device="cuda") * 0.1 if biased else None
    check_route(q, logits, k, score=score, bias=bias, scale=2.5, renormalize=E % 2 == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_ties_masks_and_bad_rows(q, score, biased):
    E, k, M = 96, 6, 200
    g = gen(5)
    # few distinct values: ties everywhere, lower index first
    logits = torch.randint(-3, 4, (M, E), generator=g, device="cuda").float()
    bias = torch.randint(-1, 2, (E,), generator=g, device="cuda").float() * 0.25 if biased else None
    logits[0] = 0.0
    logits[1] = -math.inf                       # nothing left
    logits[2] = -math.inf
    logits[2, 40:43] = 1.0                      # fewer left than asked for
    logits[3, 7] = math.nan
    logits[4, 95] = math.inf
    logits[5, ::2] = -math.inf
    logits[6] = -1e30                           # finite, however low
    logits[7, :] = torch.linspace(-200, 200, E, device="cuda")
    logits[8] = torch.where(torch.arange(E, device="cuda") % 2 == 0, 0.0, -0.0)
    check_route(q, logits, k, score=score, bias=bias)
    if biased:
        bias[3] = -math.inf
        bias[4] = math.nan
        check_route(q, logits, k, score=score, bias=bias, renormalize=False)


def test_route_scores_nearer_than_32_bits(q):
    """Sums of score and bias that differ by less than an FP32 step: the order of 64 bits."""
    E, k = 64, 32
    x = torch.linspace(-4, 4, E, device="cuda", dtype=torch.float32).repeat(40, 1)
    s = torch.sigmoid(x[0].double())
    bias = (0.9 - s).float()       # every sum is 0.9 to within an FP32 rounding
    check_route(q, x, k, score="sigmoid", bias=bias)
    check_route(q, x, 5, score="sigmoid", bias=bias)


def test_route_strided_and_empty(q):
    g = gen(9)
    wide = torch.randn(50, 100, generator=g, device="cuda")
    check_route(q, wide[:, :64], 4)
    check_route(q, wide[:, 3:60], 4, score="sigmoid")
    r = q.moe_route(wide[:0], 4)
    assert r.experts.shape == (0, 4) and int(r.offsets.abs().sum()) == 0


# ----------------------------------------------------------------- row quantiser
def silu_mul(X):
    g, u = X.double().chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * u


@pytest.mark.parametrize("M,K,k", [(1, 16, 1), (5, 128, 2), (33, 144, 8), (70, 1040, 3), (64, 5120, 8), (3, 17408, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quantize_rows_copies(q, M, K, k, dtype):
    """The codes and scales of quantize_act_e4m3, on the rows asked for."""
    g = gen(M + K)
    X = (torch.randn(M, K + 8, generator=g, device="cuda") * 3).to(DTYPES[dtype])[:, :K]
    X[0, :16] = 0.0
    out_rows = M * k + 3
    rows = torch.randperm(out_rows, generator=g, device="cuda")[:M * k].reshape(M, k).to(torch.int32)
    rows[M // 2, 0] = -1
    if M > 1:
        rows[0, k - 1] = out_rows + 5       # outside: nowhere
    Xq = torch.full((out_rows, K), 0x55, dtype=torch.uint8, device="cuda")
    Xs = torch.full((-(-K // 128), 4 * out_rows), -7.0, device="cuda")
    q.quantize_rows_e4m3(X, rows=rows, Xq=Xq, X_scale=Xs)
    ref_q, ref_s = q.quantize_act_e4m3(X.to(torch.bfloat16))
    if dtype == "fp16":     # the same rule on values that bfloat16 does not hold
        x = torch.zeros((M, Xs.shape[0] * 128), device="cuda")
        x[:, :K] = X.float()
        amax = x.view(M, -1, 128).abs().amax(dim=2)
        # by a tensor: PyTorch divides by a number with its rounded reciprocal
        sc = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), 1.0)
        ref_q = (x.view(M, -1, 128) / sc[:, :, None]).reshape(M, -1)[:, :K].to(torch.float8_e4m3fn).view(torch.uint8)
        ref_s = sc.t()
    want_q = torch.full_like(Xq, 0x55)
    want_s = torch.full_like(Xs, -7.0)
    for m in range(M):
        for r in rows[m].tolist():
            if 0 <= r < out_rows:
                want_q[r] = ref_q[m]
                want_s[:, r] = ref_s[:, m]
    assert torch.equal(Xq, want_q)
    assert torch.equal(Xs, want_s)


@pytest.mark.parametrize("M,K", [(1, 16), (7, 128), (130, 272), (65, 2048), (2, 5120)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("limit", [None, 0, 5])
def test_quantize_rows_gated(q, M, K, dtype, limit):
    g = gen(M * 3 + K)
    X = (torch.randn(M, 2 * K, generator=g, device="cuda") * 4).to(DTYPES[dtype])
    X[M // 2, :K] = -60.0      # a gate that lets nothing through
    num = None if limit is None else torch.tensor([limit], dtype=torch.int32, device="cuda")
    Xq = torch.full((M, K), 0x55, dtype=torch.uint8, device="cuda")
    Xs = torch.full((-(-K // 128), -(-M // 32) * 32), -7.0, device="cuda")
    q.quantize_rows_e4m3(X, gated=True, num_rows=num, Xq=Xq, X_scale=Xs)
    n = M if limit is None else min(M, limit)
    assert bool((Xq[n:] == 0x55).all()) and bool((Xs[:, n:] == -7.0).all())
    if n == 0:
        return
    v = silu_mul(X[:n])
    KB = Xs.shape[0]
    pad = torch.zeros((n, KB * 128), dtype=torch.float64, device="cuda")
    pad[:, :K] = v
    amax = pad.view(n, KB, 128).abs().amax(dim=2)
    s = Xs[:, :n].t().double()
    # exponential: 2^-22 + |g| 2^-24, reciprocal 2^-23, four products: with |g| <= 60, 2^-17.5
    tol = 2.0 ** -17
    assert bool((torch.where(amax > 1e-30, (s * 448 - amax).abs() <= tol * amax, True)).all())
    deq = Xq[:n].view(torch.float8_e4m3fn).double()
    ref = (pad.view(n, KB, 128) / s[:, :, None]).reshape(n, -1)[:, :K]
    off = (deq - ref).abs()
    assert bool((off <= (2.0 ** -4 + tol) * ref.abs() + 2.0 ** -10).all())


# ----------------------------------------------------------------- grouped GEMM
def offsets_of(sizes, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


def grouped_problem(sizes, N, K, seed, extra=0, first=0):
    """Codes, scales and offsets of groups of these sizes; `extra` rows behind the last."""
    g = gen(seed)
    E, R = len(sizes), first + int(sum(sizes)) + extra
    KB = -(-K // 128)
    Xq = (torch.randn(R, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    W = (torch.randn(E, N, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    Xs = torch.rand(KB, -(-max(R, 1) // 32) * 32, generator=g, device="cuda") * 0.01 + 0.005
    Ws = torch.rand(E, -(-N // 128), KB, generator=g, device="cuda") * 2e-4 + 1e-4
    return Xq, Xs, W, Ws, offsets_of(sizes, first)


def grouped_reference(Xq, Xs, W, Ws, off):
    """(Y, sum of magnitudes) in 64 bits; rows of no expert are NaN."""
    R, K = Xq.shape
    N = W.shape[1]
    y = torch.full((R, N), math.nan, dtype=torch.float64, device="cuda")
    mass = torch.zeros_like(y)
    o = off.tolist()
    over_k = torch.arange(K, device="cuda") // 128
    over_n = torch.arange(N, device="cuda") // 128
    for e in range(W.shape[0]):
        a, b = o[e], o[e + 1]
        if b > a:
            x = Xq[a:b].double() * Xs[:, a:b].t().double()[:, over_k]
            w = W[e].double() * Ws[e].double()[over_n][:, over_k]
            y[a:b] = x @ w.t()
            mass[a:b] = x.abs() @ w.abs().t()
    return y, mass


def check_grouped(q, sizes, N, K, dtype, seed=1, extra=0, first=0, pad_y=0, pad_x=0):
    Xq, Xs, W, Ws, off = grouped_problem(sizes, N, K, seed, extra, first)
    R = Xq.shape[0]
    if pad_x:
        wide = torch.zeros((R, K + pad_x), dtype=torch.uint8, device="cuda")
        wide[:, :K] = Xq.view(torch.uint8)
        x = wide[:, :K]
    else:
        x = Xq
    Y = torch.full((R, N + pad_y), -1234.0, dtype=DTYPES[dtype], device="cuda")
    q.qgemm_w8a8_grouped(x, Xs, W, Ws, off, Y=Y[:, :N])
    assert q.last_device_status() == 0
    ref, mass = grouped_reference(Xq, Xs, W, Ws, off)
    live = ~torch.isnan(ref[:, 0]) if N else torch.zeros(R, dtype=torch.bool, device="cuda")
    assert bool((Y[~live] == -1234.0).all())
    assert bool((Y[:, N:] == -1234.0).all())
    y = Y[live][:, :N].double()
    tol = HALF_STEP[dtype] * ref[live].abs() + (32 + 1) * 2.0 ** -24 * mass[live]
    bad = (y - ref[live]).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), bad.numel(), torch.nonzero(bad)[:5].tolist())
    return Y


@pytest.mark.parametrize("sizes", [[1], [0, 3, 0, 1, 0], [16, 17, 1, 15], [5] * 40, [0] * 60 + [2] + [0] * 67],
                         ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("N,K", [(128, 128), (256, 1024), (1003, 1040), (96, 16), (640, 272)])
def test_grouped_few_rows(q, sizes, N, K):
    check_grouped(q, sizes, N, K, "bf16")


@pytest.mark.parametrize("sizes", [[40, 0, 64, 65, 1, 130], [33] * 9, [200, 1, 1, 1, 1]], ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("N,K", [(128, 256), (1003, 1040), (2048, 400)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_grouped_some_rows(q, sizes, N, K, dtype):
    check_grouped(q, sizes, N, K, dtype)


@pytest.mark.parametrize("sizes", [[256, 255, 257, 1, 0, 31, 32, 33, 500], [1000], [64, 640, 0, 90]],
                         ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("N,K", [(256, 512), (384, 128), (1003, 1040), (2048, 2048)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_grouped_many_rows(q, sizes, N, K, dtype):
    check_grouped(q, sizes, N, K, dtype)


@pytest.mark.parametrize("sizes", [[3, 1], [50, 60], [300, 200]], ids=lambda s: f"{max(s)}")
def test_grouped_leaves_other_rows(q, sizes):
    """Rows in front of the first group and behind the last, and strides."""
    check_grouped(q, sizes, 264, 528, "bf16", extra=37, first=5, pad_y=8, pad_x=32)
    check_grouped(q, sizes, 261, 528, "fp16", extra=37, first=5, pad_y=3, pad_x=16)
    check_grouped(q, sizes, 261, 528, "fp32", extra=1, first=1, pad_y=3)


@pytest.mark.parametrize("rows", [4, 100, 700])
def test_grouped_nothing_routed(q, rows):
    Xq, Xs, W, Ws, off = grouped_problem([rows, 0], 256, 256, 3)
    Y = torch.full((rows, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    q.qgemm_w8a8_grouped(Xq, Xs, W, Ws, torch.zeros(3, dtype=torch.int32, device="cuda"), Y=Y)
    assert q.last_device_status() == 0 and bool((Y == 5.0).all())


@pytest.mark.parametrize("raw,meant", [([0, 10, 5, 20], [0, 10, 10, 20]), ([-7, 10, 30, 99], [0, 10, 30, 40]),
                                       ([2, 50, 3, 4], [2, 40, 40, 40])])
def test_grouped_offsets_out_of_order(q, raw, meant):
    """Offsets that are not ascending or not within the rows are taken as the nearest that are."""
    Xq, Xs, W, Ws, _ = grouped_problem([20, 10, 10], 256, 256, 3)
    Y = torch.full((40, 256), -1234.0, dtype=torch.float32, device="cuda")
    q.qgemm_w8a8_grouped(Xq, Xs, W, Ws, torch.tensor(raw, dtype=torch.int32, device="cuda"), Y=Y)
    assert q.last_device_status() == 0
    Z = torch.full((40, 256), -1234.0, dtype=torch.float32, device="cuda")
    q.qgemm_w8a8_grouped(Xq, Xs, W, Ws, torch.tensor(meant, dtype=torch.int32, device="cuda"), Y=Z)
    assert torch.equal(Y, Z)


def test_grouped_equals_ungrouped(q):
    """One expert: within two roundings of the ungrouped kernel's result."""
    Xq, Xs, W, Ws, off = grouped_problem([200], 512, 1024, 4)
    Y = q.qgemm_w8a8_grouped(Xq, Xs, W, Ws, off)
    Z = q.qgemm_w8a8_block(Xq, Xs, W[0], Ws[0])
    assert bool(((Y.double() - Z.double()).abs() <= 2.0 ** -7 * Z.double().abs() + 1e-2).all())


def test_grouped_no_columns_of_k(q):
    Y = torch.full((10, 33), 3.0, dtype=torch.bfloat16, device="cuda")
    e = lambda *s, dtype=torch.uint8: torch.empty(s, dtype=dtype, device="cuda")   # noqa: E731
    q.qgemm_w8a8_grouped(e(10, 0), e(0, 32, dtype=torch.float32), e(2, 33, 0), e(2, 1, 0, dtype=torch.float32),
                         torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda"), Y=Y)
    assert bool((Y[:8] == 0).all()) and bool((Y[8:] == 3.0).all())


# ----------------------------------------------------------------- combination
@pytest.mark.parametrize("M,K,k", [(1, 8, 1), (5, 1003, 3), (64, 5120, 8), (129, 264, 9), (3, 17408, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
def test_combine(q, M, K, k, dtype, residual):
    g = gen(M + K + k)
    R = M * k
    Y = torch.randn(R, K, generator=g, device="cuda").to(DTYPES[dtype])
    rows = torch.randperm(R, generator=g, device="cuda").reshape(M, k).to(torch.int32)
    rows[0, 0] = -1
    if M > 1:
        rows[1, 0] = R          # outside: zeros
    w = torch.rand(M, k, generator=g, device="cuda")
    res = torch.randn(M, K, generator=g, device="cuda").to(DTYPES[dtype]) if residual else None
    out = q.moe_combine(Y, rows, w, residual=res)
    at = rows.long().clamp(0, R - 1)
    live = ((rows >= 0) & (rows < R)).double()[:, :, None]
    terms = Y.double()[at] * w.double()[:, :, None] * live
    ref = terms.sum(dim=1) + (res.double() if residual else 0)
    mass = terms.abs().sum(dim=1) + (res.double().abs() if residual else 0)
    assert bool(((out.double() - ref).abs() <= HALF_STEP[dtype] * ref.abs() + (k + 2) * 2.0 ** -24 * mass).all())
    if residual:     # in place
        again = q.moe_combine(Y, rows, w, residual=res, out=res)
        assert again.data_ptr() == res.data_ptr() and torch.equal(again, out)


def test_combine_nan_weights_show(q):
    Y = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([[0, 1], [-1, -1], [-1, 2]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.5], [math.nan, math.nan], [0.0, 0.25]], device="cuda")
    out = q.moe_combine(Y, rows, w).float()
    assert bool((out[0] == 1).all()) and bool(out[1].isnan().all()) and bool((out[2] == 0.25).all())


def test_combine_strides(q):
    g = gen(2)
    Y = torch.randn(12, 100, generator=g, device="cuda")
    rows = torch.arange(12, dtype=torch.int32, device="cuda").reshape(6, 2)
    w = torch.rand(6, 2, generator=g, device="cuda")
    out = torch.full((6, 80), 9.0, device="cuda")
    q.moe_combine(Y[:, 3:67], rows, w, out=out[:, 1:65])
    ref = (Y[:, 3:67].double().reshape(6, 2, 64) * w.double()[:, :, None]).sum(dim=1)
    assert bool(((out[:, 1:65].double() - ref).abs() <= 2.0 ** -22 * ref.abs() + 1e-6).all())
    assert bool((out[:, 0] == 9).all()) and bool((out[:, 65:] == 9).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_chosen_scores_far_from_one(q, dtype, score):
    """Renormalized weights are ratios, however small the scores are: a bias keeps the
    largest logit out, and the sigmoids of the others are below what 32 bits hold."""
    M, E, k = 40, 50, 5
    g = gen(12)
    logits = torch.randn(M, E, generator=g, device="cuda") * 3
    logits -= torch.tensor([0.0, 55.0, 62.0, 90.0, 105.0, 400.0, 600.0, 2000.0], device="cuda").repeat(M // 8)[:, None]
    logits[:, 0] = 50.0
    bias = torch.zeros(E, device="cuda")
    bias[0] = -math.inf
    check_route(q, logits.to(DTYPES[dtype]), k, score=score, bias=bias)
    check_route(q, logits[:, 1:].to(DTYPES[dtype]), k, score=score, scale=2.5)


def test_workspaces_of_calls_with_counters_stay_clean(q):
    """One Workspace for scratch memory and for a GEMM whose workspace has to be zero
    before its first use."""
    ws = q.Workspace()
    M, E = 20000, 1024
    logits = torch.randn(M, E, device="cuda")
    a, b = q.moe_route(logits, 4, workspace=ws), q.moe_route(logits, 4)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    B, G, V = 2000, 4, 8192
    target = torch.randn(B, G + 1, V, device="cuda").to(torch.bfloat16)
    tok = target[:, :G].float().argmax(dim=2)
    q.verify_drafts(target, tok, workspace=ws)
    scratch = ws.buf
    assert scratch.numel() >= B * (2 * G + 1) * (V // 2048) * 8
    buf = ws.get(1 << 16)
    assert buf.data_ptr() != scratch.data_ptr() and not bool(buf.any())
    with pytest.raises(ValueError):
        q.moe_route(logits, 4, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(q.QgemmError):
        q.moe_route(logits, 4, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K", [128, 208, 3696])
def test_quantize_zeros_of_either_sign(q, dtype, K):
    """Codes of -0 are -0's, in blocks with and without other values."""
    M = 50
    g = gen(K)
    X = torch.randn(M, K, generator=g, device="cuda")
    zero = torch.where(torch.rand(M, K, generator=g, device="cuda") < 0.5, 0.0, -0.0)
    X = torch.where(torch.rand(M, K, generator=g, device="cuda") < 0.3, zero, X)
    X[::3, :128] = zero[::3, :128]
    X = X.to(DTYPES[dtype])
    Xq, Xs = q.quantize_rows_e4m3(X)
    want_q, want_s = q.quantize_act_e4m3(X) if dtype == "bf16" else (None, None)
    blocks = X.float().split(128, dim=1)
    scale = torch.stack([torch.where(b.abs().amax(dim=1) > 0, b.abs().amax(dim=1) / torch.tensor(448.0, device="cuda"), 1.0)
                         for b in blocks])
    codes = torch.cat([(b / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8) for b, s in zip(blocks, scale)], dim=1)
    assert torch.equal(Xq, codes) and torch.equal(Xs[:, :M], scale)
    if want_q is not None:
        assert torch.equal(Xq, want_q) and torch.equal(Xs[:, :M], want_s[:, :M])


# (rows of a tile, sizes, N, K): every form of the grouped GEMM, on groups that fill a
# tile, end inside one, and hold nothing
FORMS = [(16, [5, 0, 16, 17, 1, 9, 40], 1003, 1040), (16, [3] * 40, 264, 528), (16, [5, 0, 16, 17, 1, 9, 40], 96, 144),
         (32, [40, 33, 1, 0, 32, 31] * 4, 1003, 1040), (32, [40, 33, 1, 0, 32, 31] * 4, 640, 2048),
         (64, [60, 64, 65, 1, 0, 130, 33, 40] * 6, 1003, 1040), (64, [60, 64, 65, 1, 0, 130, 33, 40] * 6, 264, 528),
         (64, [64] * 60, 2041, 272), (32, [64] * 60, 96, 144),
         (256, [256, 255, 257, 1, 0, 31, 500, 33, 700] * 3, 1003, 1040), (256, [1500, 3000, 1], 2041, 272),
         (256, [256, 255, 257, 1, 0, 31, 500, 33, 700] * 3, 264, 528), (256, [1500, 3000, 1], 640, 2048)]


@pytest.mark.parametrize("rows,sizes,N,K", FORMS, ids=lambda v: f"{len(v)}x{max(v)}" if isinstance(v, list) else str(v))
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_grouped_forms(q, rows, sizes, N, K, dtype):
    """Outputs that take stores of 16, 4 and 2 bytes, and strided ones; rows of no
    expert in front of the groups and behind them."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert q.grouped_tile_rows(sum(sizes), len(sizes), N, K, sms) == rows
    check_grouped(q, sizes, N, K, dtype)
    check_grouped(q, sizes, N, K, dtype, extra=3, first=2, pad_y=2, pad_x=16)
    check_grouped(q, sizes, N, K, dtype, extra=1, pad_y=1)


@pytest.mark.parametrize("rows,sizes", [(16, [5, 2]), (32, [30, 31] * 20), (64, [64, 60] * 40), (256, [700, 300] * 10)],
                         ids=lambda v: f"{len(v)}x{max(v)}" if isinstance(v, list) else str(v))
def test_a_wait_that_runs_out_in_every_form(q, rows, sizes):
    """A load that is left out: the status says so, and the next call is right."""
    assert q.grouped_tile_rows(sum(sizes), len(sizes), 512, 2048, 152) == rows
    Xq, Xs, W, Ws, off = grouped_problem(sizes, 512, 2048, 3)
    assert q.last_device_status() == 0
    q.set_wait_timeout_ns(20_000_000)
    for unit in (0, 5):
        q.set_fault_injection(unit)
        try:
            q.qgemm_w8a8_grouped(Xq, Xs, W, Ws, off)
            assert q.last_device_status() == 5
        finally:
            q.set_fault_injection(-1)
    q.set_wait_timeout_ns(1_000_000_000)
    check_grouped(q, sizes, 512, 2048, "bf16")


# one or two K blocks a tile, and more than the 32 units whose weight scales are held at a time
@pytest.mark.parametrize("rows,sizes,N,K",
                         [(256, [1500, 3000, 1] * 4, 2056, 16), (256, [1500, 3000, 1] * 4, 2056, 128),
                          (256, [1500, 3000, 1] * 4, 2056, 144), (256, [700, 900] * 6, 640, 4368),
                          (256, [700, 900, 30] * 6, 700, 8336), (32, [5, 17], 200, 8464),
                          (32, [30, 31] * 20, 520, 8464), (64, [64, 60] * 40, 520, 8464), (64, [64, 60] * 40, 300, 16),
                          (64, [30, 31, 20] * 40, 300, 128), (16, [3, 4] * 40, 300, 16), (16, [3, 4] * 40, 300, 272)],
                         ids=lambda v: f"{len(v)}x{max(v)}" if isinstance(v, list) else str(v))
def test_grouped_short_and_long_k(q, rows, sizes, N, K):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert q.grouped_tile_rows(sum(sizes), len(sizes), N, K, sms) == rows
    check_grouped(q, sizes, N, K, "bf16")


def test_grouped_rows_of_a_full_device(q):
    """The largest number of experts, some with a row, some with many tiles."""
    E = q.MAX_EXPERTS
    g = gen(4)
    sizes = torch.randint(0, 4, (E,), generator=g, device="cuda")
    sizes[[0, 17, E - 1]] = torch.tensor([300, 0, 700], device="cuda")
    check_grouped(q, sizes.tolist(), 264, 272, "bf16")
    check_grouped(q, (sizes * 40).tolist(), 264, 272, "bf16")
