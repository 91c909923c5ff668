"""8-bit integer path (quantize_act_int8, qgemm_w8a8_int8) against plain
64-bit arithmetic.

Bounds (u = 2^-24; P = sx * sw * integer sum): the kernel's integer sum is
exact while partial sums stay under 2^24; it then rounds acc * sx, the fma
with sw and the bias, and the conversion to the output type, so
    |error| <= u (2 |P| + |b|) (1 + 2^-10) + half an ulp of the output type.
Where the sums leave 2^24, every accumulation step (one per 16 products, plus
the pieces of a split) may lose 2^-23 of the absolute mass."""
import numpy as np
import pytest
import torch

from gpu_util import qg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
OUT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}


def _codes(rng, rows, cols):
    return rng.integers(-128, 128, size=(rows, cols), dtype=np.int8)


def _problem(M, N, K, seed, lo=-128):
    rng = np.random.default_rng(seed)
    Xq = rng.integers(lo, 128, size=(M, K), dtype=np.int8)
    W = rng.integers(lo, 128, size=(N, K), dtype=np.int8)
    sx = rng.uniform(0.003, 0.05, M).astype(np.float32)
    sw = rng.uniform(1e-4, 1e-3, N).astype(np.float32)
    b = rng.standard_normal(N).astype(np.float32)
    return Xq, sx, W, sw, b


def _int_product(Xq, W):
    """The exact integer product, through float64 (every sum below 2^53)."""
    return (torch.from_numpy(Xq).double() @ torch.from_numpy(W).double().t()).numpy()


def _call(q, Xq, sx, W, sw, b, dtype, xpad=0, ypad=0, ws=None):
    M, K = Xq.shape
    N = W.shape[0]
    X = torch.zeros((M, K + xpad), dtype=torch.int8, device="cuda")
    X[:, :K] = torch.from_numpy(Xq)
    Y = torch.full((M, N + ypad), float("nan"), dtype=dtype, device="cuda")
    q.qgemm_w8a8_int8(X[:, :K], torch.from_numpy(sx).cuda(), torch.from_numpy(W).cuda(), torch.from_numpy(sw).cuda(),
                      bias=None if b is None else torch.from_numpy(b).cuda(), Y=Y[:, :N], workspace=ws)
    assert q.last_device_status() == 0
    if ypad:
        assert bool(torch.isnan(Y[:, N:]).all()), "columns past N were written"
    return Y[:, :N].double().cpu().numpy()


def _check(y, Xq, sx, W, sw, b, dtype, mass=None):
    P = _int_product(Xq, W) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    bb = np.zeros(W.shape[0]) if b is None else b.astype(np.float64)
    ref = P + bb[None, :]
    tol = U * (2 * np.abs(P) + np.abs(bb)[None, :]) * (1 + 2.0 ** -10)
    if mass is not None:
        tol = tol + mass
    tol = tol + OUT[dtype] * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == torch.float16 else 1e-38)
    bad = np.abs(y - ref) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.max(np.abs(y - ref) / tol)))


SHAPES = [
    # M, N, K: tile edges on every side, one row, one channel, K tails of every kind
    (1, 1, 16), (1, 128, 128), (1, 1024, 5120), (2, 129, 144), (16, 256, 512), (17, 200, 336), (31, 77, 64),
    (33, 128, 1040), (64, 300, 128), (65, 127, 272), (83, 1003, 1040), (128, 256, 2048), (129, 513, 528),
    (200, 384, 4096), (255, 130, 656), (256, 5120, 1024), (300, 257, 4112), (513, 640, 768),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", list(OUT), ids=["bf16", "fp16", "fp32"])
def test_gemm_matches_64_bits(M, N, K, dtype):
    Xq, sx, W, sw, b = _problem(M, N, K, 7 * M + N + K)
    y = _call(qg(), Xq, sx, W, sw, b if (M + N) % 2 else None, dtype, xpad=16 * (M % 3), ypad=5 * (N % 2))
    _check(y, Xq, sx, W, sw, b if (M + N) % 2 else None, dtype)


WIDTHS = [
    # M, N, K that take every tile width of the kernel, with ragged edges on
    # every side, few and many tiles a CTA, pieces of a tile in a cluster, split
    # tails and odd channel counts
    (17, 19001, 1040), (24, 49155, 1040), (31, 5001, 5120), (50, 9001, 4112), (64, 17408, 400),
    (50, 15001, 2064), (172, 4218, 1456), (40, 17283, 1040), (65, 17283, 1040), (128, 17408, 1552),
    (200, 9000, 2064), (384, 17155, 528), (1000, 2051, 4112), (256, 17283, 1040), (255, 5120, 17408),
    (513, 17283, 2064), (1000, 5001, 4112), (700, 6001, 1040),
    (3, 129, 4112), (24, 5001, 8208), (33, 2939, 12960), (50, 300, 16400), (129, 1000, 8208), (300, 770, 16400),
]


def test_the_shapes_take_every_width():
    assert {qg().int8_tile_rows(*shape, 152) for shape in WIDTHS} == {16, 32, 64, 128, 256}


@pytest.mark.parametrize("M,N,K", WIDTHS)
@pytest.mark.parametrize("dtype", list(OUT), ids=["bf16", "fp16", "fp32"])
def test_every_tile_width(M, N, K, dtype):
    q = qg()
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    Xq = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    W = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(M, generator=g, device="cuda") * 0.05 + 0.003
    sw = torch.rand(N, generator=g, device="cuda") * 1e-3 + 1e-4
    b = torch.randn(N, generator=g, device="cuda") if N % 2 else None
    pad = torch.full((M, N + 6), float("nan"), dtype=dtype, device="cuda")
    q.qgemm_w8a8_int8(Xq, sx, W, sw, bias=b, Y=pad[:, :N])
    assert q.last_device_status() == 0
    assert bool(torch.isnan(pad[:, N:]).all())
    P = (Xq.double() @ W.double().t()) * sx.double()[:, None] * sw.double()[None, :]   # integers below 2^53: exact
    ref = P if b is None else P + b.double()[None, :]
    tol = U * (2 * P.abs() + (0.0 if b is None else b.double().abs()[None, :])) * (1 + 2.0 ** -10)
    tol = tol + OUT[dtype] * (ref.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 1e-38)
    bad = (pad[:, :N].double() - ref).abs() > tol
    assert not bool(bad.any()), int(bad.sum())


@pytest.mark.parametrize("M,N,K", [(1, 130, 1024), (40, 256, 1024), (300, 256, 1024)])
def test_integers_are_exact(M, N, K):
    """With unit scales and 32-bit output the result is the integer product
    itself, at the extremes of the range too (1024 x 128 x 128 = 2^24)."""
    rng = np.random.default_rng(5)
    Xq = _codes(rng, M, K)
    W = _codes(rng, N, K)
    Xq[0] = -128
    W[0] = -128
    W[1] = 127
    one = np.ones
    y = _call(qg(), Xq, one(M, np.float32), W, one(N, np.float32), None, torch.float32)
    assert np.array_equal(y, _int_product(Xq, W))


@pytest.mark.parametrize("M", [3, 96, 260])
def test_sums_beyond_2_24(M):
    """One-signed codes: sums of about 2^27, rounded step by step."""
    N, K = 260, 17408
    Xq, sx, W, sw, b = _problem(M, N, K, 11, lo=90)
    mass = _int_product(np.abs(Xq), np.abs(W)) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    y = _call(qg(), Xq, sx, W, sw, b, torch.float32)
    _check(y, Xq, sx, W, sw, b, torch.float32, mass=(K / 16 + 16) * 2.0 ** -23 * mass)


@pytest.mark.parametrize("M,N,K,ctas", [(5, 300, 2048, 1), (5, 300, 2048, 7), (40, 256, 4096, 13), (100, 384, 1552, 5),
                                        (300, 300, 2064, 11), (300, 300, 2064, 37)])
def test_every_split_gives_the_same_integers(M, N, K, ctas):
    """Grids that cut tiles at any K block; the workspace's counters are back
    at zero, so a second call on it agrees bit for bit."""
    q = qg()
    Xq, sx, W, sw, b = _problem(M, N, K, ctas)
    q.dispatch_set(q.KIND_INT8, M, N, K, ctas)
    try:
        ws = q.Workspace()
        y = _call(q, Xq, sx, W, sw, b, torch.float32, ws=ws)
        assert ws.buf is None or int(ws.buf[:32768].count_nonzero()) == 0
        again = _call(q, Xq, sx, W, sw, b, torch.float32, ws=ws)
    finally:
        q.dispatch_clear()
    _check(y, Xq, sx, W, sw, b, torch.float32)
    assert np.array_equal(y, again)


def test_one_workspace_serves_changing_shapes():
    q = qg()
    ws = q.Workspace()
    for M, N, K in [(300, 512, 4096), (1, 1024, 5120), (40, 300, 2048), (700, 256, 512), (2, 5120, 1024)]:
        Xq, sx, W, sw, b = _problem(M, N, K, M)
        _check(_call(q, Xq, sx, W, sw, b, torch.bfloat16, ws=ws), Xq, sx, W, sw, b, torch.bfloat16)


def test_fp16_output_overflows_to_infinity():
    q = qg()
    Xq = np.full((3, 512), 127, np.int8)
    W = np.full((5, 512), 127, np.int8)
    W[1] = -127
    y = _call(q, Xq, np.ones(3, np.float32), W, np.ones(5, np.float32), None, torch.float16)
    assert np.all(y[:, 0] == np.inf) and np.all(y[:, 1] == -np.inf)


@pytest.mark.parametrize("M", [4, 200])
def test_gemm_on_its_own_stream_and_in_a_graph(M):
    """The quantiser and the GEMM on a stream that is not the current one, and
    captured in a CUDA graph whose replays see new inputs."""
    q = qg()
    N, K = 640, 1040
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand(N, generator=g, device="cuda") * 1e-3
    expect = q.qgemm_w8a8_int8(*q.quantize_act_int8(X), W, sw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = q.qgemm_w8a8_int8(*q.quantize_act_int8(X, stream=st), W, sw, stream=st)
    st.synchronize()
    assert torch.equal(got, expect)
    ws = q.Workspace()
    Xq, sx = q.quantize_act_int8(X)
    Y = q.qgemm_w8a8_int8(Xq, sx, W, sw, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.quantize_act_int8(X, Xq, sx)
        q.qgemm_w8a8_int8(Xq, sx, W, sw, Y=Y, workspace=ws)
    for _ in range(2):
        X.copy_(torch.randn(M, K, generator=g, device="cuda"))
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, q.qgemm_w8a8_int8(*q.quantize_act_int8(X), W, sw))
    assert q.last_device_status() == 0


def test_overlapped_chain():
    """With launch overlap on, back-to-back calls that feed one another give
    what they give without it."""
    q = qg()
    g = torch.Generator(device="cuda").manual_seed(9)
    W = torch.randint(-127, 128, (1024, 1024), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.full((1024,), 2e-4, device="cuda")
    X = torch.randn(24, 1024, generator=g, device="cuda").to(torch.bfloat16)

    def chain():
        y = X
        for _ in range(6):
            y = q.qgemm_w8a8_int8(*q.quantize_act_int8(y), W, sw)
        return y

    expect = chain()
    q.set_weight_prefetch_overlap(True)
    try:
        got = chain()
    finally:
        q.set_weight_prefetch_overlap(False)
    assert q.last_device_status() == 0
    assert torch.equal(got, expect)


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (16, 5120), (5, 17408), (2, 40960), (70, 1040), (1, 131072)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_quantiser_is_bit_exact(M, K, dtype):
    q = qg()
    g = torch.Generator(device="cuda").manual_seed(M + K)
    X = torch.zeros((M, K + 24), dtype=dtype, device="cuda")
    X[:, :K] = (torch.randn(M, K, generator=g, device="cuda") * 3).to(dtype)
    X[:, K:] = 1000.0
    if M > 2:
        X[0, :K] = 0.0
        X[1, :K] = 0.0
        X[1, K - 1] = -0.5
        X[2, :K] *= 6e-8 if dtype == torch.float16 else 1e-33   # subnormals / below the floor
    Xq = torch.full((M, K + 32), 77, dtype=torch.int8, device="cuda")
    codes, scale = q.quantize_act_int8(X[:, :K], Xq=Xq[:, :K])
    assert bool((Xq[:, K:] == 77).all())
    x = X[:, :K].float().cpu().numpy()
    amax = np.abs(x).max(axis=1)
    live = amax >= np.float32(2.0 ** -100)
    a = np.where(live, amax, np.float32(127.0)).astype(np.float32)
    inv = np.where(live, np.float32(127.0) * (np.float32(1.0) / a), np.float32(0)).astype(np.float32)
    ref = np.rint(x * inv[:, None]).astype(np.int8)
    assert np.array_equal(codes.cpu().numpy(), ref)
    assert np.array_equal(scale.cpu().numpy().view(np.uint32), (a / np.float32(127.0)).view(np.uint32))
    assert np.abs(ref.astype(np.int32)).max() <= 127


def test_empty_and_k0():
    q = qg()
    dev = "cuda"
    b = torch.randn(7, device=dev)
    y = q.qgemm_w8a8_int8(torch.empty(3, 0, dtype=torch.int8, device=dev), torch.ones(3, device=dev),
                          torch.empty(7, 0, dtype=torch.int8, device=dev), torch.ones(7, device=dev), bias=b,
                          out_dtype=torch.float32)
    assert torch.equal(y, b.expand(3, 7))
    y = q.qgemm_w8a8_int8(torch.empty(0, 32, dtype=torch.int8, device=dev), torch.empty(0, device=dev),
                          torch.zeros(7, 32, dtype=torch.int8, device=dev), torch.ones(7, device=dev))
    assert tuple(y.shape) == (0, 7)


def test_refusals():
    q = qg()
    dev = "cuda"
    Xq = torch.zeros(4, 64, dtype=torch.int8, device=dev)
    W = torch.zeros(8, 64, dtype=torch.int8, device=dev)
    sx, sw = torch.ones(4, device=dev), torch.ones(8, device=dev)
    for bad in (dict(W=W.float()), dict(sx=sx.half()), dict(sw=torch.ones(9, device=dev)), dict(W=W[:, ::2]),
                dict(b=torch.ones(4, device=dev)), dict(dt=torch.int8), dict(sx=sx.cpu())):
        with pytest.raises((TypeError, ValueError)):
            q.qgemm_w8a8_int8(Xq, bad.get("sx", sx), bad.get("W", W), bad.get("sw", sw), bias=bad.get("b"),
                              out_dtype=bad.get("dt"))
    with pytest.raises(q.QgemmError) as e:
        q.qgemm_w8a8_int8(torch.zeros(1000, 4096, dtype=torch.int8, device=dev), torch.ones(1000, device=dev),
                          torch.zeros(1024, 4096, dtype=torch.int8, device=dev), torch.ones(1024, device=dev),
                          workspace=torch.zeros(256, dtype=torch.uint8, device=dev))
    assert e.value.code == 6
    with pytest.raises(q.QgemmError) as e:   # K % 16
        q.qgemm_w8a8_int8(Xq[:, :40], sx, W[:, :40].contiguous(), sw)
    assert e.value.code == 2
    with pytest.raises(q.QgemmError) as e:   # a row not 16-byte aligned
        q.qgemm_w8a8_int8(torch.zeros(4, 72, dtype=torch.int8, device=dev)[:, 8:], sx, W, sw)
    assert e.value.code == 3
    with pytest.raises(TypeError):
        q.quantize_act_int8(torch.zeros(4, 64, device=dev))


@pytest.mark.parametrize("M,N,K", [(4, 1024, 5120), (48, 1024, 2048), (100, 700, 2048), (400, 1024, 4096)])
def test_timeout_is_reported_and_the_context_survives(M, N, K):
    """A weight copy that is never made: every wait runs out, on both CTAs of
    a pair too, the status says so, and the next call is right."""
    q = qg()
    Xq, sx, W, sw, b = _problem(M, N, K, 21)
    ws = q.Workspace()
    args = [torch.from_numpy(t).cuda() for t in (Xq, sx, W, sw)]
    q.qgemm_w8a8_int8(*args, workspace=ws)
    assert q.last_device_status() == 0
    q.set_wait_timeout_ns(20_000_000)      # 20 ms
    q.set_fault_injection(0)               # CTA 0 never loads its first unit
    try:
        q.qgemm_w8a8_int8(*args, workspace=ws)
        assert q.last_device_status() == 5  # QG_ERR_TIMEOUT
    finally:
        q.set_fault_injection(-1)
        q.set_wait_timeout_ns(1_000_000_000)
    ws.reset()
    _check(_call(q, Xq, sx, W, sw, b, torch.float32, ws=ws), Xq, sx, W, sw, b, torch.float32)
