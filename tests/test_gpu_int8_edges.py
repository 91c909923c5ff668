"""The 8-bit integer path where inputs or the work around it are unusual:
broken activations, nothing to quantise, a long kernel in front of the GEMM, one
workspace for several kinds."""
import numpy as np
import pytest
import torch

from gpu_util import qg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("K", [64, 5120, 40960])
def test_broken_rows_stay_broken(dtype, K):
    """A row with a NaN or an infinity has scale NaN, and the GEMM and the
    scores behind it give NaN for that row and no other."""
    q = qg()
    g = torch.Generator(device="cuda").manual_seed(K)
    X = torch.randn(9, K, generator=g, device="cuda").to(dtype)
    good = X.clone()
    X[1, 0] = float("nan")
    X[2, K - 1] = float("inf")
    X[3, K // 2] = -float("inf")
    X[4, 5], X[4, 6] = float("inf"), float("nan")
    X[5] = float("nan")
    X[6, 7] = -float("nan")
    broken = torch.tensor([0, 1, 1, 1, 1, 1, 1, 0, 0], dtype=torch.bool, device="cuda")
    codes, scale = q.quantize_act_int8(X)
    assert torch.equal(torch.isnan(scale), broken)
    c0, s0 = q.quantize_act_int8(good)
    assert torch.equal(codes[~broken], c0[~broken]) and torch.equal(scale[~broken], s0[~broken])
    W = torch.randint(-127, 128, (200, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.full((200,), 1e-3, device="cuda")
    y = q.qgemm_w8a8_int8(codes, scale, W, sw, out_dtype=torch.float32)
    assert torch.equal(torch.isnan(y), broken[:, None].expand_as(y))
    r = q.logprobs(y, torch.zeros(9, dtype=torch.int64, device="cuda"), top_k=3, entropy=True)
    for t in (r.token_logprobs, r.entropy, r.top_logprobs[:, 0]):
        assert torch.equal(torch.isnan(t), broken)


def test_rows_of_nothing_have_scale_one():
    """K = 0: a row's largest |x| is that of no values, 0."""
    q = qg()
    X = torch.empty(5, 0, dtype=torch.bfloat16, device="cuda")
    scale = torch.full((5,), 3.0, device="cuda")
    codes, got = q.quantize_act_int8(X, X_scale=scale)
    assert got is scale and torch.equal(scale, torch.ones(5, device="cuda")) and tuple(codes.shape) == (5, 0)
    junk = torch.full((1 << 20,), float("nan"), device="cuda")
    del junk
    st = torch.cuda.Stream()
    for stream in (None, st):
        _, fresh = q.quantize_act_int8(X, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(fresh, torch.ones(5, device="cuda"))


@pytest.mark.parametrize("overlap", [False, True], ids=["plain", "overlapped"])
@pytest.mark.parametrize("M,N,K,rows", [(1, 1024, 5120, 16), (4, 640, 1040, 16), (64, 5120, 5120, 64),
                                        (256, 5120, 5120, 256)])
def test_the_wait_limit_does_not_count_the_kernel_in_front(M, N, K, rows, overlap):
    """A GEMM that starts under a preceding kernel (here of several hundred
    microseconds on a few SMs, which lets it start at once) gives up on none of
    its waits for that, with a limit below the kernel's time."""
    q = qg()
    assert q.int8_tile_rows(M, N, K, 152) == rows
    g = torch.Generator(device="cuda").manual_seed(6)
    Xq = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    W = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sx, sw = torch.full((M,), 0.01, device="cuda"), torch.full((N,), 1e-3, device="cuda")
    ws = q.Workspace()
    expect = q.qgemm_w8a8_int8(Xq, sx, W, sw, workspace=ws)   # which grows it, and so waits for the device
    logits = torch.zeros((1, 1 << 28), dtype=torch.bfloat16, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    q.logprobs(logits, entropy=True)
    start.record()
    q.logprobs(logits, entropy=True)
    end.record()
    end.synchronize()
    limit_us = 150
    assert start.elapsed_time(end) * 1e3 > 2 * limit_us, "the kernel in front is too short for this test"
    q.set_wait_timeout_ns(limit_us * 1000)
    q.set_weight_prefetch_overlap(overlap)
    try:
        q.logprobs(logits, entropy=True)
        got = q.qgemm_w8a8_int8(Xq, sx, W, sw, workspace=ws)
        assert q.last_device_status() == 0
    finally:
        q.set_weight_prefetch_overlap(False)
        q.set_wait_timeout_ns(1_000_000_000)
    assert torch.equal(got, expect)


def test_one_workspace_object_serves_every_kind():
    """Kinds that lay their workspace out differently, in turn on one Workspace."""
    import workloads as wl
    q = qg()
    p = wl.make_fp8_problem(4, 1024, 5120, config_id=50)
    Xf = torch.from_numpy(p.X.view(np.int16)).view(torch.bfloat16).cuda()
    Wf, Sf = torch.from_numpy(p.W).cuda(), torch.from_numpy(p.S).cuda()
    g = torch.Generator(device="cuda").manual_seed(31)
    X = torch.randn(200, 5120, generator=g, device="cuda").to(torch.bfloat16)
    Wi = torch.randint(-127, 128, (1024, 5120), generator=g, device="cuda", dtype=torch.int8)
    si = torch.full((1024,), 1e-3, device="cuda")
    calls = [lambda ws: q.qgemm_fp8_block(Xf, Wf, Sf, workspace=ws),
             lambda ws: q.qgemm_w8a8_int8(*q.quantize_act_int8(X), Wi, si, workspace=ws),
             lambda ws: q.qgemm_w8a8_int8(*q.quantize_act_int8(X[:1]), Wi, si, workspace=ws),
             lambda ws: q.qgemm_w8a8(X, Wf, Sf, workspace=ws)]
    for kind, M in ((q.KIND_FP8_BLOCK, 4), (q.KIND_INT8, 200), (q.KIND_INT8, 1), (q.KIND_W8A8, 200)):
        assert q.workspace_bytes(kind, M, 1024, 5120) > 0
    expect = [c(q.Workspace()) for c in calls]
    ws = q.Workspace()
    for _ in range(3):
        for c, want in zip(calls, expect):
            out = c(ws)
            assert q.last_device_status() == 0 and torch.equal(out, want)


def test_a_graph_outlives_its_workspace_s_growth():
    """A larger call on the Workspace of a captured graph, and other tensors
    made after it: the replays give what they gave, and write to nothing else."""
    q = qg()
    g = torch.Generator(device="cuda").manual_seed(41)
    W = torch.randint(-127, 128, (1024, 5120), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.full((1024,), 1e-3, device="cuda")
    small = q.quantize_act_int8(torch.randn(200, 5120, generator=g, device="cuda").to(torch.bfloat16))
    large = q.quantize_act_int8(torch.randn(4096, 5120, generator=g, device="cuda").to(torch.bfloat16))
    ws = q.Workspace()
    want = q.qgemm_w8a8_int8(*small, W, sw, workspace=ws)
    before = ws.buf.numel()
    Y = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qgemm_w8a8_int8(*small, W, sw, Y=Y, workspace=ws)
    q.qgemm_w8a8_int8(*large, W, sw, workspace=ws)
    assert ws.buf.numel() > before
    others = [torch.full((before,), 85, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for _ in range(2):
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want) and all(bool((t == 85).all()) for t in others)
    assert q.last_device_status() == 0
