"""The forms that the 8-bit integer GEMM takes for one shape or another (one
or two launches, tiles of 16 to 256 tokens on CTAs and CTA pairs, tiles split
through the workspace or in clusters), each shape with the form that it is
meant for asserted beside it: the rule chooses by cost, and a shape may move.

Bounds as in test_gpu_int8.py; the integer sums stay below 2^24 (uniform codes:
a sum's deviation is 5461 sqrt(K), an eighth of that at K = 131072)."""
import pytest
import torch

from gpu_util import qg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
OUT = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
COUNTERS = 32768   # bytes in front of every workspace


def _form(M, N, K):
    """(tokens of a tile, CTAs, True where tiles are split through the workspace)
    of the next call, from the workspace's size: counters, expanded activations,
    two slots of 512 bytes a token of the tile for each CTA."""
    q = qg()
    ctas = q.dispatch_get(q.KIND_INT8, M, N, K)
    need = q.workspace_bytes(q.KIND_INT8, M, N, K)
    x = (2 * M * K + 255) // 256 * 256
    for rows in (16, 32, 64, 128, 256):
        expanded = x if rows > 16 else 0
        if need == COUNTERS + expanded + 1024 * rows * ctas:
            return rows, ctas, True
    rows = q.int8_tile_rows(M, N, K, 152)
    assert need == (COUNTERS + x if rows > 16 else 0)
    return rows, ctas, False


def _inputs(M, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Xq = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    W = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(M, generator=g, device="cuda") * 0.05 + 0.003
    sw = torch.rand(N, generator=g, device="cuda") * 1e-3 + 1e-4
    return Xq, sx, W, sw, torch.randn(N, generator=g, device="cuda")


def _check(y, Xq, sx, W, sw, b):
    P = torch.cat([r.double() @ W.double().t() for r in Xq.split(256)]) * sx.double()[:, None] * sw.double()[None, :]
    ref = P + b.double()[None, :]
    tol = U * (2 * P.abs() + b.double().abs()[None, :]) * (1 + 2.0 ** -10)
    tol = tol + OUT[y.dtype] * (ref.abs() + tol) + 1e-38
    bad = (y.double() - ref).abs() > tol
    assert not bool(bad.any()), int(bad.sum())


def _split_twice(M, N, K, dtype):
    """Two calls on one workspace: right, equal bit for bit, counters at zero."""
    q = qg()
    args = _inputs(M, N, K, M + N + K)
    ws = q.Workspace()
    y = q.qgemm_w8a8_int8(*args[:4], bias=args[4], out_dtype=dtype, workspace=ws)
    assert q.last_device_status() == 0
    assert int(ws.buf[:COUNTERS].count_nonzero()) == 0
    assert torch.equal(q.qgemm_w8a8_int8(*args[:4], bias=args[4], out_dtype=dtype, workspace=ws), y)
    assert q.last_device_status() == 0
    _check(y, *args)


@pytest.mark.parametrize("dtype", list(OUT), ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K,rows,ctas", [
    (128, 1024, 65536, 128, 128),     # 4 tiles in 16 equal pieces each
    (512, 768, 131072, 256, 144),     # 6 tiles in 12
    (256, 1024, 65536, 128, 144),     # 8 tiles in 9
    (349, 27822, 8288, 128, 152),     # whole tiles, then 23 in 3 equal pieces
    (267, 9911, 14096, 128, 152),     # whole tiles, then pieces that straddle tiles
    (1036, 5690, 16272, 256, 152),    # the same with the widest tiles
])
def test_pairs_sum_pieces_through_the_workspace(M, N, K, rows, ctas, dtype):
    assert _form(M, N, K) == (rows, ctas, True)
    _split_twice(M, N, K, dtype)


@pytest.mark.parametrize("M,N,K,forced,rows", [
    (100, 256, 4112, 3, 128), (200, 300, 2064, 5, 128), (500, 256, 1040, 5, 128), (256, 300, 32784, 26, 128),
    (513, 2999, 4112, 37, 128), (1000, 1500, 8208, 151, 128),
    (500, 300, 8208, 5, 256), (200, 770, 8208, 5, 256), (500, 771, 4112, 5, 256), (500, 300, 32784, 26, 256),
    (1000, 1500, 8208, 37, 256),
])
def test_forced_grids_of_pairs(M, N, K, forced, rows):
    """Dispatch-table grids whose pieces straddle tiles of pairs, few and many."""
    q = qg()
    q.dispatch_set(q.KIND_INT8, M, N, K, forced)
    try:
        assert _form(M, N, K) == (rows, (forced + 1) // 2 * 2, True)
        _split_twice(M, N, K, torch.float32)
    finally:
        q.dispatch_clear()


# shapes of every width whose call is two launches: the expansion of the
# activations into the workspace, and the GEMM that starts under it
TWO_LAUNCHES = [(64, 5120, 1040, 32), (32, 5120, 5120, 32), (64, 5120, 5120, 64), (256, 5120, 1040, 128),
                (128, 6144, 5120, 128), (512, 6144, 1040, 256), (256, 5120, 5120, 256)]


@pytest.mark.parametrize("M,N,K,rows", TWO_LAUNCHES)
def test_two_launches_on_another_stream_and_in_a_graph(M, N, K, rows):
    q = qg()
    assert q.int8_tile_rows(M, N, K, 152) == rows
    g = torch.Generator(device="cuda").manual_seed(M + K)
    _, _, W, sw, b = _inputs(M, N, K, 4)
    X = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    expect = q.qgemm_w8a8_int8(*q.quantize_act_int8(X), W, sw, bias=b)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for stream in (st, st.cuda_stream):
        got = q.qgemm_w8a8_int8(*q.quantize_act_int8(X, stream=stream), W, sw, bias=b, stream=stream)
        st.synchronize()
        assert torch.equal(got, expect)
    ws = q.Workspace()
    Xq, sx = q.quantize_act_int8(X)
    Y = q.qgemm_w8a8_int8(Xq, sx, W, sw, bias=b, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):   # the second expansion overwrites what the first GEMM has read
            q.quantize_act_int8(X, Xq, sx)
            q.qgemm_w8a8_int8(Xq, sx, W, sw, bias=b, Y=Y, workspace=ws)
    for _ in range(3):
        X.copy_(torch.randn(M, K, generator=g, device="cuda"))
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, q.qgemm_w8a8_int8(*q.quantize_act_int8(X), W, sw, bias=b))
    assert q.last_device_status() == 0


@pytest.mark.parametrize("M,K,rows", [(32, 5120, 32), (64, 5120, 64), (96, 8192, 128), (256, 5120, 256)])
def test_overlapped_chain_with_an_expansion(M, K, rows):
    """With launch overlap on, each call's expansion overwrites the workspace
    behind the GEMM before it, which the call itself feeds on."""
    q = qg()
    assert q.int8_tile_rows(M, K, K, 152) == rows
    g = torch.Generator(device="cuda").manual_seed(K + M)
    W = torch.randint(-127, 128, (K, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.full((K,), 2e-4, device="cuda")
    X = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)

    def chain():
        y = X
        for _ in range(6):
            y = q.qgemm_w8a8_int8(*q.quantize_act_int8(y), W, sw)
        return y

    expect = chain()
    q.set_weight_prefetch_overlap(True)
    try:
        for _ in range(3):
            assert torch.equal(chain(), expect)
    finally:
        q.set_weight_prefetch_overlap(False)
    assert q.last_device_status() == 0


@pytest.mark.parametrize("M,N,K,rows", [(256, 5120, 1040, 128), (128, 6144, 5120, 128), (256, 5120, 5120, 256),
                                        (128, 1024, 65536, 128)])
def test_timeout_on_pairs(M, N, K, rows):
    """A weight copy that is never made, on whole tiles of pairs, pieces in
    clusters of pairs and pieces through the workspace: every wait runs out on
    both CTAs, the status says so, and the next call is right."""
    q = qg()
    assert _form(M, N, K)[0] == rows
    args = _inputs(M, N, K, 21)
    ws = q.Workspace()
    q.qgemm_w8a8_int8(*args[:4], workspace=ws)
    assert q.last_device_status() == 0
    q.set_wait_timeout_ns(20_000_000)      # 20 ms
    q.set_fault_injection(0)               # CTA 0 never loads its first unit
    try:
        q.qgemm_w8a8_int8(*args[:4], workspace=ws)
        assert q.last_device_status() == 5  # QG_ERR_TIMEOUT
    finally:
        q.set_fault_injection(-1)
        q.set_wait_timeout_ns(1_000_000_000)
    ws.reset()
    y = q.qgemm_w8a8_int8(*args[:4], bias=args[4], out_dtype=torch.float32, workspace=ws)
    assert q.last_device_status() == 0
    _check(y, *args)
