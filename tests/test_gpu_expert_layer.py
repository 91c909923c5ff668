"""The operators of an expert layer and the draft verification as they are used
together (examples/expert_layer.py): against 64-bit arithmetic on the same codes,
captured and replayed with other routings, on another stream, with rows of no
expert, beyond 32-bit offsets, and after a wait that ran out."""
import importlib.util
import math
import os

import pytest
import torch

from gpu_util import qg
from test_gpu_experts import DTYPES, HALF_STEP, check_grouped, gen, grouped_problem, grouped_reference

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def q():
    return qg()


def _example():
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def dequant(codes, scale):
    E, N, K = codes.shape
    spread = scale.double().repeat_interleave(128, dim=1)[:, :N].repeat_interleave(128, dim=2)[:, :, :K]
    return codes.view(torch.float8_e4m3fn).double() * spread


def make_layer(E, H, F, top, seed, **kw):
    g = gen(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda") / math.sqrt(s[-1])   # noqa: E731
    return _example().ExpertLayer(n(E, H).to(torch.bfloat16), n(E, F, H), n(E, F, H), n(E, H, F), top, **kw)


@pytest.mark.parametrize("M,E,H,F,top", [(1, 8, 256, 128, 2), (7, 16, 512, 272, 4), (64, 8, 1024, 512, 2),
                                         (600, 4, 528, 256, 2), (300, 32, 256, 144, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_layer_step_by_step(q, M, E, H, F, top, score):
    """Every step against 64 bits on what the steps before it gave."""
    g = gen(M)
    bias = torch.randn(E, generator=g, device="cuda") * 0.1 if score == "sigmoid" else None
    layer = make_layer(E, H, F, top, M, bias=bias, score=score, scale=1.5)
    x = torch.randn(M, H, generator=g, device="cuda").to(torch.bfloat16)
    if M > 5:
        x[3] = 0.0
    logits = x @ layer.router.t()
    if M > 5:
        logits[4] = -math.inf           # a token of padding goes nowhere
    r = q.moe_route(logits, top, score=score, bias=bias, scale=1.5)
    live = int(r.offsets[-1])
    assert live == top * (M - (M > 5))
    codes, scales = q.quantize_rows_e4m3(x, rows=r.rows)
    h = q.qgemm_w8a8_grouped(codes, scales, *layer.gate_up, r.offsets)
    ref, mass = grouped_reference(codes.view(torch.float8_e4m3fn), scales, layer.gate_up[0].view(torch.float8_e4m3fn),
                                  layer.gate_up[1], r.offsets)
    tol = HALF_STEP["bf16"] * ref[:live].abs() + 33 * 2.0 ** -24 * mass[:live]
    assert bool(((h[:live].double() - ref[:live]).abs() <= tol).all())
    codes2, scales2 = q.quantize_rows_e4m3(h, gated=True, num_rows=r.offsets[-1:])
    y = q.qgemm_w8a8_grouped(codes2, scales2, *layer.down, r.offsets)
    ref, mass = grouped_reference(codes2.view(torch.float8_e4m3fn), scales2, layer.down[0].view(torch.float8_e4m3fn),
                                  layer.down[1], r.offsets)
    tol = HALF_STEP["bf16"] * ref[:live].abs() + 33 * 2.0 ** -24 * mass[:live]
    assert bool(((y[:live].double() - ref[:live]).abs() <= tol).all())
    out = q.moe_combine(y, r.rows, r.weights, residual=x)
    assert q.last_device_status() == 0
    terms = torch.where((r.rows >= 0)[:, :, None], y.double()[r.rows.long().clamp_min(0)] * r.weights.double()[:, :, None], 0.0)
    ref = terms.sum(dim=1) + x.double()
    mass = terms.abs().sum(dim=1) + x.double().abs()
    assert bool(((out.double() - ref).abs() <= HALF_STEP["bf16"] * ref.abs() + (top + 2) * 2.0 ** -24 * mass).all())
    if M > 5:
        assert torch.equal(out[4], x[4])
    # the example's call is the same chain
    if M <= 5:
        assert torch.equal(layer(x, residual=x), out)


@pytest.mark.parametrize("M,E,top", [(16, 8, 2), (130, 8, 4), (700, 4, 2)])
def test_captured_layer_serves_other_routings(q, M, E, top):
    """One capture, replayed on inputs that go to other experts: each replay gives
    the eager bits; two captures of one stream do not disturb one another."""
    H, F, V, G = 512, 256, 5000, 3
    layer = make_layer(E, H, F, top, 5)
    g = gen(6)
    x = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    B = M // (G + 1)
    head = torch.randn(V, H, generator=g, device="cuda").to(torch.bfloat16) * 0.05
    tok = torch.empty(B, G, dtype=torch.int64, device="cuda")
    u, z = torch.empty(B, G, device="cuda"), torch.empty(B, V, device="cuda")

    def fill(seed):
        k = gen(seed)
        x.copy_(torch.randn(M, H, generator=k, device="cuda"))
        tok.copy_(torch.randint(0, V, (B, G), generator=k, device="cuda"))
        u.copy_(torch.rand(B, G, generator=k, device="cuda"))
        z.copy_(torch.empty(B, V, device="cuda").exponential_(generator=k))

    def step():
        y = layer(x, residual=x)
        logits = (y[:B * (G + 1)] @ head.t()).view(B, G + 1, V)
        return y, q.verify_drafts(logits, tok, None, u, z)

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            graphs.append((graph, step()))
    for seed in range(1, 5):
        fill(seed)
        y, check = step()
        want = y.clone(), check.accepted.clone(), check.tokens.clone()
        torch.cuda.synchronize()
        # both at once, on streams of their own
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for s, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert q.last_device_status() == 0
        for _, (gy, gc) in graphs:
            assert torch.equal(gy, want[0]) and torch.equal(gc.accepted, want[1]) and torch.equal(gc.tokens, want[2])


def test_calls_on_another_stream(q):
    """stream=, and the current stream another one: the same bits, ordered behind
    what the stream was doing."""
    layer = make_layer(8, 512, 256, 2, 9)
    x0 = torch.randn(40, 512, device="cuda").to(torch.bfloat16)
    want = layer(x0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(10):
            busy = busy @ busy * 1e-4
        x = x0.clone()
        logits = x @ layer.router.t()
    r = q.moe_route(logits, 2, stream=s)
    codes, scales = q.quantize_rows_e4m3(x, rows=r.rows, stream=s)
    h = q.qgemm_w8a8_grouped(codes, scales, *layer.gate_up, r.offsets, stream=s)
    codes2, scales2 = q.quantize_rows_e4m3(h, gated=True, num_rows=r.offsets[-1:], stream=s)
    y = q.qgemm_w8a8_grouped(codes2, scales2, *layer.down, r.offsets, stream=s.cuda_stream)
    out = q.moe_combine(y, r.rows, r.weights, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("rows", [1, 15, 40, 300])
def test_values_beside_a_group_do_not_reach_it(q, rows):
    """NaN codes and scales in the rows of other experts and behind the last, and in
    the weights of other experts."""
    sizes = [rows, rows + 3, rows]
    Xq, Xs, W, Ws, off = grouped_problem(sizes, 200, 400, 11, extra=70)
    clean = torch.full((Xq.shape[0], 200), 7.0, device="cuda")
    q.qgemm_w8a8_grouped(Xq, Xs, W, Ws, off, Y=clean)
    a, b, end = int(off[1]), int(off[2]), int(off[3])
    Xq.view(torch.uint8)[a:b] = 0x7F
    Xq.view(torch.uint8)[end:] = 0xFF
    Xs[:, a:b] = math.nan
    Xs[:, end:] = math.inf
    W.view(torch.uint8)[1] = 0x7F
    Ws[1] = math.nan
    Y = torch.full((Xq.shape[0], 200), 7.0, device="cuda")
    q.qgemm_w8a8_grouped(Xq, Xs, W, Ws, off, Y=Y)
    assert q.last_device_status() == 0
    for c, d in ((0, a), (b, end)):
        assert torch.equal(Y[c:d], clean[c:d])
    assert bool((Y[end:] == 7.0).all())


@pytest.mark.parametrize("sizes", [[5, 2], [30, 31], [700, 300]], ids=lambda s: f"{max(s)} rows")
def test_a_wait_that_runs_out_is_reported(q, sizes):
    """A weight load that is left out: the status says so, and the next call is right."""
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


def test_equal_calls_give_equal_bits(q):
    for sizes in ([3] * 20, [50, 20, 0, 33], [500, 260, 300]):
        Xq, Xs, W, Ws, off = grouped_problem(sizes, 768, 1040, 3)
        first = q.qgemm_w8a8_grouped(Xq, Xs, W, Ws, off, out_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(first, q.qgemm_w8a8_grouped(Xq, Xs, W, Ws, off, out_dtype=torch.float32))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_outputs_beyond_32_bit_offsets(q, dtype):
    """Elements of Y, of the quantiser's output and of the combination's input from 2^31 on."""
    R, N, K = 70000, 32768, 32      # 2.3e9 elements
    Xq, Xs, W, Ws, off = grouped_problem([R - 300, 300], N, K, 5)
    Y = q.qgemm_w8a8_grouped(Xq, Xs, W, Ws, off, out_dtype=DTYPES[dtype])
    assert q.last_device_status() == 0
    for a, b, e in ((0, 64, 0), (R - 364, R - 300, 0), (R - 300, R, 1)):
        x = Xq[a:b].double() * Xs[0, a:b].double()[:, None]
        w = W[e].double() * Ws[e, :, 0].double().repeat_interleave(128)[:N, None]
        ref, mass = x @ w.t(), x.abs() @ w.abs().t()
        assert bool(((Y[a:b].double() - ref).abs() <= HALF_STEP[dtype] * ref.abs() + 33 * 2.0 ** -24 * mass).all())
    rows = torch.tensor([[R - 1, 5], [R - 2, 0]], dtype=torch.int32, device="cuda")
    weights = torch.tensor([[0.5, 0.25], [1.0, 0.0]], device="cuda")
    out = q.moe_combine(Y, rows, weights)
    ref = (Y[rows.long()].double() * weights.double()[:, :, None]).sum(dim=1)
    mass = (Y[rows.long()].double() * weights.double()[:, :, None]).abs().sum(dim=1)
    assert bool(((out.double() - ref).abs() <= HALF_STEP[dtype] * ref.abs() + 4 * 2.0 ** -24 * mass).all())


def test_quantiser_and_drafts_beyond_32_bit_offsets(q):
    K, out_rows = 17408, 130000      # 2.3e9 codes
    X = torch.randn(2, K, device="cuda").to(torch.bfloat16)
    rows = torch.tensor([[out_rows - 1], [3]], dtype=torch.int32, device="cuda")
    Xq, Xs = q.quantize_rows_e4m3(X, rows=rows, out_rows=out_rows)
    want_q, want_s = q.quantize_act_e4m3(X)
    assert torch.equal(Xq[out_rows - 1], want_q[0]) and torch.equal(Xq[3], want_q[1])
    assert torch.equal(Xs[:, out_rows - 1], want_s[:, 0]) and torch.equal(Xs[:, 3], want_s[:, 1])
    del Xq, Xs
    V, far = 9000, 2 ** 31 + 64
    memory = torch.empty(far + 3 * V, dtype=torch.bfloat16, device="cuda")
    t = memory.as_strided((2, 3, V), (far, V, 1))
    t.copy_(torch.randn(2, 3, V, device="cuda") * 3)
    tok = t[:, :2].float().argmax(dim=2)
    u, z = torch.rand(2, 2, device="cuda"), torch.empty(2, V, device="cuda").exponential_()
    a, b = q.verify_drafts(t, tok, None, u, z), q.verify_drafts(t.contiguous(), tok, None, u, z)
    assert torch.equal(a.accepted, b.accepted) and torch.equal(a.tokens, b.tokens)


def test_example_runs(capsys, monkeypatch):
    ex = _example()
    monkeypatch.setattr("sys.argv", ["expert_layer.py", "--tokens", "40", "--hidden", "256", "--inner", "128",
                                     "--vocab", "2000"])
    assert ex.main() == 0
    out = capsys.readouterr().out
    assert "of 16 experts" in out and "drafts kept" in out


FIRST = """
import torch, weight_only_quantized_qgemm_gb300 as q
torch.cuda.set_device(0)
E, M, K, N = 16, 700, 256, 272
logits, x = torch.randn(M, E, device="cuda"), torch.randn(M, K, device="cuda").to(torch.bfloat16)
W = torch.randint(0, 120, (E, N, K), device="cuda", dtype=torch.uint8)
S = torch.rand(E, -(-N // 128), K // 128, device="cuda")
t = torch.randn(40, 3, 9000, device="cuda")
tok, u, z = t[:, :2].argmax(dim=2), torch.rand(40, 2, device="cuda"), torch.rand(40, 9000, device="cuda") + 0.1
def step():
    r = q.moe_route(logits, 2)
    codes, scales = q.quantize_rows_e4m3(x, rows=r.rows)
    y = q.qgemm_w8a8_grouped(codes, scales, W, S, r.offsets)
    return q.moe_combine(y, r.rows, r.weights), *q.verify_drafts(t, tok, None, u, z)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
assert q.last_device_status() == 0
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("same")
"""


def test_first_calls_of_a_process_captured():
    import subprocess
    import sys
    out = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "same" in out.stdout, out.stderr[-2000:]


def test_threads_on_streams_of_their_own(q):
    """Two host threads, each with a stream, inputs and sizes of its own."""
    import threading
    layer = [make_layer(8, 512, 256, 2, 21), make_layer(12, 256, 144, 4, 22)]
    inputs = [torch.randn(m, h, device="cuda").to(torch.bfloat16) for m, h in ((90, 512), (2000, 256))]
    logits = [torch.randn(30, 4, 9000, device="cuda"), torch.randn(3, 2, 5000, device="cuda")]
    tokens = [t[:, :-1].argmax(dim=2) for t in logits]
    want = [(layer[i](inputs[i]), *q.verify_drafts(logits[i], tokens[i])) for i in range(2)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got = (layer[i](inputs[i]), *q.verify_drafts(logits[i], tokens[i]))
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)
        except Exception as e:   # noqa: BLE001
            wrong.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and q.last_device_status() == 0
