"""The experts' operators on the GPU at the ends of what their contracts allow,
against plain implementations in 64 bits (tolerances as in test_gpu_experts.py)."""

import pytest
import torch

from gpu_util import qg
from test_gpu_experts import DTYPES, gen, offsets_of, silu_mul

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    return qg()


# ----------------------------------------------------------------- grouped GEMM
@pytest.mark.parametrize("raw,begin,end", [([4, 6, 8], 4, 8), ([0, 10, 5], 0, 10), ([2, 50, 3], 2, 12), ([-7, 3, 3], 0, 3),
                                           ([5, 4, 2], 5, 5), ([40, 1, 50], 12, 12), ([0, 0, 0], 0, 0), ([3, -9, -2], 3, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_grouped_without_k_zeroes_the_groups_rows(q, raw, begin, end, dtype):
    """The empty sums of K = 0 go to the rows of the groups alone: not to those in
    front of the first, and offsets out of order are cut as with any other K."""
    def empty(*s, dtype=torch.uint8):
        return torch.empty(s, dtype=dtype, device="cuda")

    Y = torch.full((12, 40), 3.0, dtype=DTYPES[dtype], device="cuda")
    q.qgemm_w8a8_grouped(empty(12, 0), empty(0, 32, dtype=torch.float32), empty(2, 33, 0),
                         empty(2, 1, 0, dtype=torch.float32), torch.tensor(raw, dtype=torch.int32, device="cuda"),
                         Y=Y[:, 3:36])
    want = torch.full_like(Y, 3.0)
    want[begin:end, 3:36] = 0.0
    assert torch.equal(Y, want)


def test_grouped_without_k_and_many_experts(q):
    """More offsets than a CTA has threads, the largest anywhere among them."""
    E = q.MAX_EXPERTS
    for place in (1, 255, 256, 257, 700, E):
        off = torch.full((E + 1,), 2, dtype=torch.int32)
        off[place:] = 9
        off[place + 1:] = 4
        Y = torch.full((12, 5), 3.0, dtype=torch.float16, device="cuda")
        q.qgemm_w8a8_grouped(torch.empty(12, 0, dtype=torch.uint8, device="cuda"), torch.empty(0, 32, device="cuda"),
                             torch.empty(E, 5, 0, dtype=torch.uint8, device="cuda"), torch.empty(E, 1, 0, device="cuda"),
                             off.cuda(), Y=Y)
        assert Y[:, 0].tolist() == [3.0] * 2 + [0.0] * 7 + [3.0] * 3


@pytest.mark.parametrize("K", [16, 128, 144, 256])
@pytest.mark.parametrize("rows", [1, 37, 300])
def test_the_first_columns_of_scales(q, K, rows):
    """The quantiser's scales without their padding, in one row of scales and in several."""
    g = gen(K + rows)
    sizes = [rows, 0, 6]
    R = sum(sizes)
    X = torch.randn(R, K, generator=g, device="cuda").to(torch.bfloat16)
    codes, scales = q.quantize_rows_e4m3(X)
    W = torch.randint(0, 120, (3, 72, K), generator=g, device="cuda", dtype=torch.uint8)
    Ws = torch.rand(3, 1, -(-K // 128), generator=g, device="cuda")
    off = offsets_of(sizes)
    want = q.qgemm_w8a8_grouped(codes, scales, W, Ws, off)
    assert torch.equal(q.qgemm_w8a8_grouped(codes, scales[:, :R], W, Ws, off), want)
    if R % 4:   # nothing behind the last scale
        bare = torch.empty((scales.shape[0] - 1) * scales.shape[1] + R, device="cuda")
        bare = bare.as_strided((scales.shape[0], R), (scales.shape[1], 1))
        bare.copy_(scales[:, :R])
        with pytest.raises(ValueError, match="multiple of 4"):
            q.qgemm_w8a8_grouped(codes, bare, W, Ws, off)
    # written in place, and nothing beside them
    kept = torch.full_like(scales, -7.0)
    again, out = q.quantize_rows_e4m3(X, X_scale=kept[:, :R])
    assert torch.equal(out, scales[:, :R]) and torch.equal(again, codes) and bool((kept[:, R:] == -7.0).all())


# ----------------------------------------------------------------- row quantiser
@pytest.mark.parametrize("dtype,gates", [("bf16", [-80.0, -86.5, -87.0, -87.5, -88.0, -88.5]),
                                         ("fp16", [-80.0, -87.25, -87.375, -87.5, -88.0, -88.5, -88.6875])])
@pytest.mark.parametrize("up", [1.0, 1e4, 1e37])
def test_gates_that_let_next_to_nothing_through(q, dtype, gates, up):
    """Down to where the formula's exponential passes FP32 (g = -88.7): the product
    counts where the value is large, or the block holds nothing larger."""
    if dtype == "fp16" and up > 6e4:
        up = 6e4
    g = gen(len(gates))
    M, K = len(gates), 256
    X = torch.empty((M, 2 * K), device="cuda")
    X[:, :K] = torch.tensor(gates, device="cuda")[:, None]
    X[:, K:] = torch.randn(M, K, generator=g, device="cuda").clamp(-1, 1) * up
    X = X.to(DTYPES[dtype])
    codes, scales = q.quantize_rows_e4m3(X, gated=True)
    v = silu_mul(X).view(M, K // 128, 128)
    amax = v.abs().amax(dim=2)
    s = scales[:, :M].t().double()
    # |g| <= 88.7: the exponent's product with log2 e is off by 2^-18 and 128 x 1.4e-8 (of
    # the constant), times ln 2: 4e-6; exponential, reciprocal and products 6e-7; a
    # subnormal scale has 20 bits at least (amax > 1e-37), half a step 2^-20
    tol = 2.0 ** -17
    assert bool((amax > 1e-37).all())
    assert bool(((s * 448 - amax).abs() <= tol * amax).all())
    ref = v / s[:, :, None]
    off = (codes.view(torch.float8_e4m3fn).double().view_as(v) - ref).abs()
    assert bool((off <= (2.0 ** -4 + tol) * ref.abs() + 2.0 ** -10).all())
