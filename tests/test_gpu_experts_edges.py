"""The experts' operators on the GPU at the ends of what their contracts allow,
against plain implementations in 64 bits (tolerances as in test_gpu_experts.py)."""

import pytest
import torch

from gpu_util import qg
from test_gpu_experts import DTYPES

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
