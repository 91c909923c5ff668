"""Host side of the experts' operators at the ends of what their contracts allow
(no GPU)."""
import pytest
import torch

from test_streams_host import Tensor, built, world  # noqa: F401


class Part(Tensor):
    """A stand-in for the first columns of a tensor whose memory ends after `floats`."""

    def __init__(self, w, shape, strides, floats):
        super().__init__(w, shape, torch.float32, strides=strides)
        self.floats = floats

    def storage_offset(self):
        return 0

    def untyped_storage(self):
        return self

    def nbytes(self):
        return 4 * self.floats


@pytest.mark.parametrize("K,shape,strides,floats,pitch", [
    (128, (1, 37), (64, 1), 64, 40),      # the first columns of a padded row
    (128, (1, 37), (37, 1), 40, 40),      # a lone row's stride does not count
    (128, (1, 40), (40, 1), 40, 40),
    (128, (1, 64), (64, 1), 64, 40),
    (256, (2, 37), (64, 1), 128, 64),
    (256, (2, 37), (64, 1), 104, 64),
])
def test_scales_without_their_padding(world, K, shape, strides, floats, pitch):   # noqa: F811
    q, u8 = world.q, torch.uint8
    q.qgemm_w8a8_grouped(Tensor(world, (37, K), u8), Part(world, shape, strides, floats), Tensor(world, (2, 8, K), u8),
                         Tensor(world, (2, 1, K // 128), torch.float32), Tensor(world, (3,), torch.int32))
    name, _, args = world.calls[-1]
    assert name == "qgemm_w8a8_grouped" and args[3] == pitch
    q.quantize_rows_e4m3(Tensor(world, (37, K), torch.bfloat16), X_scale=Part(world, shape, strides, floats))
    name, _, args = world.calls[-1]
    assert name == "qg_quantize_rows_e4m3" and args[10] == pitch


@pytest.mark.parametrize("K,shape,strides,floats", [(128, (1, 37), (37, 1), 37), (128, (1, 37), (37, 1), 39),
                                                    (256, (2, 37), (64, 1), 101), (256, (2, 37), (64, 1), 103)])
def test_scales_whose_memory_ends_at_once_are_refused(world, K, shape, strides, floats):   # noqa: F811
    q, u8 = world.q, torch.uint8
    with pytest.raises(ValueError, match="multiple of 4"):
        q.qgemm_w8a8_grouped(Tensor(world, (37, K), u8), Part(world, shape, strides, floats), Tensor(world, (2, 8, K), u8),
                             Tensor(world, (2, 1, K // 128), torch.float32), Tensor(world, (3,), torch.int32))
    assert not world.calls


@pytest.mark.parametrize("sms", [1, 2, 3, 7, 8, 15, 16, 17, 64, 152])
def test_the_router_s_counts_fit_16_bits(built, sms):   # noqa: F811
    """A CTA's tokens, whatever the number of SMs: their counts by expert, of 16 bits,
    would wrap."""
    import ctypes
    need = built.lib["_ZN2qg21route_workspace_bytesEiii"]   # qg::route_workspace_bytes(M, E, sms)
    need.restype, need.argtypes = ctypes.c_size_t, [ctypes.c_int] * 3
    for E in (8, 256, 1024):
        for M in [1, 16, 17, 32, 33, 1000, 65535, 65536, 2 * 65535, 2 * 65535 + 1, 17 * 2 ** 15, 2 ** 20 - 1, 2 ** 20]:
            table = need(M, E, sms)
            ctas = table // (2 * E)   # E is a multiple of 8
            assert table == 2 * E * ctas
            if ctas:
                assert 1 < ctas <= M and -(-M // ctas) < 2 ** 16
            else:      # one CTA, whose counts have 32 bits
                assert M < 65536 or sms == 1


def test_what_is_kept_of_sizes_stays_small(world):   # noqa: F811
    """The scratch memory's size is kept for sizes that come again, not for every one ever seen."""
    q, i64 = world.q, torch.int64
    q._scratch_need.clear()
    most = 0
    for n in range(1, 2500):
        q.moe_route(Tensor(world, (n, 64), torch.float32), 4)
        q.verify_drafts(Tensor(world, (n, 2, 100), torch.float32), Tensor(world, (n, 1), i64))
        most = max(most, len(q._scratch_need))
    assert 2 <= most <= 2048
    assert sum(name in ("qg_moe_route", "qg_verify_drafts") for name, _, _ in world.calls) == 2 * 2499
    world.calls.clear()
    q._scratch_need.clear()
    for _ in range(3):
        q.moe_route(Tensor(world, (5, 64), torch.float32), 4)
    assert [c[0] for c in world.calls] == ["qg_moe_route_workspace_bytes"] + 3 * ["qg_moe_route"]
    q._scratch_need.clear()
