"""Host-side checks of the expert layer's and the draft verification's entry
points (no GPU): arguments are refused before anything is enqueued, and what a
call makes belongs to its stream."""
import os
import re

import pytest
import torch

from test_streams_host import SIDE, Device, Stream, Tensor, _check_side, built, world  # noqa: F401


@pytest.fixture(scope="module")
def qg():
    import __graft_entry__
    __graft_entry__.build_library()
    import weight_only_quantized_qgemm_gb300 as q
    return q


FAKE = 0x100000  # never dereferenced: every call below ends in its checks
BIG = 2 ** 31 - 1


@pytest.mark.parametrize("args,expect", [
    # logits, type, ld, bias, score, renormalize, scale, top_k, experts, weights, offsets, rows, M, E
    ((None, 0, 64, None, 0, 1, 1.0, 4, FAKE, FAKE, FAKE, FAKE, 8, 64), 1),
    ((FAKE, 0, 64, None, 0, 1, 1.0, 4, None, FAKE, FAKE, FAKE, 8, 64), 1),
    ((FAKE, 0, 64, None, 0, 1, 1.0, 4, FAKE, None, FAKE, FAKE, 8, 64), 1),
    ((FAKE, 0, 64, None, 0, 1, 1.0, 4, FAKE, FAKE, None, FAKE, 8, 64), 1),
    ((FAKE, 0, 64, None, 0, 1, 1.0, 4, FAKE, FAKE, FAKE, None, 8, 64), 1),
    ((FAKE, 3, 64, None, 0, 1, 1.0, 4, FAKE, FAKE, FAKE, FAKE, 8, 64), 1),     # no such type
    ((FAKE, 0, 64, None, 2, 1, 1.0, 4, FAKE, FAKE, FAKE, FAKE, 8, 64), 1),     # no such score
    ((FAKE, 0, 64, None, 0, 1, 1.0, 0, FAKE, FAKE, FAKE, FAKE, 8, 64), 1),
    ((FAKE, 0, 63, None, 0, 1, 1.0, 4, FAKE, FAKE, FAKE, FAKE, 8, 64), 1),     # ld < E
    ((FAKE, 0, 64, None, 0, 1, 1.0, 4, FAKE, FAKE, FAKE, FAKE, -1, 64), 1),
    ((FAKE, 0, 64, None, 0, 1, 1.0, 65, FAKE, FAKE, FAKE, FAKE, 8, 64), 2),    # top_k > E
    ((FAKE, 0, 64, None, 0, 1, 1.0, 33, FAKE, FAKE, FAKE, FAKE, 8, 64), 2),    # top_k > 32
    ((FAKE, 0, 2000, None, 0, 1, 1.0, 4, FAKE, FAKE, FAKE, FAKE, 8, 1025), 2),
    ((FAKE, 0, 64, None, 0, 1, 1.0, 4, FAKE, FAKE, FAKE, FAKE, 2 ** 20 + 1, 64), 2),
    ((FAKE, 0, 64, None, 0, 1, 1.0, 1, FAKE, FAKE, FAKE, FAKE, 8, 0), 2),
    ((FAKE + 1, 0, 64, None, 0, 1, 1.0, 4, FAKE, FAKE, FAKE, FAKE, 8, 64), 3),
    ((FAKE + 2, 2, 64, None, 0, 1, 1.0, 4, FAKE, FAKE, FAKE, FAKE, 8, 64), 3),
    ((FAKE, 0, 64, FAKE + 2, 0, 1, 1.0, 4, FAKE, FAKE, FAKE, FAKE, 8, 64), 3),
    ((FAKE, 0, 64, None, 0, 1, 1.0, 4, FAKE + 2, FAKE, FAKE, FAKE, 8, 64), 3),
    ((FAKE, 0, 64, None, 0, 1, 1.0, 4, FAKE, FAKE, FAKE + 1, FAKE, 8, 64), 3),
])
def test_route_argument_validation(qg, args, expect):
    assert qg.lib.qg_moe_route(*args, None, 0, None) == expect


@pytest.mark.parametrize("args,expect", [
    # X, x_type, ldx, gated, rows, top_k, num_rows, Xq, ldxq, Sx, ldsx, M, out_rows, K
    ((FAKE, 0, 512, 0, FAKE, 2, None, FAKE, 512, FAKE, 32, 0, 16, 512), 0),
    ((FAKE, 0, 512, 0, FAKE, 2, None, FAKE, 512, FAKE, 32, 8, 0, 512), 0),
    ((FAKE, 0, 512, 0, FAKE, 2, None, FAKE, 512, FAKE, 32, 8, 16, 0), 0),
    ((None, 0, 512, 0, FAKE, 2, None, FAKE, 512, FAKE, 32, 8, 16, 512), 1),
    ((FAKE, 0, 512, 0, FAKE, 2, None, None, 512, FAKE, 32, 8, 16, 512), 1),
    ((FAKE, 0, 512, 0, FAKE, 2, None, FAKE, 512, None, 32, 8, 16, 512), 1),
    ((FAKE, 2, 512, 0, FAKE, 2, None, FAKE, 512, FAKE, 32, 8, 16, 512), 1),    # FP32 X
    ((FAKE, 0, 512, 0, FAKE, 0, None, FAKE, 512, FAKE, 32, 8, 16, 512), 1),    # rows of no places
    ((FAKE, 0, 1016, 1, None, 0, None, FAKE, 512, FAKE, 32, 8, 16, 512), 1),   # gated: ldx < 2 K
    ((FAKE, 0, 512, 0, FAKE, 2, None, FAKE, 496, FAKE, 32, 8, 16, 512), 1),
    ((FAKE, 0, 512, 0, FAKE, 2, None, FAKE, 512, FAKE, 12, 8, 16, 512), 1),    # ldsx < out_rows
    ((FAKE, 0, 512, 0, FAKE, 2, None, FAKE, 512, FAKE, 32, 8, 16, 504), 2),
    ((FAKE, 0, 512, 0, FAKE, 33, None, FAKE, 512, FAKE, 32, 8, 16, 512), 2),
    ((FAKE, 0, 512, 0, FAKE, 2, None, FAKE, 512, FAKE, 32, 2 ** 22 + 1, 16, 512), 2),
    ((FAKE, 0, 2 ** 31, 0, FAKE, 2, None, FAKE, 2 ** 31, FAKE, 32, 8, 16, 2 ** 30 + 16), 2),
    ((FAKE + 8, 0, 512, 0, FAKE, 2, None, FAKE, 512, FAKE, 32, 8, 16, 512), 3),
    ((FAKE, 0, 516, 0, FAKE, 2, None, FAKE, 512, FAKE, 32, 8, 16, 512), 3),
    ((FAKE, 0, 512, 0, FAKE, 2, None, FAKE, 520, FAKE, 32, 8, 16, 512), 3),
    ((FAKE, 0, 512, 0, FAKE, 2, None, FAKE, 512, FAKE, 33, 8, 16, 512), 3),
    ((FAKE, 0, 512, 0, FAKE + 2, 2, None, FAKE, 512, FAKE, 32, 8, 16, 512), 3),
    ((FAKE, 0, 512, 0, FAKE, 2, FAKE + 2, FAKE, 512, FAKE, 32, 8, 16, 512), 3),
])
def test_row_quantiser_argument_validation(qg, args, expect):
    assert qg.lib.qg_quantize_rows_e4m3(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    # Xq, ldxq, Sx, ldsx, W, Sw, offsets, Y, y_type, ldy, R, E, N, K
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 0, 8, 256, 512), 0),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 0, 256, 512), 0),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 8, 0, 512), 0),
    ((None, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 1),
    ((FAKE, 512, None, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 1),
    ((FAKE, 512, FAKE, 64, None, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 1),
    ((FAKE, 512, FAKE, 64, FAKE, None, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 1),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, None, FAKE, 0, 256, 40, 8, 256, 512), 1),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE, None, 0, 256, 40, 8, 256, 0), 1),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 3, 256, 40, 8, 256, 512), 1),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, -1, 8, 256, 512), 1),
    ((FAKE, 496, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 1),
    ((FAKE, 512, FAKE, 36, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 1),   # ldsx < R
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 255, 40, 8, 256, 512), 1),
    ((FAKE, 520, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 520), 2),
    ((FAKE, 2 ** 31, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 2 ** 31 - 16), 2),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 1025, 256, 512), 2),
    ((FAKE, 512, FAKE, 2 ** 25, FAKE, FAKE, FAKE, FAKE, 0, 256, 2 ** 24 + 1, 8, 256, 512), 2),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 2 ** 31, 40, 8, 2 ** 28, 512), 2),   # E N = 2^31
    ((FAKE, 512, FAKE, 2 ** 24, FAKE, FAKE, FAKE, FAKE, 0, 2 ** 31, 2 ** 24, 1, 2 ** 31 - 300, 512), 2),   # tiles
    ((FAKE + 8, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 3),
    ((FAKE, 520, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 3),
    ((FAKE, 512, FAKE + 4, 64, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 3),
    ((FAKE, 512, FAKE, 63, FAKE, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 3),   # ldsx % 4
    ((FAKE, 512, FAKE, 64, FAKE + 8, FAKE, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 3),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE + 2, FAKE, FAKE, 0, 256, 40, 8, 256, 512), 3),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE + 2, FAKE, 0, 256, 40, 8, 256, 512), 3),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE + 1, 0, 256, 40, 8, 256, 512), 3),
    ((FAKE, 512, FAKE, 64, FAKE, FAKE, FAKE, FAKE + 2, 2, 256, 40, 8, 256, 512), 3),
])
def test_grouped_argument_validation(qg, args, expect):
    assert qg.lib.qgemm_w8a8_grouped(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    # Y, type, ldy, rows, weights, top_k, residual, ldr, out, ldo, M, R, K
    ((FAKE, 0, 256, FAKE, FAKE, 2, None, 0, FAKE, 256, 0, 16, 256), 0),
    ((FAKE, 0, 256, FAKE, FAKE, 2, None, 0, FAKE, 256, 8, 16, 0), 0),
    ((None, 0, 256, FAKE, FAKE, 2, None, 0, FAKE, 256, 8, 16, 256), 1),
    ((FAKE, 0, 256, None, FAKE, 2, None, 0, FAKE, 256, 8, 16, 256), 1),
    ((FAKE, 0, 256, FAKE, None, 2, None, 0, FAKE, 256, 8, 16, 256), 1),
    ((FAKE, 0, 256, FAKE, FAKE, 2, None, 0, None, 256, 8, 16, 256), 1),
    ((FAKE, 0, 256, FAKE, FAKE, 0, None, 0, FAKE, 256, 8, 16, 256), 1),
    ((FAKE, 4, 256, FAKE, FAKE, 2, None, 0, FAKE, 256, 8, 16, 256), 1),
    ((FAKE, 0, 255, FAKE, FAKE, 2, None, 0, FAKE, 256, 8, 16, 256), 1),
    ((FAKE, 0, 256, FAKE, FAKE, 2, FAKE, 255, FAKE, 256, 8, 16, 256), 1),
    ((FAKE, 0, 256, FAKE, FAKE, 2, None, 0, FAKE, 255, 8, 16, 256), 1),
    ((FAKE, 0, 256, FAKE, FAKE, 33, None, 0, FAKE, 256, 8, 16, 256), 2),
    ((FAKE, 0, 256, FAKE, FAKE, 2, None, 0, FAKE, 256, 2 ** 22 + 1, 16, 256), 2),
    ((FAKE, 0, 2 ** 30, FAKE, FAKE, 2, None, 0, FAKE, 2 ** 30, 2 ** 10, 16, 2 ** 29), 2),
    ((FAKE, 0, 2 ** 31, FAKE, FAKE, 2, None, 0, FAKE, 2 ** 31, 1, 16, BIG), 2),
    ((FAKE + 1, 0, 256, FAKE, FAKE, 2, None, 0, FAKE, 256, 8, 16, 256), 3),
    ((FAKE, 2, 256, FAKE, FAKE, 2, FAKE + 2, 256, FAKE, 256, 8, 16, 256), 3),
    ((FAKE, 0, 256, FAKE + 2, FAKE, 2, None, 0, FAKE, 256, 8, 16, 256), 3),
    ((FAKE, 0, 256, FAKE, FAKE + 2, 2, None, 0, FAKE, 256, 8, 16, 256), 3),
])
def test_combine_argument_validation(qg, args, expect):
    assert qg.lib.qg_moe_combine(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    # target, type, t_seq, t_row, draft, d_seq, d_row, tokens, ldt, uniform, ldu, noise, ldn, lengths, acc, out, B, G, V
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 0, 4, 100), 0),
    ((None, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 1),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, None, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 1),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, None, None, FAKE, 2, 4, 100), 1),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, None, FAKE, None, 2, 4, 100), 1),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, None, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 1),
    ((FAKE, 0, 500, 100, None, 400, 100, FAKE, 4, FAKE, 4, None, 100, None, FAKE, FAKE, 2, 4, 100), 1),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, None, 4, None, 100, None, FAKE, FAKE, 2, 4, 100), 1),
    ((FAKE, 3, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 1),
    ((FAKE, 0, 500, 99, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 1),
    ((FAKE, 0, 500, 100, FAKE, 400, 99, FAKE, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 1),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 3, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 1),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 3, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 1),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 99, None, FAKE, FAKE, 2, 4, 100), 1),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 32, FAKE, 32, FAKE, 100, None, FAKE, FAKE, 2, 32, 100), 2),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 65537, 4, 100), 2),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 0), 2),
    ((FAKE + 1, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 3),
    ((FAKE, 2, 500, 100, FAKE + 2, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 3),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE + 4, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 3),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE + 2, 4, FAKE, 100, None, FAKE, FAKE, 2, 4, 100), 3),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, FAKE + 2, FAKE, FAKE, 2, 4, 100), 3),
    ((FAKE, 0, 500, 100, FAKE, 400, 100, FAKE, 4, FAKE, 4, FAKE, 100, None, FAKE, FAKE + 4, 2, 4, 100), 3),
])
def test_verify_argument_validation(qg, args, expect):
    assert qg.lib.qg_verify_drafts(*args, None, 0, None) == expect


def test_the_binding_s_constants_are_the_header_s(qg):
    with open(os.path.join(os.path.dirname(qg.__file__), "..", "include", "qgemm.h")) as f:
        header = f.read()
    for name, value in (("QG_MAX_EXPERTS", qg.MAX_EXPERTS), ("QG_MAX_DRAFTS", qg.MAX_DRAFTS)):
        assert value == int(re.search(rf"#define {name} (\d+)", header).group(1))
    assert "QG_SCORE_SOFTMAX = 0, QG_SCORE_SIGMOID = 1" in header and qg._SCORES == {"softmax": 0, "sigmoid": 1}


# ----------------------------------------------------------------- the binding, on stand-ins
def _calls(w, device=None):
    q = w.q

    def T(*shape, dtype=torch.float32):
        return Tensor(w, shape, dtype, device=device)

    i32, i64, bf, u8 = torch.int32, torch.int64, torch.bfloat16, torch.uint8
    return {
        "qg_moe_route": (4, lambda st: q.moe_route(T(40, 64), 4, bias=T(64), stream=st)),
        "qg_quantize_rows_e4m3": (2, lambda st: q.quantize_rows_e4m3(T(8, 256, dtype=bf), rows=T(8, 2, dtype=i32),
                                                                     num_rows=T(1, dtype=i32), stream=st)),
        "qgemm_w8a8_grouped": (1, lambda st: q.qgemm_w8a8_grouped(T(16, 256, dtype=u8), T(2, 32), T(4, 128, 256, dtype=u8),
                                                                  T(4, 1, 2), T(5, dtype=i32), stream=st)),
        "qg_moe_combine": (1, lambda st: q.moe_combine(T(16, 128, dtype=bf), T(8, 2, dtype=i32), T(8, 2),
                                                       residual=T(8, 128, dtype=bf), stream=st)),
        "qg_verify_drafts": (2, lambda st: q.verify_drafts(T(2, 4, 100), T(2, 3, dtype=i64), T(2, 3, 100), T(2, 3),
                                                           T(2, 100), T(2, dtype=i32), stream=st)),
    }


NAMES = ["qg_moe_route", "qg_quantize_rows_e4m3", "qgemm_w8a8_grouped", "qg_moe_combine", "qg_verify_drafts"]


@pytest.mark.parametrize("stream", [Stream(SIDE), SIDE], ids=["object", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_belong_to_the_call_s_stream(world, name, stream):   # noqa: F811
    world.q._scratch_need.clear()
    count, call = _calls(world)[name]
    call(stream)
    assert world.calls[-1][0] == name and world.calls[-1][2][-1] == SIDE
    assert sum(s == SIDE for _, s in world.made) == count, "the outputs, and nothing else"
    assert world.current.cuda_stream == 0
    world.q._scratch_need.clear()


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(world, name):   # noqa: F811
    for stream in (None, SIDE):
        with pytest.raises(ValueError, match="current CUDA device"):
            _calls(world, Device(1))[name][1](stream)
    assert not world.calls


def test_scratch_memory_is_the_call_s_own(world, monkeypatch):   # noqa: F811
    """What a call needs beside its outputs it makes itself, on its stream: two
    captured graphs share none."""
    q = world.q
    q._scratch_need.clear()

    class Lib:
        def __getattr__(self, name):
            return (lambda *a: 4096) if name.endswith("workspace_bytes") else world.entry(name)

    monkeypatch.setattr(q, "lib", Lib())
    for name, at in (("qg_moe_route", -3), ("qg_verify_drafts", -3)):
        world.made.clear()
        _calls(world)[name][1](SIDE)
        own = [t for t, s in world.made if s == SIDE and t.dtype == torch.uint8]
        assert len(own) == 1 and own[0].shape == (4096,)
        assert world.calls[-1][2][at:] == (0x100000, 4096, SIDE)
    q._scratch_need.clear()


def test_the_binding_refuses_what_does_not_fit(world):   # noqa: F811
    q = world.q

    def T(*shape, dtype=torch.float32, strides=None):
        return Tensor(world, shape, dtype, strides=strides)

    i32, i64, bf, u8 = torch.int32, torch.int64, torch.bfloat16, torch.uint8
    bad = [
        lambda: q.moe_route(T(4, 64, dtype=i32), 2),
        lambda: q.moe_route(T(4, 64), 2, score="linear"),
        lambda: q.moe_route(T(4, 64), 2, bias=T(63)),
        lambda: q.moe_route(T(4, 64), 2, bias=T(64, dtype=bf)),
        lambda: q.moe_route(T(4, 64), -1),
        lambda: q.moe_route(T(4, 64, strides=(1, 4)), 2),
        lambda: q.quantize_rows_e4m3(T(4, 64)),
        lambda: q.quantize_rows_e4m3(T(4, 63, dtype=bf), gated=True),
        lambda: q.quantize_rows_e4m3(T(4, 64, dtype=bf), rows=T(3, 2, dtype=i32)),
        lambda: q.quantize_rows_e4m3(T(4, 64, dtype=bf), rows=T(4, 2, dtype=i64)),
        lambda: q.quantize_rows_e4m3(T(4, 64, dtype=bf), rows=T(4, 2, dtype=i32, strides=(1, 4))),
        lambda: q.quantize_rows_e4m3(T(4, 64, dtype=bf), num_rows=T(2, dtype=i32)),
        lambda: q.quantize_rows_e4m3(T(4, 64, dtype=bf), Xq=T(5, 64, dtype=u8), out_rows=4),
        lambda: q.quantize_rows_e4m3(T(4, 64, dtype=bf), X_scale=T(1, 3)),
        lambda: q.quantize_rows_e4m3(T(4, 64, dtype=bf), X_scale=T(2, 32)),
        lambda: q.qgemm_w8a8_grouped(T(4, 64, dtype=u8), T(1, 32), T(2, 8, 64), T(2, 1, 1), T(3, dtype=i32)),
        lambda: q.qgemm_w8a8_grouped(T(4, 64, dtype=u8), T(1, 32), T(8, 64, dtype=u8), T(1, 1), T(3, dtype=i32)),
        lambda: q.qgemm_w8a8_grouped(T(4, 64, dtype=u8), T(1, 3), T(2, 8, 64, dtype=u8), T(2, 1, 1), T(3, dtype=i32)),
        lambda: q.qgemm_w8a8_grouped(T(4, 64, dtype=u8), T(1, 32), T(2, 8, 80, dtype=u8), T(2, 1, 1), T(3, dtype=i32)),
        lambda: q.qgemm_w8a8_grouped(T(4, 64, dtype=u8), T(1, 32), T(2, 8, 64, dtype=u8), T(2, 2, 1), T(3, dtype=i32)),
        lambda: q.qgemm_w8a8_grouped(T(4, 64, dtype=u8), T(1, 32), T(2, 8, 64, dtype=u8), T(2, 1, 1), T(2, dtype=i32)),
        lambda: q.qgemm_w8a8_grouped(T(4, 64, dtype=u8), T(1, 32), T(2, 8, 64, dtype=u8), T(2, 1, 1), T(3, dtype=i64)),
        lambda: q.qgemm_w8a8_grouped(T(4, 64, dtype=u8), T(1, 32), T(2, 8, 64, dtype=u8), T(2, 1, 1), T(3, dtype=i32),
                                     Y=T(4, 9)),
        lambda: q.qgemm_w8a8_grouped(T(4, 64, dtype=u8), T(1, 32), T(2, 8, 64, dtype=u8), T(2, 1, 1), T(3, dtype=i32),
                                     out_dtype=i32),
        lambda: q.moe_combine(T(8, 64, dtype=i32), T(4, 2, dtype=i32), T(4, 2)),
        lambda: q.moe_combine(T(8, 64), T(4, 2, dtype=i64), T(4, 2)),
        lambda: q.moe_combine(T(8, 64), T(4, 2, dtype=i32), T(4, 3)),
        lambda: q.moe_combine(T(8, 64), T(4, 2, dtype=i32), T(4, 2), residual=T(4, 64, dtype=bf)),
        lambda: q.moe_combine(T(8, 64), T(4, 2, dtype=i32), T(4, 2), out=T(5, 64)),
        lambda: q.verify_drafts(T(2, 4, 100, dtype=i32), T(2, 3, dtype=i64)),
        lambda: q.verify_drafts(T(2, 100), T(2, 3, dtype=i64)),
        lambda: q.verify_drafts(T(2, 4, 100), T(2, 4, dtype=i64)),
        lambda: q.verify_drafts(T(2, 4, 100), T(2, 3, dtype=i32)),
        lambda: q.verify_drafts(T(2, 4, 100), T(2, 3, dtype=i64), uniform=T(2, 3)),
        lambda: q.verify_drafts(T(2, 4, 100), T(2, 3, dtype=i64), T(2, 3, 100)),
        lambda: q.verify_drafts(T(2, 4, 100), T(2, 3, dtype=i64), T(2, 4, 100), T(2, 3), T(2, 100)),
        lambda: q.verify_drafts(T(2, 4, 100), T(2, 3, dtype=i64), T(2, 3, 100, dtype=bf), T(2, 3), T(2, 100)),
        lambda: q.verify_drafts(T(2, 4, 100), T(2, 3, dtype=i64), None, T(2, 2), T(2, 100)),
        lambda: q.verify_drafts(T(2, 4, 100), T(2, 3, dtype=i64), None, T(2, 3), T(2, 99)),
        lambda: q.verify_drafts(T(2, 4, 100), T(2, 3, dtype=i64), None, T(2, 3), T(2, 100), T(3, dtype=i32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            call()
        assert not world.calls, i


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 16])
def test_sizes_beyond_32_bits_are_refused(world, big):   # noqa: F811
    q = world.q

    def T(*shape, dtype=torch.float32):
        return Tensor(world, shape, dtype)

    i32, i64, bf, u8 = torch.int32, torch.int64, torch.bfloat16, torch.uint8
    for call in (lambda: q.moe_route(T(big, 8), 2), lambda: q.moe_route(T(8, big), 2), lambda: q.moe_route(T(8, 8), big),
                 lambda: q.quantize_rows_e4m3(T(big, 64, dtype=bf)),
                 lambda: q.quantize_rows_e4m3(T(4, 64, dtype=bf), out_rows=big),
                 lambda: q.qgemm_w8a8_grouped(T(big, 64, dtype=u8), T(1, big), T(2, 8, 64, dtype=u8), T(2, 1, 1),
                                              T(3, dtype=i32)),
                 lambda: q.moe_combine(T(big, 8), T(4, 2, dtype=i32), T(4, 2)),
                 lambda: q.verify_drafts(T(2, 1, big), T(2, 0, dtype=i64))):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    assert not world.calls


def test_grouped_tile_rows(qg):
    """Few rows take narrow tiles, many a pair's; invalid shapes none."""
    rows = [qg.grouped_tile_rows(64 * n, 64, 4096, 2048, 152) for n in (1, 8, 16, 48, 96, 1000)]
    assert rows == sorted(rows) and rows[0] == 16 and rows[-1] == 256
    # few tiles: narrow ones, which fill more of the device
    assert qg.grouped_tile_rows(200, 4, 870, 6432, 152) < qg.grouped_tile_rows(200 * 50, 200, 870, 6432, 152)
    for bad in ((0, 4, 64, 64, 152), (4, 0, 64, 64, 152), (4, 1025, 64, 64, 152), (4, 4, 0, 64, 152), (4, 4, 64, 60, 152),
                (4, 4, 64, 0, 152), (4, 4, 64, 64, 1), (2 ** 24 + 1, 4, 64, 64, 152)):
        assert qg.grouped_tile_rows(*bad) == 0
