"""Host-side checks of the 8-bit integer and log-probability entry points (no
GPU): arguments are refused before anything is enqueued."""
import subprocess
import sys

import pytest


@pytest.fixture(scope="module")
def qg():
    import __graft_entry__
    __graft_entry__.build_library()
    import weight_only_quantized_qgemm_gb300 as q
    return q


FAKE = 0x100000  # never dereferenced: every call below ends in its checks


@pytest.mark.parametrize("args,expect", [
    # Xq, ldxq, Sx, W, Sw, bias, Y, y_type, ldy, M, N, K
    ((FAKE, 512, FAKE, FAKE, FAKE, None, FAKE, 0, 256, 0, 256, 512), 0),        # M == 0: no-op
    ((FAKE, 512, FAKE, FAKE, FAKE, None, FAKE, 0, 256, 4, 0, 512), 0),          # N == 0: no-op
    ((None, 512, FAKE, FAKE, FAKE, None, FAKE, 0, 256, 4, 256, 512), 1),
    ((FAKE, 512, None, FAKE, FAKE, None, FAKE, 0, 256, 4, 256, 512), 1),
    ((FAKE, 512, FAKE, None, FAKE, None, FAKE, 0, 256, 4, 256, 512), 1),
    ((FAKE, 512, FAKE, FAKE, None, None, FAKE, 0, 256, 4, 256, 512), 1),
    ((FAKE, 512, FAKE, FAKE, FAKE, None, None, 0, 256, 4, 256, 512), 1),
    ((FAKE, 512, FAKE, FAKE, FAKE, None, None, 0, 256, 4, 256, 0), 1),          # K == 0 writes Y too
    ((FAKE, 512, FAKE, FAKE, FAKE, None, FAKE, 3, 256, 4, 256, 512), 1),        # no such type
    ((FAKE, 512, FAKE, FAKE, FAKE, None, FAKE, 0, 256, -1, 256, 512), 1),
    ((FAKE, 512, FAKE, FAKE, FAKE, None, FAKE, 0, 256, 65537, 256, 512), 2),    # M > 65536
    ((FAKE, 520, FAKE, FAKE, FAKE, None, FAKE, 0, 256, 4, 256, 520), 2),        # K % 16
    ((FAKE, 256, FAKE, FAKE, FAKE, None, FAKE, 0, 256, 4, 256, 512), 1),        # ldxq < K
    ((FAKE, 512, FAKE, FAKE, FAKE, None, FAKE, 0, 255, 4, 256, 512), 1),        # ldy < N
    ((FAKE + 8, 512, FAKE, FAKE, FAKE, None, FAKE, 0, 256, 4, 256, 512), 3),
    ((FAKE, 520, FAKE, FAKE, FAKE, None, FAKE, 0, 256, 4, 256, 512), 3),        # ldxq % 16
    ((FAKE, 512, FAKE, FAKE + 8, FAKE, None, FAKE, 0, 256, 4, 256, 512), 3),
    ((FAKE, 512, FAKE + 2, FAKE, FAKE, None, FAKE, 0, 256, 4, 256, 512), 3),
    ((FAKE, 512, FAKE, FAKE, FAKE, FAKE + 1, FAKE, 0, 256, 4, 256, 512), 3),
    ((FAKE, 512, FAKE, FAKE, FAKE, None, FAKE + 2, 2, 256, 4, 256, 512), 3),    # FP32 Y
    ((FAKE, 512, FAKE, FAKE, FAKE, None, FAKE + 1, 1, 256, 4, 256, 512), 3),
])
def test_gemm_argument_validation(qg, args, expect):
    assert qg.lib.qgemm_w8a8_int8(*args, None, 0, None) == expect


@pytest.mark.parametrize("args,expect", [
    # X, x_type, ldx, Xq, ldxq, Sx, M, K
    ((FAKE, 0, 512, FAKE, 512, FAKE, 0, 512), 0),
    ((FAKE, 0, 512, FAKE, 512, FAKE, 4, 0), 0),
    ((None, 0, 512, FAKE, 512, FAKE, 4, 512), 1),
    ((FAKE, 0, 512, None, 512, FAKE, 4, 512), 1),
    ((FAKE, 0, 512, FAKE, 512, None, 4, 512), 1),
    ((FAKE, 2, 512, FAKE, 512, FAKE, 4, 512), 1),      # FP32 X
    ((FAKE, 0, 512, FAKE, 512, FAKE, 4, 504), 2),      # K % 16
    ((FAKE, 0, 512, FAKE, 512, FAKE, 65537, 512), 2),
    ((FAKE, 0, 504, FAKE, 512, FAKE, 4, 512), 1),
    ((FAKE, 0, 512, FAKE, 496, FAKE, 4, 512), 1),
    ((FAKE, 0, 516, FAKE, 512, FAKE, 4, 512), 3),
    ((FAKE, 1, 512, FAKE, 520, FAKE, 4, 512), 3),
    ((FAKE + 8, 1, 512, FAKE, 512, FAKE, 4, 512), 3),
    ((FAKE, 1, 512, FAKE, 512, FAKE + 2, 4, 512), 3),
])
def test_quantiser_argument_validation(qg, args, expect):
    assert qg.lib.qg_quantize_act_int8(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    # logits, type, ld, tokens, ldt, T, token_lp, entropy, top_k, top_ids, top_lp, M, V
    ((FAKE, 0, 100, FAKE, 1, 1, FAKE, FAKE, 4, FAKE, FAKE, 0, 100), 0),       # M == 0: no-op
    ((None, 0, 100, None, 0, 0, None, None, 0, None, None, 3, 100), 0),       # nothing asked
    ((None, 0, 100, FAKE, 1, 1, FAKE, FAKE, 4, FAKE, FAKE, 3, 100), 1),
    ((FAKE, 0, 100, None, 1, 1, FAKE, FAKE, 4, FAKE, FAKE, 3, 100), 1),
    ((FAKE, 0, 100, FAKE, 1, 1, None, FAKE, 4, FAKE, FAKE, 3, 100), 1),
    ((FAKE, 0, 100, FAKE, 1, 1, FAKE, None, 4, None, FAKE, 3, 100), 1),
    ((FAKE, 0, 100, FAKE, 1, 1, FAKE, None, 4, FAKE, None, 3, 100), 1),
    ((FAKE, 5, 100, FAKE, 1, 1, FAKE, FAKE, 4, FAKE, FAKE, 3, 100), 1),
    ((FAKE, 0, 100, FAKE, 1, -1, FAKE, FAKE, 4, FAKE, FAKE, 3, 100), 1),
    ((FAKE, 0, 100, FAKE, 1, 1, FAKE, FAKE, -1, FAKE, FAKE, 3, 100), 1),
    ((FAKE, 0, 99, FAKE, 1, 1, FAKE, FAKE, 4, FAKE, FAKE, 3, 100), 1),        # ld < V
    ((FAKE, 0, 100, FAKE, 1, 2, FAKE, FAKE, 4, FAKE, FAKE, 3, 100), 1),       # ldt < T
    ((FAKE, 0, 0, FAKE, 1, 1, FAKE, FAKE, 0, FAKE, FAKE, 3, 0), 2),           # V == 0
    ((FAKE, 0, 2 ** 31, FAKE, 1, 1, FAKE, FAKE, 0, FAKE, FAKE, 3, 2 ** 30 + 1), 2),   # a row longer than an index takes
    ((FAKE, 0, 100, FAKE, 1, 1, FAKE, FAKE, 33, FAKE, FAKE, 3, 100), 2),      # top_k > 32
    ((FAKE, 0, 100, FAKE, 1, 1, FAKE, FAKE, 9, FAKE, FAKE, 3, 8), 2),         # top_k > V
    ((FAKE + 1, 0, 100, FAKE, 1, 1, FAKE, FAKE, 4, FAKE, FAKE, 3, 100), 3),
    ((FAKE + 2, 2, 100, FAKE, 1, 1, FAKE, FAKE, 4, FAKE, FAKE, 3, 100), 3),
    ((FAKE, 0, 100, FAKE + 4, 1, 1, FAKE, FAKE, 4, FAKE, FAKE, 3, 100), 3),
    ((FAKE, 0, 100, FAKE, 1, 1, FAKE + 2, FAKE, 4, FAKE, FAKE, 3, 100), 3),
    ((FAKE, 0, 100, FAKE, 1, 1, FAKE, FAKE + 2, 4, FAKE, FAKE, 3, 100), 3),
    ((FAKE, 0, 100, FAKE, 1, 1, FAKE, FAKE, 4, FAKE + 4, FAKE, 3, 100), 3),
    ((FAKE, 0, 100, FAKE, 1, 1, FAKE, FAKE, 4, FAKE, FAKE + 2, 3, 100), 3),
])
def test_logprobs_argument_validation(qg, args, expect):
    assert qg.lib.qg_logprobs(*args, None) == expect


def test_dispatch_rule_covers_the_kind(qg):
    assert qg.dispatch_rule(qg.KIND_INT8, 16, 17408, 5120, 152) in range(1, 153)
    assert qg.dispatch_rule(qg.KIND_INT8, 65536, 17408, 5120, 152) in range(1, 153)
    assert qg.dispatch_rule(qg.KIND_INT8, 65537, 17408, 5120, 152) == 0
    assert qg.dispatch_rule(qg.KIND_INT8, 1, 1, 16, 152) == 1


@pytest.mark.parametrize("M,N,K,rows", [
    # the widths that measured fastest (or within 2% of it)
    (1, 1024, 5120, 16), (16, 17408, 5120, 16), (32, 32768, 5120, 32), (64, 5120, 5120, 64), (64, 17408, 5120, 64),
    (100, 1000, 1008, 16), (128, 512, 512, 16), (128, 17408, 5120, 128), (172, 4218, 1456, 64), (256, 5120, 17408, 256),
    (1024, 17408, 5120, 256), (4096, 17408, 5120, 256),
])
def test_tile_width_rule(qg, M, N, K, rows):
    assert qg.int8_tile_rows(M, N, K, 152) == rows


def test_schedule_rule_invariants(qg):
    """Any shape and SM count: a legal width, a grid of at least one CTA (an
    even one for pairs), no more than the SMs; invalid arguments give 0."""
    for sms in (1, 2, 3, 76, 132, 152):
        for M in (1, 15, 16, 17, 33, 64, 65, 129, 300, 4096, 65536):
            for N in (1, 127, 129, 5003, 151936):
                for K in (16, 128, 144, 5120):
                    rows = qg.int8_tile_rows(M, N, K, sms)
                    g = qg.dispatch_rule(qg.KIND_INT8, M, N, K, sms)
                    assert rows in (16, 32, 64, 128, 256) and (rows < 2 * M or rows == 16)
                    assert 1 <= g <= max(sms, 2) and (rows < 128 or g % 2 == 0), (M, N, K, sms, rows, g)
    assert qg.int8_tile_rows(0, 1, 16, 152) == 0 and qg.int8_tile_rows(1, 1, 16, 0) == 0


@pytest.mark.parametrize("kind,M,N,K", [
    (4, 65536, 2 ** 31 - 1, 16), (4, 65536, 2 ** 30, 5120), (4, 65536, 2 ** 24 + 1, 2 ** 31 - 16), (4, 32769, 2 ** 25, 16),
    (3, 65536, 2 ** 31 - 1, 16), (3, 65536, 2 ** 30, 5120), (3, 65536, 2 ** 25 + 1, 2 ** 31 - 16), (3, 32769, 2 ** 26, 16),
])
def test_too_many_tiles_are_refused(qg, kind, M, N, K):
    """More than 2^29 tiles (whose number leaves an int): the questions about
    the schedule answer 0 and none divides by zero.  In a process of its own."""
    code = (f"import weight_only_quantized_qgemm_gb300 as q; k, s = {kind}, ({M}, {N}, {K})\n"
            "print([q.dispatch_rule(k, *s, n) for n in (1, 76, 152)], q.workspace_bytes(k, *s), q.dispatch_get(k, *s),\n"
            "      q.lib.qg_dispatch_set(k, *s, 1), q.int8_tile_rows(*s, 152) if k == 4 else 0)")
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert p.returncode == 0, (p.returncode, p.stderr[-500:])
    assert p.stdout.split("\n")[0] == "[0, 0, 0] 0 0 2 0"


@pytest.mark.parametrize("M,N,K", [(65536, 2 ** 24, 16), (65536, 2 ** 24, 2 ** 20), (65536, 2 ** 24, 2 ** 31 - 16),
                                   (1, 2 ** 31 - 1, 16), (1, 2 ** 31 - 1, 2 ** 31 - 16)])
def test_the_most_tiles_have_a_schedule(qg, M, N, K):
    """At the limit itself, with short and long K, the rule answers as for any
    shape, with tiles as wide as a long K asks for."""
    for sms in (1, 76, 152):
        rows, g = qg.int8_tile_rows(M, N, K, sms), qg.dispatch_rule(qg.KIND_INT8, M, N, K, sms)
        assert rows == (16 if M == 1 else rows) and rows in (16, 32, 64, 128, 256)
        assert 1 <= g <= max(sms, 2), (sms, rows, g)
        if M > 1 and K >= 2 ** 20 and sms > 1:
            assert rows == 256, (sms, rows)


def test_the_binding_s_constants_are_the_header_s(qg):
    import os
    import re
    with open(os.path.join(os.path.dirname(qg.__file__), "..", "include", "qgemm.h")) as f:
        header = f.read()
    assert qg.MAX_TOP_K == int(re.search(r"#define QG_MAX_TOP_K (\d+)", header).group(1))
    assert qg.KIND_INT8 == int(re.search(r"QG_KIND_INT8 = (\d+)", header).group(1))
