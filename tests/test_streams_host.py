"""Which stream the entry points' own memory belongs to (no GPU): a call with
``stream=`` makes its outputs, copies and intermediate tensors on that stream,
where the kernel that writes or reads them runs.  Tensors, streams and the
library are stand-ins that record the current stream."""
import contextlib

import pytest
import torch


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build_library()
    import weight_only_quantized_qgemm_gb300 as q
    return q


class Device:
    def __init__(self, index=0):
        self.type, self.index = "cuda", index

    def __eq__(self, other):
        return isinstance(other, Device) and other.index == self.index

    def __hash__(self):
        return hash(self.index)


class Stream:
    def __init__(self, handle, device=0):
        self.cuda_stream, self.device_index = int(handle), device


class Tensor:
    def __init__(self, world, shape, dtype, strides=None, device=None):
        self.world, self.shape, self.dtype = world, tuple(shape), dtype
        self.device, self.is_cuda = device or Device(), True
        if strides is None:
            strides, n = [], 1
            for s in reversed(self.shape):
                strides.insert(0, n)
                n *= s
        self.strides = tuple(strides)
        world.made.append((self, world.current.cuda_stream))

    def dim(self):
        return len(self.shape)

    def stride(self, d=None):
        return self.strides if d is None else self.strides[d]

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def element_size(self):
        return 1

    def is_contiguous(self):
        n = 1
        for s, t in zip(reversed(self.shape), reversed(self.strides)):
            if s != 1 and t != n:
                return False
            n *= s
        return True

    def contiguous(self):
        return self if self.is_contiguous() else Tensor(self.world, self.shape, self.dtype, device=self.device)

    def zero_(self):
        return self.fill_(0)

    def fill_(self, value):
        self.world.made.append((self, self.world.current.cuda_stream))
        return self

    def __getitem__(self, item):
        return self

    def data_ptr(self):
        return 0x100000


class World:
    """The stand-in for torch and the library: `made` holds (tensor, stream it
    was made on), `calls` (entry point, stream that was current, arguments)."""

    def __init__(self):
        self.current = Stream(0)
        self.device = 0
        self.made, self.calls = [], []
        self.cuda = self
        self.Stream = Stream

    def __getattr__(self, name):   # dtypes and the like
        return getattr(torch, name)

    # torch
    def empty(self, shape, dtype=None, device=None):
        return Tensor(self, shape, dtype)

    def empty_like(self, t):
        return Tensor(self, t.shape, t.dtype)

    def zeros(self, shape, dtype=None, device=None):
        return Tensor(self, (shape,) if isinstance(shape, int) else shape, dtype)

    # torch.cuda
    def current_stream(self, device=None):
        return self.current

    def current_device(self):
        return self.device

    def default_stream(self, device=None):
        return Stream(0)

    def ExternalStream(self, handle, device=None):
        return Stream(handle)

    def synchronize(self, device=None):
        pass

    @contextlib.contextmanager
    def stream(self, s):
        before, device = self.current, self.device
        self.current, self.device = s, s.device_index
        try:
            yield
        finally:
            self.current, self.device = before, device

    # the library
    def entry(self, name):
        def call(*args):
            self.calls.append((name, self.current.cuda_stream, args))
            return 0
        return call


@pytest.fixture
def world(built, monkeypatch):
    w = World()

    class Lib:
        def __getattr__(self, name):
            return (lambda *a: 4096) if name == "qg_workspace_bytes" else w.entry(name)

    monkeypatch.setattr(built, "lib", Lib())
    monkeypatch.setattr(built, "_torch", lambda: w)
    monkeypatch.setattr(built, "_raw_stream", lambda index: w.current.cuda_stream)
    monkeypatch.setattr(built, "_current_device", lambda: w.device, raising=False)
    monkeypatch.setattr(built, "_dtype_codes", {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    monkeypatch.setattr(built, "_default_ws", {})
    monkeypatch.setattr(built, "_ws_need", {})
    w.q = built
    return w


SIDE = 0x7000


def _check_side(w, before, name):
    """All that was made since `before`, and the call, belong to the side stream."""
    assert w.calls and w.calls[-1][0] == name and w.calls[-1][2][-1] == SIDE
    made = w.made[before:]
    assert made and all(s == SIDE for _, s in made), [(t.shape, s) for t, s in made]
    assert w.current.cuda_stream == 0, "the caller's stream is current again"


@pytest.mark.parametrize("stream", [Stream(SIDE), SIDE], ids=["object", "handle"])
@pytest.mark.parametrize("strides", [(0, 0), (1, 7), (0, 1)], ids=["expanded", "transposed", "one row of tokens"])
def test_logprobs_copies_strided_tokens_on_its_stream(world, stream, strides):
    x = Tensor(world, (7, 100), torch.bfloat16)
    tokens = Tensor(world, (7, 3), torch.int64, strides=strides)
    n = len(world.made)
    world.q.logprobs(x, tokens, top_k=2, entropy=True, stream=stream)
    copies = [t for t, _ in world.made[n:] if t.dtype == torch.int64 and t.shape == (7, 3)]
    assert len(copies) == 1
    _check_side(world, n, "qg_logprobs")


@pytest.mark.parametrize("stream", [Stream(SIDE), SIDE], ids=["object", "handle"])
def test_int8_outputs_belong_to_the_call_s_stream(world, stream):
    q = world.q
    X = Tensor(world, (4, 64), torch.bfloat16)
    n = len(world.made)
    q.quantize_act_int8(X, stream=stream)
    _check_side(world, n, "qg_quantize_act_int8")
    Xq, W = Tensor(world, (4, 64), torch.int8), Tensor(world, (8, 64), torch.int8)
    sx, sw = Tensor(world, (4,), torch.float32), Tensor(world, (8,), torch.float32)
    n = len(world.made)
    q.qgemm_w8a8_int8(Xq, sx, W, sw, out_dtype=torch.float16, stream=stream)   # Y and its stream's workspace
    _check_side(world, n, "qgemm_w8a8_int8")
    assert {t.dtype for t, _ in world.made[n:]} == {torch.float16, torch.uint8}
    # the same call on the caller's stream has a workspace of its own
    n = len(world.made)
    q.qgemm_w8a8_int8(Xq, sx, W, sw)
    assert [s for _, s in world.made[n:]] == [0, 0]


def test_a_stream_of_zero_is_the_default_stream(world):
    x = Tensor(world, (7, 100), torch.bfloat16)
    with world.stream(Stream(SIDE)):
        n = len(world.made)
        world.q.logprobs(x, entropy=True, stream=0)
        assert world.calls[-1][2][-1] == 0 and all(s == 0 for _, s in world.made[n:])
        assert world.current.cuda_stream == SIDE


def _older_calls(w):
    q, T, K = w.q, lambda *a, **k: Tensor(w, *a, **k), 256
    bf = lambda r: T((r, K), torch.bfloat16)     # noqa: E731
    codes = lambda n: (T((n, K), torch.uint8), T((-(-n // 128), 2), torch.float32))   # noqa: E731
    lut = (T((1 << 14,), torch.uint8), T((8,), torch.float16), T((128, 2), torch.float16), 128)
    return {
        "qgemm_fp8_block": lambda st: q.qgemm_fp8_block(bf(4), *codes(128), stream=st),
        "qgemm_fp8_block_multi": lambda st: q.qgemm_fp8_block_multi(bf(4), [codes(128), codes(200)], stream=st),
        "qgemm_lut3": lambda st: q.qgemm_lut3(T((4, K), torch.float16), *lut, stream=st),
        "qgemm_bf16": lambda st: q.qgemm_bf16(bf(4), bf(128), stream=st),
        "qg_quantize_act_e4m3": lambda st: q.quantize_act_e4m3(bf(4), stream=st),
        "qgemm_w8a8_block": lambda st: q.qgemm_w8a8(bf(4), *codes(128), stream=st),
        "qg_debug_fp8_split": lambda st: q.debug_fp8_split(T((3, 128), torch.bfloat16), stream=st),
        "qg_dequant_lut3": lambda st: q.dequant_lut3(*lut, K, stream=st),
    }


@pytest.mark.parametrize("name", ["qgemm_fp8_block", "qgemm_fp8_block_multi", "qgemm_lut3", "qgemm_bf16",
                                  "qg_quantize_act_e4m3", "qgemm_w8a8_block", "qg_debug_fp8_split", "qg_dequant_lut3"])
def test_outputs_of_every_entry_point_belong_to_its_stream(world, monkeypatch, name):
    monkeypatch.setattr(world.q, "lut3_packed_bytes", lambda N, K: 1 << 14)
    world.calls.clear()
    _older_calls(world)[name](SIDE)
    inputs = [t for t, s in world.made if s == 0]
    assert all(c[2][-1] == SIDE for c in world.calls) and world.calls[-1][0] == name
    assert len(world.made) > len(inputs)
    # what the call made itself: everything that is not one of its inputs
    outputs = {"qgemm_fp8_block": 2, "qgemm_fp8_block_multi": 3, "qgemm_lut3": 2, "qgemm_bf16": 2,
               "qg_quantize_act_e4m3": 2, "qgemm_w8a8_block": 4, "qg_debug_fp8_split": 3, "qg_dequant_lut3": 1}
    assert sum(s == SIDE for _, s in world.made) == outputs[name]


def test_tensors_of_another_device_are_refused(world):
    """The library launches on the current device: tensors of another one are
    refused before the call, under a stream of this device too."""
    q, other = world.q, Device(1)

    def T(*shape, dtype=torch.int8):
        return Tensor(world, shape, dtype, device=other)

    f = torch.float32
    for stream in (None, SIDE):
        for call in (lambda: q.quantize_act_int8(T(4, 64, dtype=torch.bfloat16), stream=stream),
                     lambda: q.qgemm_w8a8_int8(T(4, 64), T(4, dtype=f), T(8, 64), T(8, dtype=f), stream=stream),
                     lambda: q.logprobs(T(4, 100, dtype=f), entropy=True, stream=stream)):
            with pytest.raises(ValueError, match="current CUDA device"):
                call()
    assert not world.calls
    with world.stream(Stream(SIDE, device=1)):   # which makes device 1 current
        q.logprobs(T(4, 100, dtype=f), entropy=True)
    q.logprobs(T(4, 100, dtype=f), entropy=True, stream=Stream(SIDE, device=1))
    assert len(world.calls) == 2


def test_scales_of_rows_of_nothing_are_filled_on_the_call_s_stream(world):
    X = Tensor(world, (4, 0), torch.bfloat16)
    n = len(world.made)
    world.q.quantize_act_int8(X, stream=SIDE)
    filled = [t for t, _ in world.made[n:] if t.shape == (4,)]
    assert len(filled) == 2 and filled[0] is filled[1]   # made, then filled
    assert all(s == SIDE for _, s in world.made[n:])


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 16])
def test_sizes_beyond_32_bits_are_refused(world, big):
    """The library takes sizes as 32-bit numbers: larger ones would arrive as
    what is left of them."""
    q, f = world.q, torch.float32

    def T(*shape, dtype=torch.int8):
        return Tensor(world, shape, dtype)

    bf = torch.bfloat16
    for call in (lambda: q.quantize_act_int8(T(big, 64, dtype=bf)),
                 lambda: q.quantize_act_int8(T(4, big, dtype=bf)),
                 lambda: q.qgemm_w8a8_int8(T(big, 64), T(big, dtype=f), T(8, 64), T(8, dtype=f)),
                 lambda: q.qgemm_w8a8_int8(T(4, big), T(4, dtype=f), T(8, big), T(8, dtype=f)),
                 lambda: q.qgemm_w8a8_int8(T(4, 64), T(4, dtype=f), T(big, 64), T(big, dtype=f)),
                 lambda: q.logprobs(T(big, 16, dtype=f), entropy=True),
                 lambda: q.logprobs(T(4, big, dtype=f), entropy=True),
                 lambda: q.logprobs(T(4, 16, dtype=f), T(4, big, dtype=torch.int64)),
                 lambda: q.logprobs(T(4, 16, dtype=f), top_k=big)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    assert not world.calls


def test_a_workspace_keeps_the_buffers_that_it_outgrows(world):
    """A captured graph holds the addresses of the buffers of its calls: they
    stay allocated when a larger call needs a new one, and each is at least
    twice the one before, so that they add up to less than the newest."""
    import gc
    import weakref
    q = world.q
    ws = q.Workspace()
    seen, sizes = [], []
    for n in (1 << 20, (1 << 20) + 1, 3 << 20, 5 << 20, 1 << 24):
        buf = ws.get(n, q.KIND_INT8)
        assert buf.numel() >= n
        if not sizes or buf.numel() != sizes[-1]:
            sizes.append(buf.numel())
            seen.append(weakref.ref(buf))
    del buf
    world.made.clear()
    gc.collect()
    assert len(sizes) > 2 and all(r() is not None for r in seen)
    assert all(b >= 2 * a for a, b in zip(sizes, sizes[1:]))
    assert ws.get(64, q.KIND_INT8) is seen[-1]()


def test_the_current_stream_is_not_switched_to(world, monkeypatch):
    """stream= the current one: nothing to switch, which costs the host as much
    as a small call."""
    q = world.q
    x = Tensor(world, (4, 64), torch.bfloat16)
    for current in (Stream(SIDE), Stream(0)):
        with world.stream(current):
            with monkeypatch.context() as mp:
                mp.setattr(world, "stream", None, raising=False)
                for stream in (current, current.cuda_stream):
                    q.quantize_act_int8(x, stream=stream)
                    q.logprobs(x, entropy=True, stream=stream)
                    q.qgemm_bf16(x, Tensor(world, (128, 64), torch.bfloat16), stream=stream)
                    assert world.calls[-1][2][-1] == current.cuda_stream
    # the default streams of two devices have one handle
    y = Tensor(world, (4, 64), torch.bfloat16, device=Device(1))
    q.logprobs(y, entropy=True, stream=Stream(0, device=1))
    assert world.device == 0


def test_calls_with_all_outputs_given_hand_the_stream_on(world, monkeypatch):
    q = world.q

    def T(*shape, dtype=torch.bfloat16):
        return Tensor(world, shape, dtype)

    X, W, i8, f = T(4, 256), T(128, 256), torch.int8, torch.float32
    codes = T(128, 256, dtype=torch.uint8), T(1, 2, dtype=f)
    Xq, sx = T(4, 256, dtype=i8), T(4, dtype=f)
    ws = q.Workspace()
    for kind in (q.KIND_FP8_BLOCK, q.KIND_W8A8, q.KIND_INT8):
        ws.get(4096, kind)
    n = len(world.made)
    monkeypatch.setattr(world, "stream", None, raising=False)
    for call in (lambda st: q.qgemm_fp8_block(X, *codes, Y=X, workspace=ws, stream=st),
                 lambda st: q.qgemm_fp8_block_multi(X, [codes], Ys=[X], workspace=ws, stream=st),
                 lambda st: q.qgemm_bf16(X, W, Y=X, workspace=ws, stream=st),
                 lambda st: q.quantize_act_int8(X, Xq, sx, stream=st),
                 lambda st: q.qgemm_w8a8_int8(Xq, sx, Xq, sx, Y=T4, workspace=ws, stream=st)):
        T4 = Tensor(world, (4, 4), torch.bfloat16)
        n += 1
        for st in (Stream(SIDE), SIDE):
            call(st)
            assert world.calls[-1][2][-1] == SIDE
    assert len(world.made) == n


def test_tuners_buffers_belong_to_their_stream(world, monkeypatch):
    q = world.q
    monkeypatch.setattr(q, "workspace_bytes_max", lambda N: 4096)
    monkeypatch.setattr(q, "workspace_bytes_max_w8a8", lambda M, N: 4096)
    X, W = Tensor(world, (4, 256), torch.bfloat16), Tensor(world, (128, 256), torch.bfloat16)
    n = len(world.made)
    q.tune_bf16(X, [W], stream=SIDE)
    _check_side(world, n, "qg_tune_bf16")
