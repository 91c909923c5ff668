"""Python binding of libqgemm (weight-only quantized decode GEMMs for GB300).

Argument marshalling only: every step of the GEMM runs in the library's CUDA
kernels.  PyTorch provides device memory and the current stream.  If the
compiled library is missing this module raises on import; there is no
fallback implementation.

The names follow the C ABI in ``include/qgemm.h``:

* :func:`qgemm_fp8_block` -- W8A16 FP8 E4M3 weights with [128 x 128] FP32
  block scales, BF16 activations and output, two-level FP32 fold.
* :func:`qgemm_fp8_block_multi` -- several of those GEMMs sharing X (e.g. the
  Q, K and V projections) in one launch, each with its own output.
* :func:`qgemm_fp8_block_host` -- the same GEMM with X and Y in pinned host
  memory (staged in and stored out by the library's kernels).
* :func:`qgemm_lut3` -- 3-bit learned-LUT weights (see :func:`pack_lut3`),
  FP16 activations and output.
* :func:`qgemm_bf16` -- unquantised BF16 weights (e.g. an lm_head), BF16
  activations and output.
* :func:`quantize_act_e4m3` / :func:`qgemm_w8a8_block` -- the W8A8 path for
  larger batches: BF16 activations quantised to E4M3 per (row, 128-wide K
  block) with FP32 scales, then an E4M3 x E4M3 block-scaled GEMM
  (:func:`qgemm_w8a8` runs both).
* :func:`quantize_act_int8` / :func:`qgemm_w8a8_int8` -- 8-bit integer
  activations (one scale per token) and weights (one scale per channel), BF16,
  FP16 or FP32 output, optional bias.
* :func:`logprobs` -- over rows of logits: log probabilities of given tokens,
  entropy and the top alternatives.
* :func:`verify_drafts` -- drafted tokens against the target's probabilities:
  how many are kept, and the token that follows.
* :func:`moe_route`, :func:`quantize_rows_e4m3`, :func:`qgemm_w8a8_grouped`,
  :func:`moe_combine` -- layers of experts: router and order by expert, E4M3
  activations on the experts' rows (or of silu(gate) * up), the W8A8 GEMM grouped
  by expert, and the weighted sum back to the tokens.
* :func:`pack_lut3` / :func:`unpack_lut3` -- offline nibble packer (host).
* :func:`debug_fp8_split` / :func:`dequant_lut3` -- test aids: the FP8
  kernel's activation split and the LUT3 kernel's dequantiser on their own,
  exposed for value-by-value checks.

A call with ``stream=`` (a torch stream or a raw handle) is the call made under
``torch.cuda.stream(stream)``: its kernels run there, and the tensors that it
allocates belong to that stream.
"""
from __future__ import annotations

import ctypes
import os
from typing import Any, NamedTuple

import numpy as np

__all__ = [
    "QgemmError", "LIB_PATH", "lib", "status_string", "workspace_bytes", "Workspace",
    "qgemm_fp8_block", "qgemm_fp8_block_multi", "qgemm_fp8_block_host", "Fp8Segment", "MAX_SEGMENTS", "qgemm_lut3", "pack_lut3", "unpack_lut3", "lut3_packed_bytes",
    "debug_fp8_split", "dequant_lut3", "last_device_status", "set_wait_timeout_ns",
    "set_fault_injection", "set_weight_prefetch_overlap", "dispatch_set", "dispatch_get", "dispatch_rule", "dispatch_clear",
    "debug_schedule", "tune_fp8", "tune_lut3", "workspace_bytes_max", "qgemm_bf16", "KIND_BF16", "KIND_FP8_BLOCK", "KIND_LUT3", "STATUS",
    "quantize_act_e4m3", "qgemm_w8a8_block", "qgemm_w8a8", "KIND_W8A8", "MAX_M_W8A8",
    "tune_bf16", "tune_w8a8", "workspace_bytes_max_w8a8",
    "quantize_act_int8", "qgemm_w8a8_int8", "int8_tile_rows", "KIND_INT8", "logprobs", "LogProbs", "MAX_TOP_K",
    "moe_route", "MoeRoute", "quantize_rows_e4m3", "qgemm_w8a8_grouped", "grouped_tile_rows", "moe_combine", "MAX_EXPERTS",
    "verify_drafts", "DraftCheck", "MAX_DRAFTS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqgemm.so")

KIND_FP8_BLOCK = 0
KIND_LUT3 = 1
KIND_BF16 = 2
KIND_W8A8 = 3
KIND_INT8 = 4
MAX_M_W8A8 = 65536
STATUS = {
    0: "QG_OK", 1: "QG_ERR_INVALID_ARG", 2: "QG_ERR_UNSUPPORTED_SHAPE", 3: "QG_ERR_MISALIGNED",
    4: "QG_ERR_CUDA", 5: "QG_ERR_TIMEOUT", 6: "QG_ERR_WORKSPACE",
}


class QgemmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)} ({status_string(code)})")


if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libqgemm.so not found at {LIB_PATH}; build it first with "
        "`python -c 'import __graft_entry__ as g; g.build()'` from the repository root (needs nvcc)")

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_S = ctypes.c_size_t

lib = ctypes.CDLL(LIB_PATH)
_SIGS = {
    "qg_workspace_bytes": (_S, [_I, _I, _I, _I]),
    "qgemm_fp8_block": (_I, [_P, _L, _P, _P, _P, _L, _I, _I, _I, _P, _S, _P]),
    "qgemm_fp8_block_multi": (_I, [_P, _L, _P, _I, _I, _I, _P, _S, _P]),
    "qgemm_fp8_block_host": (_I, [_P, _L, _P, _P, _P, _L, _I, _I, _I, _P, _P, _S, _P]),
    "qgemm_lut3": (_I, [_P, _L, _P, _P, _P, _P, _L, _I, _I, _I, _P, _S, _P]),
    "qgemm_bf16": (_I, [_P, _L, _P, _P, _L, _I, _I, _I, _P, _S, _P]),
    "qg_quantize_act_e4m3": (_I, [_P, _L, _P, _L, _P, _L, _I, _I, _P]),
    "qgemm_w8a8_block": (_I, [_P, _L, _P, _L, _P, _P, _P, _L, _I, _I, _I, _P, _S, _P]),
    "qg_quantize_act_int8": (_I, [_P, _I, _L, _P, _L, _P, _I, _I, _P]),
    "qgemm_w8a8_int8": (_I, [_P, _L, _P, _P, _P, _P, _P, _I, _L, _I, _I, _I, _P, _S, _P]),
    "qg_logprobs": (_I, [_P, _I, _L, _P, _L, _I, _P, _P, _I, _P, _P, _I, _I, _P]),
    "qg_moe_route_workspace_bytes": (_S, [_I, _I]),
    "qg_moe_route": (_I, [_P, _I, _L, _P, _I, _I, ctypes.c_float, _I, _P, _P, _P, _P, _I, _I, _P, _S, _P]),
    "qg_quantize_rows_e4m3": (_I, [_P, _I, _L, _I, _P, _I, _P, _P, _L, _P, _L, _I, _I, _I, _P]),
    "qgemm_w8a8_grouped": (_I, [_P, _L, _P, _L, _P, _P, _P, _P, _I, _L, _I, _I, _I, _I, _P]),
    "qg_moe_combine": (_I, [_P, _I, _L, _P, _P, _I, _P, _L, _P, _L, _I, _I, _I, _P]),
    "qg_verify_drafts_workspace_bytes": (_S, [_I, _I, _I]),
    "qg_verify_drafts": (_I, [_P, _I, _L, _L, _P, _L, _L, _P, _L, _P, _L, _P, _L, _P, _P, _P, _I, _I, _I, _P, _S, _P]),
    "qg_lut3_packed_bytes": (_S, [_I, _I]),
    "pack_lut3": (_I, [_P, _P, _I, _I]),
    "unpack_lut3": (_I, [_P, _P, _I, _I]),
    "qg_debug_fp8_split": (_I, [_P, _L, _P, _P, _P, _P]),
    "qg_debug_schedule": (_I, [_I, _I, _I, _I, _P, _P, _P, _I, _P]),
    "qg_dispatch_set": (_I, [_I, _I, _I, _I, _I]),
    "qg_dispatch_get": (_I, [_I, _I, _I, _I]),
    "qg_dispatch_rule": (_I, [_I, _I, _I, _I, _I]),
    "qg_dispatch_clear": (None, []),
    "qg_int8_tile_rows": (_I, [_I, _I, _I, _I]),
    "qg_grouped_tile_rows": (_I, [_I, _I, _I, _I, _I]),
    "qg_workspace_bytes_max": (_S, [_I]),
    "qg_workspace_bytes_max_w8a8": (_S, [_I, _I]),
    "qg_tune_bf16": (_I, [_P, _L, _P, _I, _P, _L, _P, _I, _I, _I, _P, _S, _I, _P, _P, _P]),
    "qg_tune_w8a8": (_I, [_P, _L, _P, _L, _P, _I, _P, _P, _L, _P, _I, _I, _I, _P, _S, _I, _P, _P, _P]),
    "qg_tune_fp8": (_I, [_P, _L, _P, _I, _P, _P, _L, _P, _I, _I, _I, _P, _S, _I, _P, _P, _P]),
    "qg_tune_lut3": (_I, [_P, _L, _P, _I, _P, _P, _P, _L, _P, _I, _I, _I, _P, _S, _I, _P, _P, _P]),
    "qg_dequant_lut3": (_I, [_P, _P, _P, _P, _I, _I, _P]),
    "qg_last_device_status": (_I, [_P]),
    "qg_set_wait_timeout_ns": (None, [ctypes.c_uint64]),
    "qg_set_fault_injection": (None, [_I]),
    "qg_set_weight_prefetch_overlap": (None, [_I]),
    "qg_status_string": (ctypes.c_char_p, [_I]),
    "qg_version": (ctypes.c_char_p, []),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def status_string(code: int) -> str:
    return lib.qg_status_string(int(code)).decode()


def _check(code: int, where: str) -> None:
    if code != 0:
        raise QgemmError(code, where)


_dtype_codes = {}
_raw_stream = None       # the current stream of a device, as a raw handle
_current_device = None


def _torch():
    """torch, with what the entry points look up on every call."""
    global _raw_stream, _current_device
    import torch
    if _raw_stream is None:
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        # without building a stream object (0.1 us instead of 3 us a call)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: int(torch.cuda.current_stream(index).cuda_stream))
        _dtype_codes.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})   # QG_BF16, QG_FP16, QG_FP32
    return torch


def _stream_ptr(stream) -> int:
    if stream is None:
        _torch()
        return _raw_stream(_current_device())
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _elsewhere(stream) -> bool:
    """True when `stream` is not the current stream of the current device."""
    return _stream_ptr(stream) != _stream_ptr(None) or \
        getattr(stream, "device_index", None) not in (None, _current_device())


def _on_stream(stream, call, *args):
    """call(*args) with `stream` (a torch stream or a raw handle) as the current
    one, so that whatever the call allocates, copies or fills belongs to the
    stream that its kernels run on.  (Made on the caller's stream, a copy would
    not be ordered with the kernel, and memory of the caller's pool may still be
    in use by work queued there.)  It costs the host 9 us, so that calls with
    nothing to make, all outputs given, hand the stream on instead."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_ptr(stream)
        # 0 and 1 are the legacy default stream
        stream = torch.cuda.default_stream() if handle <= 1 else torch.cuda.ExternalStream(handle)
    with torch.cuda.stream(stream):
        return call(*args)


def workspace_bytes(kind: int, M: int, N: int, K: int) -> int:
    """Device workspace a call needs on the current device (may be 0)."""
    return int(lib.qg_workspace_bytes(kind, M, N, K))


# the kinds whose workspaces share a layout: each of these alone, all others together
_SCRATCH = "scratch"   # of calls that keep no counters
_OWN_LAYOUT = (KIND_W8A8, KIND_INT8, _SCRATCH)


class Workspace:
    """Zero-filled device byte buffers that grow on demand, one for each
    workspace layout (the W8A8 and INT8 kinds and calls with scratch memory alone
    have their own, the others share one).  Calls leave their arrival counters at zero again (the rest is
    scratch), so one Workspace serves any sequence of calls of any kind on one
    stream (calls that may run at the same time, on different streams, need one
    each).  Growing synchronises the device, so that the zero fill has landed
    before any stream uses the new buffer.  The buffers that it outgrows are
    kept: captured graphs hold their addresses.  (Each is at least twice the one
    before, so that they add up to less than the newest.)

    ``buf`` is the buffer that was asked for last."""

    def __init__(self, device=None):
        self.device = device
        self.buf = None
        self._bufs = {}   # by layout: the buffers so far, the newest last

    def get(self, nbytes: int, kind: int = KIND_FP8_BLOCK):
        """The buffer of the kind's layout, of at least nbytes (None for 0)."""
        torch = _torch()
        if nbytes == 0:
            return None
        layout = kind if kind in _OWN_LAYOUT else None
        bufs = self._bufs.setdefault(layout, [])
        if not bufs or bufs[-1].numel() < nbytes:
            dev = self.device or torch.cuda.current_device()
            least = 2 * bufs[-1].numel() if bufs else 1 << 20
            bufs.append(torch.zeros(max(nbytes, least), dtype=torch.uint8, device=dev))
            torch.cuda.synchronize(dev)
        self.buf = bufs[-1]
        return self.buf

    def reset(self):
        for bufs in self._bufs.values():
            for buf in bufs:
                buf.zero_()


_default_ws = {}


_ws_need = {}


def _workspace_for(kind, M, N, K, workspace, device, stream=None):
    key = (kind, M, N, K, device)
    need = _ws_need.get(key)
    if need is None:
        need = _ws_need[key] = workspace_bytes(kind, M, N, K)
    if need == 0:
        return None, 0
    if workspace is None:
        # a default one per device and stream (calls on different streams may overlap)
        key = (device, _stream_ptr(stream))
        workspace = _default_ws.get(key)
        if workspace is None:
            workspace = _default_ws[key] = Workspace(device)
    buf = workspace.get(need, kind) if isinstance(workspace, Workspace) else workspace
    return buf.data_ptr(), buf.numel() * buf.element_size()


def _ld(t) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit stride in its last dimension")
    return t.stride(0)


def qgemm_fp8_block(X, W, W_scale, Y=None, workspace=None, stream=None):
    """Y[M, N] = X[M, K] . dequant(W)[N, K]^T (BF16 out).

    X: bf16 CUDA [M, K] (row stride a multiple of 8); W: uint8 (E4M3 codes) or
    float8_e4m3fn [N, K] contiguous; W_scale: float32 [ceil(N/128), ceil(K/128)]
    contiguous.  Y (optional): bf16 [M, N] with unit column stride.
    """
    if stream is not None and Y is None and _elsewhere(stream):
        return _on_stream(stream, qgemm_fp8_block, X, W, W_scale, Y, workspace)
    torch = _torch()
    if X.dtype != torch.bfloat16:
        raise TypeError("X must be bfloat16")
    if W.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError("W must hold E4M3 codes (uint8 or float8_e4m3fn)")
    if W_scale.dtype != torch.float32 or not W_scale.is_contiguous() or not W.is_contiguous():
        raise TypeError("W must be contiguous and W_scale contiguous float32")
    M, K = X.shape
    N = W.shape[0]
    if W.shape[1] != K or tuple(W_scale.shape) != (-(-N // 128), -(-K // 128)):
        raise ValueError("shape mismatch between X, W and W_scale")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    ws, wsb = _workspace_for(KIND_FP8_BLOCK, M, N, K, workspace, X.device, stream)
    _check(lib.qgemm_fp8_block(X.data_ptr(), _ld(X), W.data_ptr(), W_scale.data_ptr(), Y.data_ptr(),
                               _ld(Y), M, N, K, ws, wsb, _stream_ptr(stream)), "qgemm_fp8_block")
    return Y


MAX_SEGMENTS = 4


class Fp8Segment(ctypes.Structure):
    """qg_fp8_segment of include/qgemm.h."""
    _fields_ = [("W", ctypes.c_void_p), ("W_scale", ctypes.c_void_p), ("Y", ctypes.c_void_p),
                ("ldy", ctypes.c_int64), ("N", ctypes.c_int)]


def qgemm_fp8_block_multi(X, weights, Ys=None, workspace=None, stream=None):
    """Y_j = X . dequant(W_j)^T for every (W_j, W_scale_j) in `weights`
    (1 to MAX_SEGMENTS of them, sharing X), in one launch; returns the list of
    Y_j (BF16 [M, N_j]).  Ys (optional): the output tensors, each with unit
    column stride."""
    if stream is not None and Ys is None and _elsewhere(stream):
        return _on_stream(stream, qgemm_fp8_block_multi, X, weights, Ys, workspace)
    torch = _torch()
    if X.dtype != torch.bfloat16:
        raise TypeError("X must be bfloat16")
    if not 1 <= len(weights) <= MAX_SEGMENTS:
        raise ValueError(f"between 1 and {MAX_SEGMENTS} weight matrices")
    M, K = X.shape
    segs = (Fp8Segment * len(weights))()
    outs = []
    rows = 0
    for j, (W, S) in enumerate(weights):
        if W.dtype not in (torch.uint8, torch.float8_e4m3fn) or not W.is_contiguous():
            raise TypeError("W must hold contiguous E4M3 codes (uint8 or float8_e4m3fn)")
        N = W.shape[0]
        if W.shape[1] != K or tuple(S.shape) != (-(-N // 128), -(-K // 128)) or S.dtype != torch.float32 \
                or not S.is_contiguous():
            raise ValueError(f"segment {j}: shape mismatch between X, W and W_scale")
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device) if Ys is None else Ys[j]
        outs.append(Y)
        segs[j] = Fp8Segment(W.data_ptr(), S.data_ptr(), Y.data_ptr(), _ld(Y), N)
        rows += -(-N // 128) * 128
    ws, wsb = _workspace_for(KIND_FP8_BLOCK, M, rows, K, workspace, X.device, stream)
    _check(lib.qgemm_fp8_block_multi(X.data_ptr(), _ld(X), ctypes.cast(segs, ctypes.c_void_p), len(weights), M, K,
                                     ws, wsb, _stream_ptr(stream)), "qgemm_fp8_block_multi")
    return outs


_default_stage = {}


def qgemm_fp8_block_host(X, W, W_scale, Y=None, X_stage=None, workspace=None, stream=None):
    """:func:`qgemm_fp8_block` with X and Y in pinned host memory.

    X: bf16 CPU [M, K], pinned (``tensor.pin_memory()``), row stride a
    multiple of 8; Y (optional, allocated pinned if absent): bf16 CPU [M, N],
    pinned, unit column stride.  W and W_scale are on the device as for
    :func:`qgemm_fp8_block`.  X_stage (optional): a device buffer of at least
    M*K bf16 elements that the call copies X into; a per-device buffer is
    kept when absent.  The call is asynchronous: Y is complete after the
    stream is synchronised.
    """
    if stream is not None and (Y is None or X_stage is None) and _elsewhere(stream):
        return _on_stream(stream, qgemm_fp8_block_host, X, W, W_scale, Y, X_stage, workspace)
    torch = _torch()
    if X.dtype != torch.bfloat16:
        raise TypeError("X must be bfloat16")
    if W.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError("W must hold E4M3 codes (uint8 or float8_e4m3fn)")
    if W_scale.dtype != torch.float32 or not W_scale.is_contiguous() or not W.is_contiguous():
        raise TypeError("W must be contiguous and W_scale contiguous float32")
    if X.is_cuda or not X.is_pinned():
        raise ValueError("X must be a pinned host tensor")
    M, K = X.shape
    N = W.shape[0]
    if W.shape[1] != K or tuple(W_scale.shape) != (-(-N // 128), -(-K // 128)):
        raise ValueError("shape mismatch between X, W and W_scale")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16).pin_memory()
    elif Y.dtype != torch.bfloat16 or Y.is_cuda or not Y.is_pinned():
        raise ValueError("Y must be a pinned bfloat16 host tensor")
    if X_stage is None:
        X_stage = _default_stage.get(W.device)
        if X_stage is None or X_stage.numel() < M * K:
            X_stage = _default_stage[W.device] = torch.empty(max(M * K, 1 << 16), dtype=torch.bfloat16,
                                                             device=W.device)
    elif not X_stage.is_cuda or X_stage.numel() * X_stage.element_size() < M * K * 2:
        raise ValueError("X_stage must be a device buffer of at least M*K bfloat16 elements")
    ws, wsb = _workspace_for(KIND_FP8_BLOCK, M, N, K, workspace, W.device, stream)
    _check(lib.qgemm_fp8_block_host(X.data_ptr(), _ld(X), W.data_ptr(), W_scale.data_ptr(), Y.data_ptr(),
                                    _ld(Y), M, N, K, X_stage.data_ptr(), ws, wsb, _stream_ptr(stream)),
           "qgemm_fp8_block_host")
    return Y


def qgemm_lut3(X, Wq, qmap, scales, N: int, Y=None, workspace=None, stream=None):
    """Y[M, N] = X[M, K] . dequant(Wq)^T with the 3-bit learned-LUT format (FP16 out).

    X: fp16 CUDA [M, K]; Wq: the packed bytes from :func:`pack_lut3` on the
    device; qmap: fp16 [8]; scales: fp16 [N, K/128] contiguous.
    """
    if stream is not None and Y is None and _elsewhere(stream):
        return _on_stream(stream, qgemm_lut3, X, Wq, qmap, scales, N, Y, workspace)
    torch = _torch()
    if X.dtype != torch.float16 or qmap.dtype != torch.float16 or scales.dtype != torch.float16:
        raise TypeError("X, qmap and scales must be float16")
    M, K = X.shape
    if tuple(scales.shape) != (N, K // 128) or not scales.is_contiguous():
        raise ValueError("scales must be a contiguous [N, K/128] tensor")
    if Wq.numel() * Wq.element_size() < lut3_packed_bytes(N, K):
        raise ValueError("packed weights are smaller than pack_lut3 produces for this shape")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=X.device)
    ws, wsb = _workspace_for(KIND_LUT3, M, N, K, workspace, X.device, stream)
    _check(lib.qgemm_lut3(X.data_ptr(), _ld(X), Wq.data_ptr(), qmap.data_ptr(), scales.data_ptr(),
                          Y.data_ptr(), _ld(Y), M, N, K, ws, wsb, _stream_ptr(stream)), "qgemm_lut3")
    return Y


def quantize_act_e4m3(X, Xq=None, X_scale=None, stream=None):
    """E4M3 codes and FP32 scales of BF16 activations, per (row, 128-wide K
    block): scale = block max |x| / 448 (1 for a zero block), code =
    e4m3_rne_satfinite(x / scale).

    X: bf16 CUDA [M, K] (row stride a multiple of 8, K % 16 == 0).  Returns
    (Xq uint8 [M, K] (a view with row stride rounded up to 16), X_scale
    float32 [ceil(K/128), ldsx] with ldsx = M rounded up to 32; columns
    [M, ldsx) are 0).  Xq and X_scale (optional) are written in place.
    """
    if stream is not None and (Xq is None or X_scale is None) and _elsewhere(stream):
        return _on_stream(stream, quantize_act_e4m3, X, Xq, X_scale)
    torch = _torch()
    if X.dtype != torch.bfloat16:
        raise TypeError("X must be bfloat16")
    M, K = X.shape
    KB = -(-K // 128)
    if Xq is None:
        Xq = torch.empty((M, -(-K // 16) * 16), dtype=torch.uint8, device=X.device)[:, :K]
    if X_scale is None:
        X_scale = torch.empty((KB, max(32, -(-M // 32) * 32)), dtype=torch.float32, device=X.device)
    if Xq.dtype not in (torch.uint8, torch.float8_e4m3fn) or X_scale.dtype != torch.float32:
        raise TypeError("Xq must be uint8 or float8_e4m3fn, X_scale float32")
    if tuple(Xq.shape) != (M, K) or X_scale.shape[0] != KB:
        raise ValueError("shape mismatch between X, Xq and X_scale")
    _check(lib.qg_quantize_act_e4m3(X.data_ptr(), _ld(X), Xq.data_ptr(), _ld(Xq), X_scale.data_ptr(),
                                    _ld(X_scale), M, K, _stream_ptr(stream)), "qg_quantize_act_e4m3")
    return Xq, X_scale


def qgemm_w8a8_block(Xq, X_scale, W, W_scale, Y=None, workspace=None, stream=None):
    """Y[M, N] = sum over 128-wide K blocks kb of X_scale[kb, m] *
    W_scale[n/128, kb] * (Xq[m, kb] . W[n, kb]) (E4M3 x E4M3, FP32 fold, BF16
    out), with Xq, X_scale as :func:`quantize_act_e4m3` returns them."""
    if stream is not None and Y is None and _elsewhere(stream):
        return _on_stream(stream, qgemm_w8a8_block, Xq, X_scale, W, W_scale, Y, workspace)
    torch = _torch()
    if Xq.dtype not in (torch.uint8, torch.float8_e4m3fn) or W.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError("Xq and W must hold E4M3 codes (uint8 or float8_e4m3fn)")
    if X_scale.dtype != torch.float32 or W_scale.dtype != torch.float32:
        raise TypeError("X_scale and W_scale must be float32")
    if not W.is_contiguous() or not W_scale.is_contiguous():
        raise TypeError("W and W_scale must be contiguous")
    M, K = Xq.shape
    N = W.shape[0]
    if W.shape[1] != K or tuple(W_scale.shape) != (-(-N // 128), -(-K // 128)) or X_scale.shape[0] != -(-K // 128):
        raise ValueError("shape mismatch between Xq, X_scale, W and W_scale")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=Xq.device)
    ws, wsb = _workspace_for(KIND_W8A8, M, N, K, workspace, Xq.device, stream)
    _check(lib.qgemm_w8a8_block(Xq.data_ptr(), _ld(Xq), X_scale.data_ptr(), _ld(X_scale), W.data_ptr(),
                                W_scale.data_ptr(), Y.data_ptr(), _ld(Y), M, N, K, ws, wsb, _stream_ptr(stream)),
           "qgemm_w8a8_block")
    return Y


def qgemm_w8a8(X, W, W_scale, Y=None, workspace=None, stream=None):
    """The W8A8 path from BF16 activations: :func:`quantize_act_e4m3` then
    :func:`qgemm_w8a8_block` (two launches on one stream)."""
    if stream is not None and _elsewhere(stream):
        return _on_stream(stream, qgemm_w8a8, X, W, W_scale, Y, workspace)
    Xq, X_scale = quantize_act_e4m3(X)
    return qgemm_w8a8_block(Xq, X_scale, W, W_scale, Y=Y, workspace=workspace)


def _rows(t, what: str):
    """(rows, columns, row stride) of a 2-D CUDA tensor with unit column
    stride; a lone row's stride is arbitrary and counts as its length."""
    if t.dim() != 2:
        raise ValueError(what + " must be a 2-D tensor")
    r, c = t.shape
    ld, step = t.stride()
    if step != 1 and c > 1:
        raise ValueError(what + " must have unit stride in its last dimension")
    if not t.is_cuda:
        raise ValueError(what + " must be on a CUDA device")
    return r, c, (ld if r > 1 else c)


_SIZE = "sizes of 2^31 and more are not supported"   # which ctypes would cut to 32 bits


def quantize_act_int8(X, Xq=None, X_scale=None, stream=None):
    """8-bit integer codes and one FP32 scale per row of BF16 or FP16
    activations: scale = max |x| / 127, code = x * (127 * (1 / max |x|)) rounded
    half to even (a row whose largest |x| is below 2^-100 has codes 0, scale 1;
    one with a NaN or an infinity has scale NaN).

    X: CUDA [M, K] (row stride a multiple of 8, K % 16 == 0).  Returns (Xq
    int8 [M, K], X_scale float32 [M]).  Xq and X_scale (optional) are written
    in place.
    """
    if stream is not None and (Xq is None or X_scale is None) and _elsewhere(stream):
        return _on_stream(stream, quantize_act_int8, X, Xq, X_scale)
    torch = _torch()
    code = _dtype_codes.get(X.dtype)
    if code != 0 and code != 1:
        raise TypeError("X must be bfloat16 or float16")
    M, K, ld = _rows(X, "X")
    if (M | K) >> 31:
        raise ValueError(_SIZE)
    dev = X.device
    index = dev.index
    if index != _current_device():   # where the library launches
        raise ValueError("the tensors must be on the current CUDA device")
    if Xq is None:
        Xq = torch.empty((M, K), dtype=torch.int8, device=dev)
        ldq = K
    else:
        if Xq.dtype != torch.int8:
            raise TypeError("Xq must be int8")
        rows, cols, ldq = _rows(Xq, "Xq")
        if rows != M or cols != K or Xq.device != dev:
            raise ValueError("Xq must be [M, K] on X's device")
    if X_scale is None:
        X_scale = torch.empty((M,), dtype=torch.float32, device=dev)
    else:
        if X_scale.dtype != torch.float32 or not X_scale.is_contiguous():
            raise TypeError("X_scale must be contiguous float32")
        if X_scale.shape != (M,) or X_scale.device != dev:
            raise ValueError("X_scale must be [M] on X's device")
    if K == 0:   # rows of nothing, which the library leaves alone
        if stream is not None and _elsewhere(stream):
            return _on_stream(stream, quantize_act_int8, X, Xq, X_scale)
        return Xq, X_scale.fill_(1.0)
    st = _raw_stream(index) if stream is None else _stream_ptr(stream)
    r = lib.qg_quantize_act_int8(X.data_ptr(), code, ld, Xq.data_ptr(), ldq, X_scale.data_ptr(), M, K, st)
    if r:
        raise QgemmError(r, "qg_quantize_act_int8")
    return Xq, X_scale


def qgemm_w8a8_int8(Xq, X_scale, W, W_scale, bias=None, out_dtype=None, Y=None, workspace=None, stream=None):
    """Y[m, n] = X_scale[m] * W_scale[n] * (Xq[m] . W[n]) (+ bias[n]): 8-bit
    integer activations with one scale per token, 8-bit integer weights with
    one scale per channel.

    Xq: int8 CUDA [M, K] (row stride a multiple of 16), X_scale: float32 [M] as
    :func:`quantize_act_int8` returns them; W: int8 [N, K] contiguous; W_scale:
    float32 [N]; bias (optional): float32 [N].  Y (optional): [M, N] with unit
    column stride, in bfloat16 (the default), float16 or float32 (out_dtype).

    The products are summed in FP32: exactly while every partial sum stays below
    2^24 in magnitude (always for K <= 1024, with codes of mixed signs far
    longer), beyond that with up to 2^-23 of the sum lost, towards zero, every 16
    products (see include/qgemm.h).
    """
    if stream is not None and Y is None and _elsewhere(stream):
        return _on_stream(stream, qgemm_w8a8_int8, Xq, X_scale, W, W_scale, bias, out_dtype, Y, workspace)
    torch = _torch()
    i8, f32 = torch.int8, torch.float32
    if Xq.dtype != i8 or W.dtype != i8:
        raise TypeError("Xq and W must be int8")
    if X_scale.dtype != f32 or W_scale.dtype != f32:
        raise TypeError("X_scale and W_scale must be float32")
    if not (W.is_contiguous() and X_scale.is_contiguous() and W_scale.is_contiguous()):
        raise TypeError("W and the scales must be contiguous")
    M, K, ldq = _rows(Xq, "Xq")
    N = W.shape[0]
    if (M | N | K) >> 31:
        raise ValueError(_SIZE)
    dev = Xq.device
    index = dev.index
    if index != _current_device():   # where the library launches
        raise ValueError("the tensors must be on the current CUDA device")
    if W.shape != (N, K) or X_scale.shape != (M,) or W_scale.shape != (N,):
        raise ValueError("shape mismatch between Xq, X_scale, W and W_scale")
    if W.device != dev or X_scale.device != dev or W_scale.device != dev:
        raise ValueError("all tensors must be on one CUDA device")
    b = None
    if bias is not None:
        if bias.dtype != f32 or not bias.is_contiguous():
            raise TypeError("bias must be contiguous float32")
        if bias.shape != (N,) or bias.device != dev:
            raise ValueError("bias must be [N] on the same device")
        b = bias.data_ptr()
    if Y is None:
        if out_dtype is None:
            out_dtype = torch.bfloat16
        code = _dtype_codes.get(out_dtype)
        if code is None:
            raise TypeError("the output must be bfloat16, float16 or float32")
        Y = torch.empty((M, N), dtype=out_dtype, device=dev)
        ldy = N
    else:
        code = _dtype_codes.get(Y.dtype)
        if code is None or (out_dtype is not None and Y.dtype != out_dtype):
            raise TypeError("Y must be bfloat16, float16 or float32, as out_dtype says")
        rows, cols, ldy = _rows(Y, "Y")
        if rows != M or cols != N or Y.device != dev:
            raise ValueError("Y must be [M, N] on the same device")
    st = _raw_stream(index) if stream is None else _stream_ptr(stream)
    ws, wsb = _workspace_for(KIND_INT8, M, N, K, workspace, dev, st)
    r = lib.qgemm_w8a8_int8(Xq.data_ptr(), ldq, X_scale.data_ptr(), W.data_ptr(), W_scale.data_ptr(), b,
                            Y.data_ptr(), code, ldy, M, N, K, ws, wsb, st)
    if r:
        raise QgemmError(r, "qgemm_w8a8_int8")
    return Y


def int8_tile_rows(M: int, N: int, K: int, sms: int) -> int:
    """The tokens of a tile that the schedule rule of :func:`qgemm_w8a8_int8`
    picks for this shape on a device with `sms` SMs (host only; 0 for invalid
    arguments)."""
    return int(lib.qg_int8_tile_rows(M, N, K, sms))


MAX_TOP_K = 32


class LogProbs(NamedTuple):
    """What :func:`logprobs` returns; a part not asked for is None."""
    token_logprobs: Any   # float32, shaped like tokens
    entropy: Any          # float32 [M], nats
    top_ids: Any          # int64 [M, top_k]
    top_logprobs: Any     # float32 [M, top_k]


def logprobs(logits, tokens=None, top_k: int = 0, entropy: bool = False, stream=None) -> LogProbs:
    """Over the softmax of every row of logits: the log probabilities of given
    tokens, the entropy, and the top alternatives (by value, then by lower
    index).

    logits: bf16, fp16 or fp32 CUDA [M, V] with unit column stride; tokens
    (optional): int64 [M] or [M, T]; top_k: 0 .. MAX_TOP_K and <= V.  A logit
    of -inf is a masked token; a row with nothing left has log probabilities
    of -inf and entropy 0; a token outside the vocabulary has -inf; a row with
    a NaN or +inf gives NaN (see include/qgemm.h).
    """
    if stream is not None and _elsewhere(stream):
        return _on_stream(stream, logprobs, logits, tokens, top_k, entropy)
    torch = _torch()
    f32, i64 = torch.float32, torch.int64
    code = _dtype_codes.get(logits.dtype)
    if code is None:
        raise TypeError("logits must be bfloat16, float16 or float32")
    M, V, ld = _rows(logits, "logits")
    if (M | V) >> 31:
        raise ValueError(_SIZE)
    dev = logits.device
    index = dev.index
    if index != _current_device():   # where the library launches
        raise ValueError("the tensors must be on the current CUDA device")
    T = ldt = 0
    tok = token_lp = token_p = ent = ent_p = ids = ids_p = top = top_p = None
    if tokens is not None:
        if tokens.dtype != i64:
            raise TypeError("tokens must be int64")
        if tokens.device != dev:
            raise ValueError("logits and tokens must be on one CUDA device")
        shape = tokens.shape
        if len(shape) not in (1, 2) or shape[0] != M:
            raise ValueError("tokens must be [M] or [M, T]")
        T = shape[1] if len(shape) == 2 else 1
        if T >> 31:
            raise ValueError(_SIZE)
        strides = tokens.stride()
        ldt = strides[0] if M > 1 else T
        if ldt < T or (T > 1 and strides[1] != 1):   # expanded or transposed
            tokens = tokens.contiguous()
            ldt = T
        tok = tokens.data_ptr()
        token_lp = torch.empty(shape, dtype=f32, device=dev)
        token_p = token_lp.data_ptr()
    if entropy:
        ent = torch.empty((M,), dtype=f32, device=dev)
        ent_p = ent.data_ptr()
    if top_k > 0:   # a negative one is refused by the library
        if top_k >> 31:
            raise ValueError(_SIZE)
        ids = torch.empty((M, top_k), dtype=i64, device=dev)
        top = torch.empty((M, top_k), dtype=f32, device=dev)
        ids_p, top_p = ids.data_ptr(), top.data_ptr()
    st = _raw_stream(index)
    r = lib.qg_logprobs(logits.data_ptr(), code, ld, tok, ldt, T, token_p, ent_p, top_k, ids_p, top_p, M, V, st)
    if r:
        raise QgemmError(r, "qg_logprobs")
    return LogProbs(token_lp, ent, ids, top)


MAX_EXPERTS = 1024
_SCORES = {"softmax": 0, "sigmoid": 1}


class MoeRoute(NamedTuple):
    """What :func:`moe_route` returns."""
    experts: Any   # int32 [M, top_k]
    weights: Any   # float32 [M, top_k]
    offsets: Any   # int32 [E + 1]
    rows: Any      # int32 [M, top_k]


_scratch_need = {}   # of the sizes seen lately
_MOST_NEEDS = 1024   # prompts have many lengths: then it starts anew


def _scratch(key, ask, workspace, device):
    """(tensor to keep until the call is made, address, bytes) of the scratch memory
    of a call, whose need `ask` says (kept by key).  Nothing is expected in it, so
    that without a workspace every call has some of its own, from PyTorch's
    allocator: calls of other streams and captured graphs share none."""
    need = _scratch_need.get(key)
    if need is None:
        if len(_scratch_need) >= _MOST_NEEDS:
            _scratch_need.clear()
        need = _scratch_need[key] = int(ask())
    if need == 0:
        return None, None, 0
    if workspace is None:
        torch = _torch()
        buf = torch.empty((need,), dtype=torch.uint8, device=device)
    else:
        buf = workspace.get(need, _SCRATCH) if isinstance(workspace, Workspace) else workspace
        if buf.device != device or not buf.is_contiguous():
            raise ValueError("the workspace must be contiguous, on the tensors' device")
    return buf, buf.data_ptr(), buf.numel() * buf.element_size()


def _vector(t, dtype, n, dev, what: str):
    """The address of a contiguous tensor of n elements."""
    if t.dtype != dtype or not t.is_contiguous():
        raise TypeError(what + " must be contiguous " + str(dtype).replace("torch.", ""))
    if t.numel() != n or t.device != dev:
        raise ValueError(f"{what} must have {n} elements on the same device")
    return t.data_ptr()


def moe_route(logits, top_k: int, score: str = "softmax", bias=None, renormalize: bool = True, scale: float = 1.0,
              workspace=None, stream=None) -> MoeRoute:
    """Router of a layer of experts: for every token (row of logits [M, E], bf16,
    fp16 or fp32) the top_k experts by score, their weights, and the order of all
    choices by expert.

    score: "softmax" or "sigmoid" of the logits; bias (optional, float32 [E]) is
    added for the choice alone.  Ties go to the lower index; -inf masks an expert.
    weights: the scores over their sum (renormalize) times scale.  Expert e's rows
    are offsets[e] .. offsets[e + 1] - 1, in the order of the tokens; rows[m, j] is
    the row of token m's j-th choice.  Where fewer than top_k experts are left,
    experts and rows are -1 and the weight 0; a token with a NaN or +inf logit is
    routed nowhere, with weights of NaN.  workspace (optional, a :class:`Workspace` or
    uint8 tensor): scratch memory, which calls that may run at the same time must not
    share; without one every call makes its own.
    """
    if stream is not None and _elsewhere(stream):
        return _on_stream(stream, moe_route, logits, top_k, score, bias, renormalize, scale, workspace)
    torch = _torch()
    code = _dtype_codes.get(logits.dtype)
    if code is None:
        raise TypeError("logits must be bfloat16, float16 or float32")
    kind = _SCORES.get(score)
    if kind is None:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    M, E, ld = _rows(logits, "logits")
    if (M | E | top_k) >> 31:
        raise ValueError(_SIZE)
    dev = logits.device
    index = dev.index
    if index != _current_device():   # where the library launches
        raise ValueError("the tensors must be on the current CUDA device")
    b = None if bias is None else _vector(bias, torch.float32, E, dev, "bias")
    i32 = torch.int32
    experts = torch.empty((M, top_k), dtype=i32, device=dev)
    weights = torch.empty((M, top_k), dtype=torch.float32, device=dev)
    offsets = torch.empty((E + 1,), dtype=i32, device=dev)
    rows = torch.empty((M, top_k), dtype=i32, device=dev)
    st = _raw_stream(index)
    buf, ws, wsb = _scratch(("route", M, E, index), lambda: lib.qg_moe_route_workspace_bytes(M, E), workspace, dev)
    r = lib.qg_moe_route(logits.data_ptr(), code, ld, b, kind, 1 if renormalize else 0, scale, top_k,
                         experts.data_ptr(), weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), M, E, ws, wsb, st)
    if r:
        raise QgemmError(r, "qg_moe_route")
    return MoeRoute(experts, weights, offsets, rows)


def quantize_rows_e4m3(X, gated: bool = False, rows=None, num_rows=None, out_rows=None, Xq=None, X_scale=None,
                       stream=None):
    """E4M3 codes and FP32 scales per (row, 128 columns), as
    :func:`quantize_act_e4m3` makes them, of the rows that a layer of experts needs.

    X: bf16 or fp16 CUDA [M, K] (row stride a multiple of 8, K % 16 == 0); gated:
    [M, 2 K], and silu(X[:, :K]) * X[:, K:] is quantised.  rows (optional, int32
    [M, top_k] as :func:`moe_route` returns it): row m goes to rows rows[m, :] of the
    output (-1: nowhere; no place may be named by two rows), of out_rows rows (M * top_k
    when absent).  num_rows
    (optional, int32, one element on the device, e.g. ``route.offsets[-1:]``): only
    the rows before it are read.  Output rows that nothing goes to are left as they
    were.  Returns (Xq uint8 [out_rows, K], X_scale float32 [ceil(K/128), ldsx]) with
    ldsx = out_rows rounded up to 32.  Xq and X_scale (optional: [ceil(K/128), out_rows
    or more], row stride a multiple of 4) are written in place.
    """
    if stream is not None and (Xq is None or X_scale is None) and _elsewhere(stream):
        return _on_stream(stream, quantize_rows_e4m3, X, gated, rows, num_rows, out_rows, Xq, X_scale)
    torch = _torch()
    code = _dtype_codes.get(X.dtype)
    if code != 0 and code != 1:
        raise TypeError("X must be bfloat16 or float16")
    M, K, ld = _rows(X, "X")
    if gated:
        if K % 2:
            raise ValueError("gated: X must have an even number of columns")
        K //= 2
    dev = X.device
    index = dev.index
    if index != _current_device():   # where the library launches
        raise ValueError("the tensors must be on the current CUDA device")
    top_k, at, n = 0, None, None
    if rows is not None:
        if rows.dim() != 2 or rows.shape[0] != M:
            raise ValueError("rows must be [M, top_k]")
        top_k = rows.shape[1]
        at = _vector(rows, torch.int32, M * top_k, dev, "rows")
    if num_rows is not None:
        n = _vector(num_rows, torch.int32, 1, dev, "num_rows")
    if out_rows is None:
        out_rows = Xq.shape[0] if Xq is not None else M if rows is None else M * top_k
    if (M | K | out_rows) >> 31:
        raise ValueError(_SIZE)
    KB = -(-K // 128)
    if Xq is None:
        Xq = torch.empty((out_rows, K), dtype=torch.uint8, device=dev)
        ldq = K
    else:
        if Xq.dtype not in (torch.uint8, torch.float8_e4m3fn):
            raise TypeError("Xq must be uint8 or float8_e4m3fn")
        r, c, ldq = _rows(Xq, "Xq")
        if r != out_rows or c != K or Xq.device != dev:
            raise ValueError("Xq must be [out_rows, K] on X's device")
    if X_scale is None:
        X_scale = torch.empty((KB, max(32, -(-out_rows // 32) * 32)), dtype=torch.float32, device=dev)
        lds = X_scale.shape[1]
    else:
        if X_scale.dtype != torch.float32:
            raise TypeError("X_scale must be float32")
        r, c, lds = _rows(X_scale, "X_scale")
        if r != KB or c < out_rows or X_scale.device != dev:
            raise ValueError("X_scale must be [ceil(K/128), out_rows or more] on X's device")
        if r == 1:   # no row behind it: any stride does
            lds = -(-out_rows // 4) * 4
    if rows is not None and top_k == 0:   # rows that go nowhere
        return Xq, X_scale
    st = _raw_stream(index) if stream is None else _stream_ptr(stream)
    r = lib.qg_quantize_rows_e4m3(X.data_ptr(), code, ld, 1 if gated else 0, at, top_k, n, Xq.data_ptr(), ldq,
                                  X_scale.data_ptr(), lds, M, out_rows, K, st)
    if r:
        raise QgemmError(r, "qg_quantize_rows_e4m3")
    return Xq, X_scale


def qgemm_w8a8_grouped(Xq, X_scale, W, W_scale, offsets, out_dtype=None, Y=None, stream=None):
    """:func:`qgemm_w8a8_block` grouped by expert: for the rows r of each expert e,
    offsets[e] <= r < offsets[e + 1], Y[r] = dequant(Xq[r]) . dequant(W[e])^T with
    FP32 sums per 128-wide K block.

    Xq: uint8 (E4M3 codes) or float8_e4m3fn CUDA [R, K] (row stride a multiple of
    16) and X_scale: float32 [ceil(K/128), R or more] (row stride a multiple of 4) as
    :func:`quantize_rows_e4m3` returns them, or its first R columns; W: uint8 or
    float8_e4m3fn [E, N, K] contiguous; W_scale: float32 [E, ceil(N/128), ceil(K/128)]
    contiguous; offsets: int32 [E + 1] on the device.
    Y (optional): [R, N] with unit column stride, in bfloat16 (the default), float16
    or float32 (out_dtype).  Rows of no expert are left as they were.
    """
    if stream is not None and Y is None and _elsewhere(stream):
        return _on_stream(stream, qgemm_w8a8_grouped, Xq, X_scale, W, W_scale, offsets, out_dtype, Y)
    torch = _torch()
    codes = (torch.uint8, torch.float8_e4m3fn)
    if Xq.dtype not in codes or W.dtype not in codes:
        raise TypeError("Xq and W must hold E4M3 codes (uint8 or float8_e4m3fn)")
    f32 = torch.float32
    if X_scale.dtype != f32 or W_scale.dtype != f32:
        raise TypeError("X_scale and W_scale must be float32")
    if not (W.is_contiguous() and W_scale.is_contiguous()):
        raise TypeError("W and W_scale must be contiguous")
    R, K, ldq = _rows(Xq, "Xq")
    sr, sc, lds = _rows(X_scale, "X_scale")
    if W.dim() != 3:
        raise ValueError("W must be [E, N, K]")
    E, N, WK = W.shape
    if (R | E | N | K) >> 31:
        raise ValueError(_SIZE)
    KB = -(-K // 128)
    if WK != K or sr != KB or sc < R or W_scale.shape != (E, -(-N // 128), KB):
        raise ValueError("shape mismatch between Xq, X_scale, W and W_scale")
    fours = -(-R // 4) * 4   # the scales are read by fours
    if sr == 1:   # no row behind it: any stride does
        lds = fours
    if sc < fours and 0 < sr and \
            X_scale.untyped_storage().nbytes() < 4 * (X_scale.storage_offset() + (sr - 1) * lds + fours):
        raise ValueError("X_scale's memory must reach up to a multiple of 4 columns")
    dev = Xq.device
    index = dev.index
    if index != _current_device():   # where the library launches
        raise ValueError("the tensors must be on the current CUDA device")
    if W.device != dev or X_scale.device != dev or W_scale.device != dev:
        raise ValueError("all tensors must be on one CUDA device")
    off = _vector(offsets, torch.int32, E + 1, dev, "offsets")
    if Y is None:
        if out_dtype is None:
            out_dtype = torch.bfloat16
        code = _dtype_codes.get(out_dtype)
        if code is None:
            raise TypeError("the output must be bfloat16, float16 or float32")
        Y = torch.empty((R, N), dtype=out_dtype, device=dev)
        ldy = N
    else:
        code = _dtype_codes.get(Y.dtype)
        if code is None or (out_dtype is not None and Y.dtype != out_dtype):
            raise TypeError("Y must be bfloat16, float16 or float32, as out_dtype says")
        r, c, ldy = _rows(Y, "Y")
        if r != R or c != N or Y.device != dev:
            raise ValueError("Y must be [R, N] on the same device")
    st = _raw_stream(index) if stream is None else _stream_ptr(stream)
    r = lib.qgemm_w8a8_grouped(Xq.data_ptr(), ldq, X_scale.data_ptr(), lds, W.data_ptr(), W_scale.data_ptr(), off,
                               Y.data_ptr(), code, ldy, R, E, N, K, st)
    if r:
        raise QgemmError(r, "qgemm_w8a8_grouped")
    return Y


def grouped_tile_rows(R: int, E: int, N: int, K: int, sms: int) -> int:
    """The rows of a tile that :func:`qgemm_w8a8_grouped` takes for this shape on a
    device with `sms` SMs (host only; 0 for invalid arguments)."""
    return int(lib.qg_grouped_tile_rows(R, E, N, K, sms))


def moe_combine(Y, rows, weights, residual=None, out=None, stream=None):
    """out[m] = sum over j of weights[m, j] * Y[rows[m, j]] (+ residual[m]) in FP32,
    rounded once: the experts' results back to the tokens.

    Y: bf16, fp16 or fp32 CUDA [R, K]; rows: int32 and weights: float32 [M, top_k] as
    :func:`moe_route` returns them (a row of -1 counts as zeros); residual (optional)
    and out (optional): [M, K] of Y's type, which may be the same tensor, apart from Y.
    """
    if stream is not None and out is None and _elsewhere(stream):
        return _on_stream(stream, moe_combine, Y, rows, weights, residual, out)
    torch = _torch()
    code = _dtype_codes.get(Y.dtype)
    if code is None:
        raise TypeError("Y must be bfloat16, float16 or float32")
    R, K, ldy = _rows(Y, "Y")
    if rows.dim() != 2:
        raise ValueError("rows must be [M, top_k]")
    M, top_k = rows.shape
    if (M | K | R) >> 31:
        raise ValueError(_SIZE)
    dev = Y.device
    index = dev.index
    if index != _current_device():   # where the library launches
        raise ValueError("the tensors must be on the current CUDA device")
    at = _vector(rows, torch.int32, M * top_k, dev, "rows")
    w = _vector(weights, torch.float32, M * top_k, dev, "weights")
    res, ldr = None, K
    if residual is not None:
        if residual.dtype != Y.dtype:
            raise TypeError("residual must have Y's type")
        r, c, ldr = _rows(residual, "residual")
        if r != M or c != K or residual.device != dev:
            raise ValueError("residual must be [M, K] on the same device")
        res = residual.data_ptr()
    if out is None:
        out = torch.empty((M, K), dtype=Y.dtype, device=dev)
        ldo = K
    else:
        if out.dtype != Y.dtype:
            raise TypeError("out must have Y's type")
        r, c, ldo = _rows(out, "out")
        if r != M or c != K or out.device != dev:
            raise ValueError("out must be [M, K] on the same device")
    st = _raw_stream(index) if stream is None else _stream_ptr(stream)
    r = lib.qg_moe_combine(Y.data_ptr(), code, ldy, at, w, top_k, res, ldr, out.data_ptr(), ldo, M, R, K, st)
    if r:
        raise QgemmError(r, "qg_moe_combine")
    return out


MAX_DRAFTS = 31


class DraftCheck(NamedTuple):
    """What :func:`verify_drafts` returns."""
    accepted: Any   # int32 [B]: drafts that are kept
    tokens: Any     # int64 [B, G + 1]: those, the token that follows, then -1


def _batch_rows(t, what: str):
    """(sequences, rows, columns, sequence stride, row stride) of a 3-D CUDA tensor
    with unit column stride; strides of lone sequences and rows do not count."""
    if t.dim() != 3:
        raise ValueError(what + " must be a 3-D tensor")
    b, r, c = t.shape
    sb, sr, step = t.stride()
    if step != 1 and c > 1:
        raise ValueError(what + " must have unit stride in its last dimension")
    if not t.is_cuda:
        raise ValueError(what + " must be on a CUDA device")
    return b, r, c, (sb if b > 1 else 0), (sr if r > 1 else c)


def verify_drafts(target_logits, draft_tokens, draft_logits=None, uniform=None, noise=None, lengths=None,
                  workspace=None, stream=None) -> DraftCheck:
    """Drafted tokens against the target's probabilities, from given random numbers.

    target_logits: bf16, fp16 or fp32 CUDA [B, G + 1, V] (unit column stride), as
    tokens are drawn from them (divided by the temperature, -inf where a filter
    leaves a token out); draft_tokens: int64 [B, G], G <= MAX_DRAFTS; draft_logits
    (optional): [B, G, V] of the same type that the drafts were drawn from; without
    it they count as certain.  uniform: float32 [B, G] in [0, 1), noise: float32 [B, V]
    exponential.  lengths (optional): int32 [B], how many drafts a sequence has.

    Drafts are kept while uniform * q(d) < p(d); the next token is drawn from
    max(p - q, 0) at the first that is not kept, from p behind the last one, as the
    largest ratio of probability to noise.  Without uniform and noise: greedy, drafts
    are kept while they are the largest logit, and the largest follows.  (A row with
    a NaN, +inf or nothing left keeps no draft and yields -1; see include/qgemm.h.)
    workspace: as :func:`moe_route`'s.
    """
    if stream is not None and _elsewhere(stream):
        return _on_stream(stream, verify_drafts, target_logits, draft_tokens, draft_logits, uniform, noise, lengths,
                          workspace)
    torch = _torch()
    code = _dtype_codes.get(target_logits.dtype)
    if code is None:
        raise TypeError("target_logits must be bfloat16, float16 or float32")
    B, rows, V, t_seq, t_row = _batch_rows(target_logits, "target_logits")
    G = rows - 1
    if G < 0:
        raise ValueError("target_logits must have a row for each draft and one more")
    if (B | V) >> 31 or G >> 31:
        raise ValueError(_SIZE)
    dev = target_logits.device
    index = dev.index
    if index != _current_device():   # where the library launches
        raise ValueError("the tensors must be on the current CUDA device")
    if draft_tokens.dtype != torch.int64:
        raise TypeError("draft_tokens must be int64")
    if draft_tokens.shape != (B, G):
        raise ValueError("draft_tokens must be [B, G], target_logits [B, G + 1, V]")
    if draft_tokens.device != dev:
        raise ValueError("all tensors must be on one CUDA device")
    if not draft_tokens.is_contiguous():
        draft_tokens = draft_tokens.contiguous()
    if (uniform is None) != (noise is None):
        raise ValueError("uniform and noise belong together")
    d, d_seq, d_row = None, 0, V
    if draft_logits is not None:
        if noise is None:
            raise ValueError("draft_logits need uniform and noise")
        if draft_logits.dtype != target_logits.dtype:
            raise TypeError("draft_logits must have target_logits' type")
        b, r, c, d_seq, d_row = _batch_rows(draft_logits, "draft_logits")
        if (b, r, c) != (B, G, V) or draft_logits.device != dev:
            raise ValueError("draft_logits must be [B, G, V] on the same device")
        d = draft_logits.data_ptr() if G > 0 else None
    u = z = n = None
    ldu, ldn = G, V
    if noise is not None:
        f32 = torch.float32
        if uniform.dtype != f32 or noise.dtype != f32:
            raise TypeError("uniform and noise must be float32")
        r, c, ldu = _rows(uniform, "uniform")
        r2, c2, ldn = _rows(noise, "noise")
        if (r, c) != (B, G) or (r2, c2) != (B, V) or uniform.device != dev or noise.device != dev:
            raise ValueError("uniform must be [B, G] and noise [B, V] on the same device")
        z = noise.data_ptr()
        u = uniform.data_ptr() if G > 0 else z   # not read without drafts
    if lengths is not None:
        n = _vector(lengths, torch.int32, B, dev, "lengths")
    accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    tokens = torch.empty((B, G + 1), dtype=torch.int64, device=dev)
    st = _raw_stream(index)
    buf, ws, wsb = _scratch(("drafts", B, G, V, index), lambda: lib.qg_verify_drafts_workspace_bytes(B, G, V),
                            workspace, dev)
    r = lib.qg_verify_drafts(target_logits.data_ptr(), code, t_seq, t_row, d, d_seq, d_row, draft_tokens.data_ptr(), G,
                             u, ldu, z, ldn, n, accepted.data_ptr(), tokens.data_ptr(), B, G, V, ws, wsb, st)
    if r:
        raise QgemmError(r, "qg_verify_drafts")
    return DraftCheck(accepted, tokens)


def qgemm_bf16(X, W, Y=None, workspace=None, stream=None):
    """Y[M, N] = X[M, K] . W[N, K]^T with BF16 X, W and Y (FP32 sums).

    X: bf16 CUDA [M, K] (row stride a multiple of 8); W: bf16 [N, K]
    contiguous; Y (optional): bf16 [M, N] with unit column stride.
    """
    if stream is not None and Y is None and _elsewhere(stream):
        return _on_stream(stream, qgemm_bf16, X, W, Y, workspace)
    torch = _torch()
    if X.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise TypeError("X and W must be bfloat16")
    if not W.is_contiguous():
        raise TypeError("W must be contiguous")
    M, K = X.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("shape mismatch between X and W")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    ws, wsb = _workspace_for(KIND_BF16, M, N, K, workspace, X.device, stream)
    _check(lib.qgemm_bf16(X.data_ptr(), _ld(X), W.data_ptr(), Y.data_ptr(), _ld(Y), M, N, K, ws, wsb,
                          _stream_ptr(stream)), "qgemm_bf16")
    return Y


def lut3_packed_bytes(N: int, K: int) -> int:
    return int(lib.qg_lut3_packed_bytes(N, K))


def pack_lut3(codes: np.ndarray) -> np.ndarray:
    """Pack an [N, K] uint8 matrix of 3-bit codes (host) into the kernel layout."""
    c = np.ascontiguousarray(codes, dtype=np.uint8)
    N, K = c.shape
    out = np.empty(lut3_packed_bytes(N, K), dtype=np.uint8)
    _check(lib.pack_lut3(c.ctypes.data, out.ctypes.data, N, K), "pack_lut3")
    return out


def unpack_lut3(packed: np.ndarray, N: int, K: int) -> np.ndarray:
    p = np.ascontiguousarray(packed, dtype=np.uint8)
    if p.size < lut3_packed_bytes(N, K):
        raise ValueError("packed buffer too small")
    out = np.empty((N, K), dtype=np.uint8)
    _check(lib.unpack_lut3(p.ctypes.data, out.ctypes.data, N, K), "unpack_lut3")
    return out


def debug_fp8_split(X, stream=None):
    """The FP8 GEMM's activation split of BF16 X [B, 128] (one 128-wide K
    block per row): returns (hi, lo, e) with hi, lo uint8 E4M3 codes [B, 128]
    and e int32 [B], such that x * 2^e = hi + lo / 16 (see include/qgemm.h)."""
    if stream is not None and _elsewhere(stream):
        return _on_stream(stream, debug_fp8_split, X)
    torch = _torch()
    if X.dtype != torch.bfloat16 or X.dim() != 2 or X.shape[1] != 128 or not X.is_contiguous():
        raise ValueError("X must be a contiguous bfloat16 [B, 128] tensor")
    B = X.shape[0]
    hi = torch.empty((B, 128), dtype=torch.uint8, device=X.device)
    lo = torch.empty((B, 128), dtype=torch.uint8, device=X.device)
    e = torch.empty((B,), dtype=torch.int32, device=X.device)
    _check(lib.qg_debug_fp8_split(X.data_ptr(), B, hi.data_ptr(), lo.data_ptr(), e.data_ptr(), _stream_ptr(None)),
           "qg_debug_fp8_split")
    return hi, lo, e


def dequant_lut3(Wq, qmap, scales, N: int, K: int, out=None, stream=None):
    """Packed LUT3 weights -> FP16 [N, K], with the LUT3 GEMM's own dequantiser."""
    if stream is not None and out is None and _elsewhere(stream):
        return _on_stream(stream, dequant_lut3, Wq, qmap, scales, N, K, out)
    torch = _torch()
    if out is None:
        out = torch.empty((N, K), dtype=torch.float16, device=Wq.device)
    _check(lib.qg_dequant_lut3(Wq.data_ptr(), qmap.data_ptr(), scales.data_ptr(), out.data_ptr(), N, K,
                               _stream_ptr(stream)), "qg_dequant_lut3")
    return out


def last_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the kernels' status code."""
    return int(lib.qg_last_device_status(_stream_ptr(stream)))


def set_wait_timeout_ns(ns: int) -> None:
    lib.qg_set_wait_timeout_ns(int(ns))


def set_fault_injection(unit: int) -> None:
    lib.qg_set_fault_injection(int(unit))


def set_weight_prefetch_overlap(enable: bool) -> None:
    """Let consecutive GEMMs on a stream overlap (weights stream early); see
    include/qgemm.h for the condition under which this is safe."""
    lib.qg_set_weight_prefetch_overlap(1 if enable else 0)


def dispatch_set(kind: int, M: int, N: int, K: int, ctas: int) -> None:
    """Set (ctas > 0) or remove (ctas == 0) the dispatch-table grid of a shape."""
    _check(lib.qg_dispatch_set(kind, M, N, K, ctas), "qg_dispatch_set")
    _ws_need.clear()   # a shape's workspace need follows its grid


def dispatch_get(kind: int, M: int, N: int, K: int) -> int:
    """The grid (CTA count) the next call of this shape launches."""
    return int(lib.qg_dispatch_get(kind, M, N, K))


def dispatch_rule(kind: int, M: int, N: int, K: int, sms: int) -> int:
    """The grid the built-in cost rule picks for this shape on a device with
    `sms` SMs, ignoring the dispatch table (host only; 0 for invalid
    arguments)."""
    return int(lib.qg_dispatch_rule(kind, M, N, K, sms))


def dispatch_clear() -> None:
    lib.qg_dispatch_clear()
    _ws_need.clear()


def debug_schedule(kind: int, M: int, N: int, K: int, stream=None):
    """The device's work split of a shape: (ranges int64 [G, 2], info int32
    [G, 6]) as numpy arrays (see include/qgemm.h)."""
    if stream is not None and _elsewhere(stream):
        return _on_stream(stream, debug_schedule, kind, M, N, K)
    torch = _torch()
    g = ctypes.c_int(0)
    _check(lib.qg_debug_schedule(kind, M, N, K, ctypes.byref(g), None, None, 0, None), "qg_debug_schedule")
    G = g.value
    ranges = torch.empty((G, 2), dtype=torch.int64, device="cuda")
    info = torch.empty((G, 6), dtype=torch.int32, device="cuda")
    _check(lib.qg_debug_schedule(kind, M, N, K, ctypes.byref(g), ranges.data_ptr(), info.data_ptr(), G,
                                 _stream_ptr(None)), "qg_debug_schedule")
    torch.cuda.synchronize()
    return ranges.cpu().numpy(), info.cpu().numpy()


def workspace_bytes_max(N: int) -> int:
    """The workspace any grid of a shape with N output rows may need."""
    return int(lib.qg_workspace_bytes_max(N))


def _tune_common(M, N, X, Y_ref, workspace, nbytes=None, kind=KIND_FP8_BLOCK):
    if workspace is None:
        workspace = Workspace(X.device)
    need = workspace_bytes_max(N) if nbytes is None else nbytes
    buf = workspace.get(need, kind) if isinstance(workspace, Workspace) else workspace
    return buf, (buf.numel() * buf.element_size() if buf is not None else 0)


def tune_fp8(X, W_copies, W_scale, calls: int = 200, workspace=None, stream=None):
    """Exactness-gated tuning of the dispatch table for the shape of X and W
    (see qg_tune_fp8 in include/qgemm.h).  W_copies: equal E4M3 weight
    tensors the timed calls rotate over.  Returns (grid, us per call)."""
    if stream is not None and _elsewhere(stream):
        return _on_stream(stream, tune_fp8, X, W_copies, W_scale, calls, workspace)
    torch = _torch()
    M, K = X.shape
    N = W_copies[0].shape[0]
    Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    Y_ref = torch.empty_like(Y)
    buf, nb = _tune_common(M, N, X, Y_ref, workspace)
    ptrs = (ctypes.c_void_p * len(W_copies))(*[w.data_ptr() for w in W_copies])
    g, us = ctypes.c_int(0), ctypes.c_float(0)
    _check(lib.qg_tune_fp8(X.data_ptr(), _ld(X), ctypes.cast(ptrs, ctypes.c_void_p), len(W_copies),
                           W_scale.data_ptr(), Y.data_ptr(), N, Y_ref.data_ptr(), M, N, K,
                           buf.data_ptr() if buf is not None else None, nb, calls, ctypes.byref(g), ctypes.byref(us),
                           _stream_ptr(None)), "qg_tune_fp8")
    _ws_need.clear()
    return g.value, us.value


def workspace_bytes_max_w8a8(M: int, N: int) -> int:
    """The largest workspace any grid of a W8A8 shape with M activation rows
    and N output rows may need on the current device."""
    return int(lib.qg_workspace_bytes_max_w8a8(M, N))


def tune_bf16(X, W_copies, calls: int = 200, workspace=None, stream=None):
    """As tune_fp8 for the dense BF16 GEMM (W_copies: equal BF16 weights)."""
    if stream is not None and _elsewhere(stream):
        return _on_stream(stream, tune_bf16, X, W_copies, calls, workspace)
    torch = _torch()
    M, K = X.shape
    N = W_copies[0].shape[0]
    Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    Y_ref = torch.empty_like(Y)
    buf, nb = _tune_common(M, N, X, Y_ref, workspace)
    ptrs = (ctypes.c_void_p * len(W_copies))(*[w.data_ptr() for w in W_copies])
    g, us = ctypes.c_int(0), ctypes.c_float(0)
    _check(lib.qg_tune_bf16(X.data_ptr(), _ld(X), ctypes.cast(ptrs, ctypes.c_void_p), len(W_copies), Y.data_ptr(),
                            N, Y_ref.data_ptr(), M, N, K, buf.data_ptr() if buf is not None else None, nb, calls,
                            ctypes.byref(g), ctypes.byref(us), _stream_ptr(None)), "qg_tune_bf16")
    _ws_need.clear()
    return g.value, us.value


def tune_w8a8(Xq, X_scale, W_copies, W_scale, calls: int = 100, workspace=None, stream=None):
    """As tune_fp8 for the W8A8 GEMM on quantised activations (Xq, X_scale as
    quantize_act_e4m3 returns them; W_copies: equal E4M3 weights)."""
    if stream is not None and _elsewhere(stream):
        return _on_stream(stream, tune_w8a8, Xq, X_scale, W_copies, W_scale, calls, workspace)
    torch = _torch()
    M, K = Xq.shape
    N = W_copies[0].shape[0]
    Y = torch.empty((M, N), dtype=torch.bfloat16, device=Xq.device)
    Y_ref = torch.empty_like(Y)
    buf, nb = _tune_common(M, N, Xq, Y_ref, workspace, workspace_bytes_max_w8a8(M, N), KIND_W8A8)
    ptrs = (ctypes.c_void_p * len(W_copies))(*[w.data_ptr() for w in W_copies])
    g, us = ctypes.c_int(0), ctypes.c_float(0)
    _check(lib.qg_tune_w8a8(Xq.data_ptr(), _ld(Xq), X_scale.data_ptr(), _ld(X_scale),
                            ctypes.cast(ptrs, ctypes.c_void_p), len(W_copies), W_scale.data_ptr(), Y.data_ptr(), N,
                            Y_ref.data_ptr(), M, N, K, buf.data_ptr() if buf is not None else None, nb, calls,
                            ctypes.byref(g), ctypes.byref(us), _stream_ptr(None)), "qg_tune_w8a8")
    _ws_need.clear()
    return g.value, us.value


def tune_lut3(X, Wq_copies, qmap, scales, N: int, calls: int = 200, workspace=None, stream=None):
    """As tune_fp8 for the 3-bit LUT GEMM (Wq_copies: equal packed weights)."""
    if stream is not None and _elsewhere(stream):
        return _on_stream(stream, tune_lut3, X, Wq_copies, qmap, scales, N, calls, workspace)
    torch = _torch()
    M, K = X.shape
    Y = torch.empty((M, N), dtype=torch.float16, device=X.device)
    Y_ref = torch.empty_like(Y)
    buf, nb = _tune_common(M, N, X, Y_ref, workspace)
    ptrs = (ctypes.c_void_p * len(Wq_copies))(*[w.data_ptr() for w in Wq_copies])
    g, us = ctypes.c_int(0), ctypes.c_float(0)
    _check(lib.qg_tune_lut3(X.data_ptr(), _ld(X), ctypes.cast(ptrs, ctypes.c_void_p), len(Wq_copies),
                            qmap.data_ptr(), scales.data_ptr(), Y.data_ptr(), N, Y_ref.data_ptr(), M, N, K,
                            buf.data_ptr() if buf is not None else None, nb, calls, ctypes.byref(g),
                            ctypes.byref(us), _stream_ptr(None)), "qg_tune_lut3")
    _ws_need.clear()
    return g.value, us.value
