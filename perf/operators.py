"""Cases, inputs and plain forms of the 8-bit integer scoring path.

Three operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and through the library's entry points:

* ``quantize``  -- activations [M, K] to 8-bit integers with one scale per
  token (row): inv = 127 / max |x|, code = round-half-even(x * inv),
  scale = max |x| / 127; a row whose largest |x| is below 2^-100 has codes 0
  and scale 1.
* ``gemm``      -- Y[m, n] = sx[m] * sw[n] * sum_k xq[m, k] * w[n, k] (+ bias[n])
  of such codes with 8-bit integer weights and one scale per channel (row of W).
* ``logprobs``  -- for every row of logits, over the softmax of the row: the
  log probabilities of given tokens, the entropy in nats, and the top
  alternatives with their log probabilities (ties to the lower index).

``own`` selects the side; ``run`` is one call of a user's program.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step's activations before an FFN projection
        dict(name="quantize decode", op="quantize", M=16, K=5120, x="bf16"),
        # a long prompt's activations before the down projection
        dict(name="quantize prompt", op="quantize", M=4096, K=17408, x="bf16"),
        # one token through a small attention projection: latency
        dict(name="gemm one token", op="gemm", M=1, N=1024, K=5120, y="bf16", bias=False),
        # a decode batch through the FFN gate or up projection
        dict(name="gemm decode", op="gemm", M=16, N=17408, K=5120, y="bf16", bias=False),
        # a full decode batch's logits, kept in 32 bits for the scoring that follows
        dict(name="gemm logits", op="gemm", M=32, N=32768, K=5120, y="fp32", bias=False),
        # odd sizes: a ragged chunk of tokens, an odd channel count, a short K, a bias
        dict(name="gemm ragged", op="gemm", M=83, N=5003, K=1040, y="fp16", bias=True),
        # a prefill chunk or a batched verification through the down projection
        dict(name="gemm chunk", op="gemm", M=256, N=5120, K=17408, y="bf16", bias=False),
        # a long prompt through the gate or up projection: bound by the tensor cores
        dict(name="gemm prompt", op="gemm", M=4096, N=17408, K=5120, y="bf16", bias=False),
        # one sampled token's log probability with a few alternatives: latency
        dict(name="logprobs one row", op="logprobs", M=1, V=32768, x="bf16", T=1, top=5, masked=False, pad=0),
        # a decode batch over a large vocabulary, 32-bit logits, the most alternatives usually asked for
        dict(name="logprobs decode", op="logprobs", M=32, V=131072, x="fp32", T=1, top=20, masked=False, pad=0),
        # odd vocabulary, rows apart in memory, a part of each row's tokens banned, several candidate tokens a row
        dict(name="logprobs banned", op="logprobs", M=333, V=50021, x="fp16", T=4, top=8, masked=True, pad=27),
        # scoring a long prompt's tokens
        dict(name="logprobs prompt", op="logprobs", M=4096, V=131072, x="bf16", T=1, top=1, masked=False, pad=0),
    ]


def _log_int(rng, lo, hi):
    """A whole number in lo..hi, uniform over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "logprobs", "logprobs"])
    if op == "quantize":
        K = 16 * _log_int(rng, 4, 1280)
        M = _log_int(rng, 1, min(8192, 4096 * 17408 // K))
        return dict(op=op, M=M, K=K, x=rng.choice(["bf16", "fp16"]))
    if op == "gemm":
        K = 16 * _log_int(rng, 4, 1088)
        N = _log_int(rng, 64, 32768)
        M = _log_int(rng, 1, 4096)
        while M * N * K > 4096 * 17408 * 5120:
            M //= 2
        return dict(op=op, M=M, N=N, K=K, y=rng.choice(["bf16", "fp16", "fp32"]), bias=rng.random() < 0.3)
    x = rng.choice(["bf16", "fp16", "fp32"])
    V = _log_int(rng, 1000, 160000)
    M = _log_int(rng, 1, min(4096, 2 ** (30 if x != "fp32" else 29) // 2 // V))
    return dict(op=op, M=M, V=V, x=x, T=rng.choice([1, 1, 2, 4]), top=rng.choice([0, 1, 5, 8, 20]),
                masked=rng.random() < 0.3, pad=rng.choice([0, 0, 5, 64]))


# ----------------------------------------------------------------- the inputs
def _quantized_rows(t):
    """Codes and scales of a float tensor's rows, symmetric in -127..127."""
    amax = t.abs().amax(dim=1).clamp_min(1e-20)
    q = torch.round(t * (127.0 / amax)[:, None]).to(torch.int8)
    return q, amax / 127.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)

    def normal(*size):
        return torch.randn(*size, generator=g, device="cuda", dtype=torch.float32)

    if case["op"] == "quantize":
        # activations with a few channels far above the others
        gain = torch.where(torch.rand(case["K"], generator=g, device="cuda") < 0.01, 12.0, 1.0)
        X = (normal(case["M"], case["K"]) * gain).to(_DTYPES[case["x"]])
        return {"case": case, "X": X}
    if case["op"] == "gemm":
        Xq, sx = _quantized_rows(normal(case["M"], case["K"]))
        W, sw = _quantized_rows(normal(case["N"], case["K"]).mul_(0.02))
        bias = normal(case["N"]) if case["bias"] else None
        return {"case": case, "Xq": Xq, "sx": sx, "W": W, "sw": sw, "bias": bias}
    M, V = case["M"], case["V"]
    rows = torch.empty((M, V + case["pad"]), dtype=_DTYPES[case["x"]], device="cuda")
    rows[:, V:] = 0.0
    sharp = 1.0 + 2.0 * torch.rand(M, 1, generator=g, device="cuda")   # from flat to peaked rows
    step = max(1, (1 << 27) // V)
    for a in range(0, M, step):
        b = min(M, a + step)
        part = normal(b - a, V).mul_(sharp[a:b])
        if case["masked"]:
            part.masked_fill_(torch.rand(b - a, V, generator=g, device="cuda") < 0.3, float("-inf"))
        rows[a:b, :V] = part
    tokens = torch.randint(0, V, (M, case["T"]), generator=g, device="cuda", dtype=torch.int64)
    return {"case": case, "logits": rows[:, :V], "tokens": tokens}


# ----------------------------------------------------------------- plain forms
def _plain_quantize(X):
    x = X.float()
    amax = x.abs().amax(dim=1)
    live = amax >= 2.0 ** -100
    a = torch.where(live, amax, torch.full_like(amax, 127.0))
    codes = torch.where(live[:, None], torch.round(x * (127.0 / a)[:, None]), 0.0).to(torch.int8)
    return codes, a / 127.0


def _plain_gemm(Xq, sx, W, sw, bias, dtype):
    y = (Xq.float() @ W.float().t()) * sx[:, None] * sw[None, :]
    if bias is not None:
        y = y + bias[None, :]
    return y.to(dtype)


def _plain_logprobs(logits, tokens, top):
    x = logits.float()
    m = x.amax(dim=1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    s = e.sum(dim=1, keepdim=True)
    log_s = torch.log(s)
    entropy = log_s - torch.where(e > 0, e * d, 0.0).sum(dim=1, keepdim=True) / s
    token = torch.gather(d, 1, tokens) - log_s
    if top == 0:
        return {"token": token, "entropy": entropy[:, 0]}
    # one whole number per logit that orders by value, then by lower index
    bits = (x + 0.0).view(torch.int32)
    bits = bits ^ ((bits >> 31) & 0x7FFFFFFF)
    key = bits.to(torch.int64) * (1 << 32) + ((1 << 32) - 1 - torch.arange(x.shape[1], device=x.device))
    ids = (1 << 32) - 1 - (torch.topk(key, top, dim=1).values & ((1 << 32) - 1))
    return {"token": token, "entropy": entropy[:, 0], "top_ids": ids, "top": torch.gather(d, 1, ids) - log_s}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import weight_only_quantized_qgemm_gb300 as qg
        if op == "quantize":
            codes, scale = qg.quantize_act_int8(state["X"])
            return {"codes": codes, "scale": scale}
        if op == "gemm":
            return qg.qgemm_w8a8_int8(state["Xq"], state["sx"], state["W"], state["sw"], bias=state["bias"],
                                      out_dtype=_DTYPES[case["y"]])
        r = qg.logprobs(state["logits"], state["tokens"], top_k=case["top"], entropy=True)
        if case["top"] == 0:
            return {"token": r.token_logprobs, "entropy": r.entropy}
        return {"token": r.token_logprobs, "entropy": r.entropy, "top_ids": r.top_ids, "top": r.top_logprobs}
    if op == "quantize":
        codes, scale = _plain_quantize(state["X"])
        return {"codes": codes, "scale": scale}
    if op == "gemm":
        return _plain_gemm(state["Xq"], state["sx"], state["W"], state["sw"], state["bias"], _DTYPES[case["y"]])
    return _plain_logprobs(state["logits"], state["tokens"], case["top"])


def work(case):
    if case["op"] == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": 3.0 * n + 4.0 * case["M"], "flops": 3.0 * n}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        nbytes = M * K + N * K + M * N * _BYTES[case["y"]] + 4.0 * (M + N) + (4.0 * N if case["bias"] else 0.0)
        return {"bytes": float(nbytes), "flops": 2.0 * M * N * K}
    M, V = case["M"], case["V"]
    nbytes = M * V * _BYTES[case["x"]] + M * (12.0 * case["T"] + 4.0 + 12.0 * case["top"])
    return {"bytes": float(nbytes), "flops": 5.0 * M * V}


# ----------------------------------------------------------------- 64 bits
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "quantize":
        largest = torch.stack([r.double().abs().max() for r in s["X"].split(1)]) if case["M"] <= 64 else \
            torch.cat([r.double().abs().max(dim=1).values for r in s["X"].split(256)])
        scale = torch.where(largest < 2.0 ** -100, torch.ones_like(largest), largest / 127)
        return {"codes": None, "scale": scale}   # a code's tie goes by the 32-bit rounding of the inverse scale
    if case["op"] == "gemm":
        wt = (s["W"].double() * s["sw"].double().unsqueeze(1)).t()
        out = [(q.double() * a.double().unsqueeze(1)) @ wt for q, a in zip(s["Xq"].split(512), s["sx"].split(512))]
        y = torch.cat(out)
        return y if s["bias"] is None else y + s["bias"].double()
    token, entropy, ids, top = [], [], [], []
    step = max(1, (1 << 27) // case["V"])
    for rows, asked in zip(s["logits"].split(step), s["tokens"].split(step)):
        lp = torch.log_softmax(rows.double(), dim=1)
        token.append(lp.gather(1, asked))
        entropy.append(torch.special.entr(lp.exp()).sum(dim=1))
        if case["top"]:
            top.append(lp.topk(case["top"], dim=1).values)
    out = {"token": torch.cat(token), "entropy": torch.cat(entropy)}
    if case["top"]:
        out["top_ids"] = None   # whole numbers: held to the plain form's
        out["top"] = torch.cat(top)
    return out
