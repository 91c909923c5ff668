"""Cases, inputs and plain forms of the expert layers' operators and of the
verification of drafted tokens.

Five operators, each in its plain form (elementary torch operations in 32 bits,
rounded once at the end) and through the library's entry points:

* ``route``    -- router of a layer of experts: for every token the top_k experts
  by score (softmax or sigmoid of the logits, plus a bias per expert where one is
  given; ties to the lower index; -inf: masked), their weights (the score without
  the bias, over the sum of the chosen, times a scale), where each expert's rows
  begin in the order by expert, and the row of every choice in that order.
* ``quantize`` -- activations to E4M3 with a scale for each row and 128 columns
  (largest |x| / 448), either copied to the rows of a token's experts, or of
  silu(gate) * up between an expert's two products.
* ``gemm``     -- Y[r] = sum over blocks kb of 128: sx[kb, r] * s[e, n/128, kb] *
  (xq[r, kb] . w[e, n, kb]) for the rows r of each expert e: groups of ragged size.
* ``combine``  -- out[m] = sum_j weight[m, j] * Y[row[m, j]] (+ residual[m]).
* ``verify``   -- drafted tokens against the target's probabilities: token j is
  kept while u_j q_j(d_j) < p_j(d_j); at the first one that is not, a token is
  drawn from max(p - q, 0), behind the last one from p: the largest ratio of
  probability to an exponential random number.  The random numbers are inputs.

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
        # one decode step of 16 sequences through a layer's router: latency
        dict(name="route decode", op="route", M=16, E=128, k=8, x="fp32", score="softmax", bias=False, scale=1.0),
        # a long prompt through a router with sigmoid scores and balancing biases
        dict(name="route prompt", op="route", M=8192, E=256, k=8, x="bf16", score="sigmoid", bias=True, scale=2.5),
        # a long prompt's activations, once for each of a token's eight experts
        dict(name="quantize to experts", op="quantize", M=4096, K=5120, E=128, k=8, gated=False),
        # between the experts' two products, an odd number of rows
        dict(name="quantize gated", op="quantize", M=32763, K=2048, E=64, k=1, gated=True),
        # one token's eight experts of 128, gate and up in one product: latency
        dict(name="gemm one token", op="gemm", M=1, E=128, k=8, N=4096, K=2048, y="bf16"),
        # a decode batch: most experts hold a few tokens, bound by the weights
        dict(name="gemm decode", op="gemm", M=64, E=128, k=8, N=2048, K=5120, y="bf16"),
        # odd sizes: ragged groups around a tile's size, odd channels, a short K, 32-bit output
        dict(name="gemm ragged", op="gemm", M=333, E=20, k=4, N=1003, K=1040, y="fp32"),
        # a long prompt through the experts' gate and up products: bound by the tensor cores
        dict(name="gemm prompt", op="gemm", M=8192, E=64, k=8, N=4096, K=4096, y="bf16"),
        # a decode batch's experts' results back to the tokens: latency
        dict(name="combine decode", op="combine", M=64, K=5120, E=128, k=8, y="bf16", residual=True),
        # a long prompt's, an odd number of tokens
        dict(name="combine prompt", op="combine", M=8191, K=5120, E=128, k=8, y="bf16", residual=False),
        # one sequence with four drafted tokens: latency
        dict(name="verify one", op="verify", B=1, G=4, V=32768, x="bf16", draft="sampled", pad=0),
        # a batch of sequences with up to five drafted tokens over a large vocabulary
        dict(name="verify batch", op="verify", B=64, G=5, V=131072, x="bf16", draft="sampled", pad=0),
    ]


def _log_int(rng, lo, hi):
    """A whole number in lo..hi, uniform over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quantize", "gemm", "gemm", "gemm", "combine", "verify", "verify"])
    E = _log_int(rng, 2, 256)
    k = rng.randint(1, min(8, E))
    if op == "route":
        return dict(op=op, M=_log_int(rng, 1, 16384), E=E, k=k, x=rng.choice(["bf16", "fp16", "fp32"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    if op == "quantize":
        K = 16 * _log_int(rng, 4, 448)
        if rng.random() < 0.5:
            return dict(op=op, M=_log_int(rng, 1, min(32768, 2 ** 27 // K)), K=K, E=E, k=1, gated=True)
        return dict(op=op, M=_log_int(rng, 1, min(8192, 2 ** 27 // K // k)), K=K, E=E, k=k, gated=False)
    if op == "gemm":
        K = 16 * _log_int(rng, 8, 448)
        N = _log_int(rng, 64, 8192)
        while E * N * K > 5 * 2 ** 28:
            E = max(k, E // 2)
            N = max(64, N // 2)
        M = _log_int(rng, 1, 8192)
        while M * k * N * K > 2 ** 40:
            M //= 2
        return dict(op=op, M=M, E=E, k=k, N=N, K=K, y=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "combine":
        K = 8 * _log_int(rng, 8, 1024)
        return dict(op=op, M=_log_int(rng, 1, min(16384, 2 ** 28 // K // k)), K=K, E=E, k=k,
                    y=rng.choice(["bf16", "bf16", "fp16", "fp32"]), residual=rng.random() < 0.5)
    x = rng.choice(["bf16", "fp16", "fp32"])
    V = _log_int(rng, 1000, 160000)
    G = rng.randint(1, 8)
    return dict(op=op, B=_log_int(rng, 1, max(1, min(128, 2 ** 27 // (2 * G + 1) // V))), G=G, V=V, x=x,
                draft=rng.choice(["sampled", "sampled", "certain", "greedy"]), pad=rng.choice([0, 0, 5, 64]))


# ----------------------------------------------------------------- the inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _normal(g, *size):
    return torch.randn(*size, generator=g, device="cuda", dtype=torch.float32)


def _router_logits(g, M, E):
    """Experts of unlike popularity."""
    return _normal(g, M, E).mul_(1.5).add_(_normal(g, 1, E).mul_(0.7))


def _by_expert(experts, E):
    """Where each expert's rows begin, and the row of every choice in the order by expert and token."""
    flat = experts.reshape(-1).to(torch.int64)
    order = torch.sort(flat, stable=True).indices
    rows = torch.empty_like(flat)
    rows[order] = torch.arange(flat.numel(), device=flat.device)
    sizes = (flat[:, None] == torch.arange(E, device=flat.device)[None, :]).sum(dim=0)
    offsets = torch.cat([sizes.new_zeros(1), torch.cumsum(sizes, dim=0)])
    return offsets.to(torch.int32), rows.reshape(experts.shape).to(torch.int32)


def _e4m3(t):
    return t.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "verify":
        B, G, V = case["B"], case["G"], case["V"]
        sharp = 1.5 + 2.0 * torch.rand(B, 1, 1, generator=g, device="cuda")
        target = torch.zeros((B, G + 1, V + case["pad"]), dtype=_DTYPES[case["x"]], device="cuda")
        tokens = torch.empty((B, G), dtype=torch.int64, device="cuda")
        drafts = torch.zeros((B, G, V + case["pad"]), dtype=_DTYPES[case["x"]], device="cuda")
        for b in range(B):
            t = _normal(g, G + 1, V).mul_(sharp[b])
            target[b, :, :V] = t
            d = (t[:G] + 0.6 * _normal(g, G, V)).to(_DTYPES[case["x"]])
            drafts[b, :, :V] = d
            if case["draft"] == "greedy":
                # a draft model that mostly agrees with the target's likeliest token
                tokens[b] = torch.where(torch.rand(G, generator=g, device="cuda") < 0.8,
                                        target[b, :G, :V].float().argmax(dim=1), d.float().argmax(dim=1))
            elif case["draft"] == "certain":
                tokens[b] = d.float().argmax(dim=1)
            else:
                race = torch.empty(G, V, device="cuda").exponential_(generator=g)
                tokens[b] = (torch.softmax(d.float(), dim=1) / race).argmax(dim=1)
        uniform = torch.rand(B, G, generator=g, device="cuda")
        noise = torch.empty(B, V, device="cuda").exponential_(generator=g).clamp_min_(1e-30)
        # all sequences of a batch draft the most, but every third one
        lengths = torch.full((B,), G, dtype=torch.int32, device="cuda")
        lengths[2::3] = G // 2
        return {"case": case, "target": target[:, :, :V], "drafts": drafts[:, :, :V], "tokens": tokens,
                "uniform": uniform, "noise": noise, "lengths": lengths}
    M, E, k = case["M"], case["E"], case["k"]
    logits = _router_logits(g, M, E)
    if op == "route":
        bias = _normal(g, E).mul_(0.1) if case["bias"] else None
        return {"case": case, "logits": logits.to(_DTYPES[case["x"]]), "bias": bias}
    chosen = torch.topk(logits, k, dim=1)
    offsets, rows = _by_expert(chosen.indices, E)
    K = case["K"]
    state = {"case": case, "offsets": offsets, "rows": rows}
    if op == "quantize":
        # activations with a few channels far above the others
        gain = torch.where(torch.rand(K * (1 + case["gated"]), generator=g, device="cuda") < 0.01, 8.0, 1.0)
        X = torch.empty((M, K * (1 + case["gated"])), dtype=torch.bfloat16, device="cuda")
        for a in range(0, M, 4096):
            X[a:a + 4096] = _normal(g, min(M, a + 4096) - a, X.shape[1]).mul_(gain)
        state["X"] = X
        return state
    if op == "combine":
        Y = torch.empty((M * k, K), dtype=_DTYPES[case["y"]], device="cuda")
        for a in range(0, M * k, 8192):
            Y[a:a + 8192] = _normal(g, min(M * k, a + 8192) - a, K)
        state["Y"] = Y
        state["weights"] = torch.softmax(chosen.values, dim=1)
        state["residual"] = _normal(g, M, K).to(_DTYPES[case["y"]]) if case["residual"] else None
        return state
    N, R, KB = case["N"], M * k, -(-K // 128)
    Xq = torch.empty((R, K), dtype=torch.float8_e4m3fn, device="cuda")
    for a in range(0, R, 8192):
        Xq[a:a + 8192] = _e4m3(_normal(g, min(R, a + 8192) - a, K).mul_(100.0))
    X_scale = torch.zeros((KB, -(-R // 32) * 32), device="cuda")
    X_scale[:, :R] = torch.rand(KB, R, generator=g, device="cuda").mul_(0.01).add_(0.005)
    W = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(E):
        W[e] = _e4m3(_normal(g, N, K).mul_(100.0))
    W_scale = torch.rand(E, -(-N // 128), KB, generator=g, device="cuda").mul_(2e-4).add_(1e-4)
    # for the plain form: the experts that hold a row, and the largest group
    sizes = offsets[1:] - offsets[:-1]
    state.update(Xq=Xq, X_scale=X_scale, W=W, W_scale=W_scale, active=torch.nonzero(sizes)[:, 0], most=int(sizes.max()))
    return state


# ----------------------------------------------------------------- plain forms
def _plain_route(logits, bias, k, score, scale):
    x = logits.float()
    masked = torch.isinf(x)
    # the scores that decide are next to one another: in 64 bits
    wide = torch.sigmoid(x.double()) if score == "sigmoid" else torch.softmax(x.double(), dim=1)
    by = x.double() if bias is None else wide + bias.double()[None, :]
    by = torch.where(masked, -math.inf, by)
    first = torch.sort(by, dim=1, descending=True, stable=True)
    experts = first.indices[:, :k]
    live = first.values[:, :k] > -math.inf
    if score == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        s = torch.exp(x - x.amax(dim=1, keepdim=True))
    w = torch.where(live, torch.gather(s, 1, experts), 0.0)
    w = w * (scale / w.sum(dim=1, keepdim=True))
    offsets, rows = _by_expert(experts, x.shape[1])
    return {"experts": experts.to(torch.int32), "weights": w, "offsets": offsets, "rows": rows}


def _plain_quantize(X, gated, rows):
    x = X.float()
    if gated:
        gate, up = x[:, :x.shape[1] // 2], x[:, x.shape[1] // 2:]
        x = gate / (1.0 + torch.exp(-gate)) * up
    M, K = x.shape
    KB = -(-K // 128)
    padded = torch.zeros((M, KB * 128), device=x.device)
    padded[:, :K] = x
    blocks = padded.view(M, KB, 128)
    amax = blocks.abs().amax(dim=2)
    scale = torch.where(amax > 0, amax / 448.0, 1.0)
    codes = (blocks / scale[:, :, None]).reshape(M, KB * 128)[:, :K].to(torch.float8_e4m3fn)
    if gated:
        return codes, scale.t().contiguous()
    at = rows.reshape(-1).to(torch.int64)
    token = torch.arange(M, device=x.device)[:, None].expand(rows.shape).reshape(-1)
    out = torch.empty((at.numel(), K), dtype=torch.uint8, device=x.device)
    out[at] = codes.view(torch.uint8)[token]
    out_scale = torch.empty((KB, at.numel()), device=x.device)
    out_scale[:, at] = scale.t()[:, token]
    return out.view(torch.float8_e4m3fn), out_scale


def _plain_gemm(Xq, X_scale, W, W_scale, offsets, active, most, dtype):
    R, K = Xq.shape
    N, KB = W.shape[1], X_scale.shape[0]
    row = torch.arange(R, device=Xq.device)
    expert = (row[:, None] >= offsets[None, 1:]).sum(dim=1)
    place = row - offsets.to(torch.int64)[expert]
    group = (expert[:, None] > active[None, :]).sum(dim=1)        # its number among the active ones
    over = torch.arange(KB, device=Xq.device).repeat_interleave(128)[:K]
    x = torch.zeros((active.numel(), most, K), device=Xq.device)
    x[group, place] = Xq.float() * X_scale[:, :R].t()[:, over]
    channel = torch.arange(N, device=Xq.device) // 128
    w = W.view(torch.uint8)[active].view(torch.float8_e4m3fn).float()
    w *= W_scale[active][:, channel][:, :, over]
    return torch.bmm(x, w.transpose(1, 2))[group, place].to(dtype)


def _plain_combine(Y, rows, weights, residual):
    out = (Y[rows.to(torch.int64)].float() * weights[:, :, None]).sum(dim=1)
    if residual is not None:
        out = out + residual.float()
    return out.to(Y.dtype)


def _plain_verify(target, drafts, tokens, uniform, noise, lengths, draft, wide):
    B, G1, V = target.shape
    G = G1 - 1
    at = torch.arange(G, device=target.device)
    x = target.to(wide)
    if draft == "greedy":
        best = torch.where(x == x.amax(dim=2, keepdim=True), torch.arange(V, device=x.device), V).amin(dim=2)
        keep = tokens == best[:, :G]
    else:
        p = torch.exp(x - x.amax(dim=2, keepdim=True))
        p = p / p.sum(dim=2, keepdim=True)
        if draft == "certain":
            q = (torch.arange(V, device=x.device)[None, None, :] == tokens[:, :, None]).to(wide)
        else:
            q = drafts.to(wide)
            q = torch.exp(q - q.amax(dim=2, keepdim=True))
            q = q / q.sum(dim=2, keepdim=True)
        ask = tokens[:, :, None]
        keep = uniform.to(wide) * torch.gather(q, 2, ask)[:, :, 0] < torch.gather(p, 2, ask)[:, :, 0]
    keep = keep & (at[None, :] < lengths[:, None])
    accepted = torch.cumprod(keep.to(torch.int32), dim=1).sum(dim=1)
    if draft == "greedy":
        last = torch.gather(best, 1, accepted[:, None])
    else:
        each = torch.arange(B, device=x.device)
        rest = p[each, accepted]
        drafted = accepted < lengths
        left = (rest - q[each, accepted.clamp_max(G - 1)]).clamp_min(0.0)
        rest = torch.where((drafted & (left.amax(dim=1) > 0))[:, None], left, rest)
        last = (rest / noise.to(wide)).argmax(dim=1, keepdim=True)
    out = torch.cat([tokens, last], dim=1)
    place = torch.arange(G1, device=x.device)[None, :]
    out = torch.where(place < accepted[:, None], out, torch.where(place == accepted[:, None], last, -1))
    return {"accepted": accepted.to(torch.int32), "tokens": out}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import weight_only_quantized_qgemm_gb300 as qg
        if op == "route":
            r = qg.moe_route(state["logits"], case["k"], score=case["score"], bias=state["bias"], scale=case["scale"])
            return {"experts": r.experts, "weights": r.weights, "offsets": r.offsets, "rows": r.rows}
        if op == "quantize":
            codes, scale = qg.quantize_rows_e4m3(state["X"], gated=case["gated"],
                                                 rows=None if case["gated"] else state["rows"])
            return {"codes": codes.view(torch.float8_e4m3fn), "scale": scale[:, :codes.shape[0]]}
        if op == "gemm":
            return qg.qgemm_w8a8_grouped(state["Xq"], state["X_scale"], state["W"], state["W_scale"], state["offsets"],
                                         out_dtype=_DTYPES[case["y"]])
        if op == "combine":
            return qg.moe_combine(state["Y"], state["rows"], state["weights"], residual=state["residual"])
        draft = case["draft"]
        r = qg.verify_drafts(state["target"], state["tokens"],
                             draft_logits=state["drafts"] if draft == "sampled" else None,
                             uniform=None if draft == "greedy" else state["uniform"],
                             noise=None if draft == "greedy" else state["noise"], lengths=state["lengths"])
        return {"accepted": r.accepted, "tokens": r.tokens}
    if op == "route":
        return _plain_route(state["logits"], state["bias"], case["k"], case["score"], case["scale"])
    if op == "quantize":
        codes, scale = _plain_quantize(state["X"], case["gated"], state["rows"])
        return {"codes": codes, "scale": scale}
    if op == "gemm":
        return _plain_gemm(state["Xq"], state["X_scale"], state["W"], state["W_scale"], state["offsets"],
                           state["active"], state["most"], _DTYPES[case["y"]])
    if op == "combine":
        return _plain_combine(state["Y"], state["rows"], state["weights"], state["residual"])
    return _plain_verify(state["target"], state["drafts"], state["tokens"], state["uniform"], state["noise"],
                         state["lengths"], case["draft"], torch.float32)


def work(case):
    op = case["op"]
    if op == "verify":
        B, G, V = case["B"], case["G"], case["V"]
        rows = B * (G + 1) + (B * G if case["draft"] == "sampled" else 0)
        nbytes = rows * V * _BYTES[case["x"]] + (0 if case["draft"] == "greedy" else 4 * B * V) + B * (20.0 * G + 16)
        return {"bytes": float(nbytes), "flops": 4.0 * rows * V}
    M, E, k = case["M"], case["E"], case["k"]
    if op == "route":
        return {"bytes": float(M * E * _BYTES[case["x"]] + 12 * M * k + 4 * (E + 1)), "flops": 8.0 * M * E}
    K = case["K"]
    if op == "quantize":
        wide = 2 if case["gated"] else 1
        return {"bytes": float(M * K * 2 * wide + M * k * (K + 4 * -(-K // 128)) + (0 if case["gated"] else 4 * M * k)),
                "flops": (10.0 if case["gated"] else 3.0) * M * K}
    if op == "combine":
        n = _BYTES[case["y"]]
        return {"bytes": float(M * k * (K * n + 8) + M * K * n * (2 if case["residual"] else 1)), "flops": 2.0 * M * k * K}
    N, R = case["N"], M * k
    held = E * (1.0 - (1.0 - k / E) ** M)     # experts that hold a token, on the average of an even routing
    return {"bytes": held * N * (K + 4.0 / 128 * -(-K // 128)) + R * (K + 4.0 * -(-K // 128) + N * _BYTES[case["y"]]),
            "flops": 2.0 * R * N * K}


# ----------------------------------------------------------------- 64 bits
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        x = s["logits"].double()
        score = 1 / (1 + torch.exp(-x)) if case["score"] == "sigmoid" else torch.exp(torch.log_softmax(x, dim=1))
        by = x if s["bias"] is None else score + s["bias"].double()
        experts = torch.argsort(by, dim=1, descending=True, stable=True)[:, :case["k"]]
        w = score.gather(1, experts)
        # the whole numbers are held to the plain form's
        return {"experts": None, "weights": case["scale"] * w / w.sum(dim=1, keepdim=True), "offsets": None, "rows": None}
    if op == "quantize":
        scale = []
        for x in s["X"].split(1024):
            x = x.double()
            if case["gated"]:
                x = torch.nn.functional.silu(x[:, :case["K"]]) * x[:, case["K"]:]
            largest = torch.stack([b.abs().amax(dim=1) for b in x.split(128, dim=1)])
            scale.append(torch.where(largest == 0, torch.ones_like(largest), largest / 448))
        scale = torch.cat(scale, dim=1)
        if not case["gated"]:
            moved = torch.empty((scale.shape[0], case["M"] * case["k"]), dtype=torch.float64, device=scale.device)
            for j in range(case["k"]):
                moved[:, s["rows"][:, j].long()] = scale
            scale = moved
        return {"codes": None, "scale": scale}   # a code's tie goes by the 32-bit quotient
    if op == "gemm":
        if 2.0 * case["M"] * case["k"] * case["N"] * case["K"] > 3e12:
            return None
        K, N = case["K"], case["N"]
        y = torch.empty((case["M"] * case["k"], N), dtype=torch.float64, device="cuda")
        begin = s["offsets"].tolist()
        for e in range(case["E"]):
            a, b = begin[e], begin[e + 1]
            if a == b:
                continue
            total = torch.zeros((b - a, N), dtype=torch.float64, device="cuda")
            for kb in range(s["X_scale"].shape[0]):
                cols = slice(128 * kb, min(K, 128 * kb + 128))
                inner = s["Xq"][a:b, cols].to(torch.float64) @ s["W"][e, :, cols].to(torch.float64).t()
                per = s["W_scale"][e, :, kb].double().repeat_interleave(128)[:N]
                total += inner * s["X_scale"][kb, a:b].double()[:, None] * per[None, :]
            y[a:b] = total
        return y
    if op == "combine":
        out = torch.zeros((case["M"], case["K"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            out += s["weights"][:, j:j + 1].double() * s["Y"][s["rows"][:, j].long()].double()
        return out if s["residual"] is None else out + s["residual"].double()
    accepted, tokens = [], []
    for b in range(case["B"]):
        p = torch.softmax(s["target"][b].double(), dim=1)
        n, length = 0, int(s["lengths"][b])
        if case["draft"] == "greedy":
            while n < length and int(s["target"][b, n].float().argmax()) == int(s["tokens"][b, n]):
                n += 1
            last = int(s["target"][b, n].float().argmax())
        else:
            q = torch.zeros_like(p[:case["G"]])
            if case["draft"] == "sampled":
                q = torch.softmax(s["drafts"][b].double(), dim=1)
            else:
                q.scatter_(1, s["tokens"][b][:, None], 1.0)
            while n < length:
                d = int(s["tokens"][b, n])
                if not float(s["uniform"][b, n]) * float(q[n, d]) < float(p[n, d]):
                    break
                n += 1
            rest = p[n]
            if n < length and float((p[n] - q[n]).max()) > 0:
                rest = (p[n] - q[n]).clamp_min(0)
            last = int((rest / s["noise"][b].double()).argmax())
        accepted.append(n)
        tokens.append([int(t) for t in s["tokens"][b, :n]] + [last] + [-1] * (case["G"] - n))
    return {"accepted": torch.tensor(accepted, dtype=torch.int32), "tokens": torch.tensor(tokens)}
