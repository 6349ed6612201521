"""Measured cases of the 4-bit (MXFP4) and mixture-of-experts operators.

``run`` computes an operator either in its plain form (elementary torch
operations in 32 or 64 bits) or, with ``own`` set, through this package's
public entry points.  ``exact`` evaluates the operator's definition in 64 bits
by another route.  Operators:

    quantize   BF16 -> MXFP4 (E2M1 codes, one E8M0 scale per 32 values), rowwise
               and, for training, the transposed columnwise copy; the outputs are
               the BF16 values that codes and scales stand for (every E2M1 value
               times a power of two is a BF16 value)
    gemm       C = bf16(dq(A) dq(B)^T) of MXFP4 operands
    grouped    the same per expert on ragged row ranges, optionally with the
               SwiGLU epilogue
    route      expert choice and weights from router logits, with the gradient
    dispatch   stable counting sort of the (token, slot) pairs by expert
    combine    weighted sum of the experts' outputs, with the gradients
"""

import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # activations of 32 sequences in front of a projection, one token each
        {"name": "quantize-decode", "op": "quantize", "rows": 32, "cols": 4096, "colwise": False},
        # a training step's activations: the copy for fprop and the one for wgrad
        {"name": "quantize-train", "op": "quantize", "rows": 8192, "cols": 4096, "colwise": True},
        # one token through an up projection: the weights are read once
        {"name": "gemm-one-token", "op": "gemm", "m": 1, "n": 14336, "k": 4096},
        # a training or prefill step's up projection
        {"name": "gemm-train", "op": "gemm", "m": 8192, "n": 14336, "k": 4096},
        # 37 tokens with 4 experts each: a few rows per expert, some experts without any
        {"name": "grouped-decode", "op": "grouped", "m": 148, "n": 1024, "k": 4096, "experts": 32, "swiglu": True},
        # prefill or training through 8 experts, ragged groups
        {"name": "grouped-prefill", "op": "grouped", "m": 16384, "n": 7168, "k": 4096, "experts": 8, "swiglu": True},
        # 16 tokens, many experts in 8 groups, balance bias
        {"name": "route-decode", "op": "route", "tokens": 16, "experts": 256, "top_k": 8, "scores": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renormalize": True, "dtype": "float32",
         "backward": False},
        # a training step's router: choice, weights and the gradient of the logits
        {"name": "route-train", "op": "route", "tokens": 16384, "experts": 128, "top_k": 8, "scores": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_top": 1, "renormalize": True, "dtype": "bfloat16",
         "backward": True},
        # one decoding step's slots
        {"name": "dispatch-decode", "op": "dispatch", "tokens": 16, "experts": 256, "top_k": 8},
        # a long prefill, odd token count
        {"name": "dispatch-prefill", "op": "dispatch", "tokens": 16383, "experts": 128, "top_k": 8},
        # one decoding step's outputs
        {"name": "combine-decode", "op": "combine", "tokens": 16, "top_k": 8, "hidden": 4096, "backward": False},
        # a training step: forward, gradients of the experts' outputs and of the weights
        {"name": "combine-train", "op": "combine", "tokens": 8191, "top_k": 8, "hidden": 4096, "backward": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    # 3072 is not among the sizes
    return {k: 2944 if v == 3072 else v for k, v in _draw(rng).items()}


def _draw(rng):
    op = rng.choice(("quantize", "gemm", "grouped", "route", "dispatch", "combine"))
    if op == "quantize":
        colwise = rng.random() < 0.5
        cols = 128 * _log_int(rng, 1, 64)
        rows = _log_int(rng, 1, 32768)
        if colwise:   # whole scale words along the rows too
            rows = 128 * max(1, rows // 128)
        while rows * cols > 8192 * 14336:
            rows = rows // 256 * 128 if colwise else rows // 2
        return {"op": op, "rows": rows, "cols": cols, "colwise": colwise}
    if op == "gemm":
        m, n, k = _log_int(rng, 1, 16384), 32 * _log_int(rng, 8, 512), 128 * _log_int(rng, 2, 64)
        while m * n * k > 8192 * 14336 * 4096:
            m //= 2
        return {"op": op, "m": m, "n": n, "k": k}
    if op == "grouped":
        experts = _log_int(rng, 2, 64)
        swiglu = rng.random() < 0.5
        m, n, k = _log_int(rng, 1, 16384), 32 * _log_int(rng, 8, 224), 128 * _log_int(rng, 2, 32)
        while experts * n * k > 8 * 7168 * 4096:
            n = 32 * max(1, n // 64)
        while m * n * k > 16384 * 7168 * 4096:
            m //= 2
        return {"op": op, "m": m, "n": n, "k": k, "experts": experts, "swiglu": swiglu}
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        experts = groups * _log_int(rng, max(2, 8 // groups), 384 // groups)
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(12, top_groups * (experts // groups)))
        return {"op": op, "tokens": _log_int(rng, 1, 32768), "experts": experts, "top_k": top_k,
                "scores": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5, "groups": groups,
                "top_groups": top_groups, "group_top": rng.choice((1, 2)), "renormalize": rng.random() < 0.7,
                "dtype": rng.choice(("float32", "bfloat16", "float16")), "backward": rng.random() < 0.5}
    experts = _log_int(rng, 4, 384)
    top_k = rng.randint(1, min(8, experts))
    if op == "dispatch":
        return {"op": op, "tokens": _log_int(rng, 1, 32768), "experts": experts, "top_k": top_k}
    tokens, hidden = _log_int(rng, 1, 16384), 8 * _log_int(rng, 32, 1024)
    while tokens * top_k * hidden > 8191 * 8 * 4096:
        tokens //= 2
    return {"op": op, "tokens": tokens, "top_k": top_k, "hidden": hidden, "backward": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _e2m1(v):
    """Nearest E2M1 value of |v| (ties to the even code), saturated at 6."""
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    return torch.clamp(torch.round(v / step) * step, max=6.0)


def _block_scale(x32):
    """2^X per block of 32 along the last axis, X = floor(log2 amax) - 2 >= -127."""
    amax = x32.abs().amax(-1, keepdim=True)
    exponent = torch.frexp(amax).exponent - 3
    exponent = torch.where(amax > 0, exponent, -127).clamp(min=-127)
    return exponent, torch.ldexp(torch.ones_like(amax), exponent)


def _values(x):
    """The BF16 values of the MXFP4 copy of x along its last axis."""
    r, c = x.shape
    b = x.float().view(r, c // 32, 32)
    _, scale = _block_scale(b)
    v = b / scale
    return torch.copysign(_e2m1(v.abs()) * scale, b).view(r, c).bfloat16()


def _encode(x):
    """Codes uint8 [R, C / 2] and packed scale words int32 [C / 128, R] of a matrix."""
    r, c = x.shape
    b = x.float().view(r, c // 32, 32)
    exponent, scale = _block_scale(b)
    mag = _e2m1((b / scale).abs())
    code = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(b).to(torch.uint8)).view(r, c // 2, 2)
    codes = code[..., 0] + 16 * code[..., 1]
    byte = (exponent + 127).to(torch.uint8).view(r, c // 128, 4)
    return codes.contiguous(), byte.view(torch.int32).view(r, c // 128).t().contiguous()


def _ragged(m, experts, gen):
    """Row counts of the experts: uneven, one in eight or so without rows."""
    share = torch.rand(experts, generator=gen) ** 2 + 0.02
    share[torch.rand(experts, generator=gen) < 0.125] = 0
    share[0] = share[0].clamp(min=0.1)
    cum = torch.round(torch.cumsum(share, 0) / share.sum() * m).long()
    cum[-1] = m
    return torch.diff(cum, prepend=torch.zeros(1, dtype=torch.long)).tolist()


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev) * std

    s = dict(case)
    op = case["op"]
    if op == "quantize":
        # activations: normal values, some channels with a larger spread
        spread = torch.exp2(torch.randint(-2, 3, (1, case["cols"]), generator=g, device=dev).float())
        s["x"] = (normal(case["rows"], case["cols"]) * spread).bfloat16()
    elif op == "gemm":
        s["a"], s["ap"] = _encode(normal(case["m"], case["k"]))
        s["b"], s["bp"] = _encode(normal(case["n"], case["k"], std=0.02))
    elif op == "grouped":
        rows = case["n"] * (2 if case["swiglu"] else 1)
        s["counts"] = _ragged(case["m"], case["experts"], host)
        s["offsets"] = torch.tensor([0] + s["counts"]).cumsum(0).to(torch.int32).to(dev)
        s["a"], s["ap"] = _encode(normal(case["m"], case["k"]))
        b, s["bp"] = _encode(normal(case["experts"] * rows, case["k"], std=0.02))
        s["b"] = b.view(case["experts"], rows, case["k"] // 2)
    elif op == "route":
        dtype = getattr(torch, case["dtype"])
        s["logits"] = normal(case["tokens"], case["experts"]).to(dtype).requires_grad_(case["backward"])
        s["balance"] = normal(case["experts"], std=0.05) if case["bias"] else None
        s["dweights"] = normal(case["tokens"], case["top_k"])
    elif op == "dispatch":
        # every token's experts are distinct; a popularity makes the groups uneven
        popular = normal(1, case["experts"], std=0.5)
        score = normal(case["tokens"], case["experts"]) + popular
        s["choice"] = score.topk(case["top_k"], dim=1).indices.to(torch.int32).contiguous()
    else:
        slots = case["tokens"] * case["top_k"]
        s["y"] = normal(slots, case["hidden"]).bfloat16().requires_grad_(case["backward"])
        s["position"] = torch.randperm(slots, generator=g, device=dev).to(torch.int32).view(-1, case["top_k"])
        s["w"] = torch.softmax(normal(case["tokens"], case["top_k"]), 1).requires_grad_(case["backward"])
        s["dout"] = normal(case["tokens"], case["hidden"]).bfloat16()
    return s


# ------------------------------------------------------------ plain forms

def _decode(codes, words):
    """fp32 values [R, K] of codes [R, K / 2] and packed words [K / 128, R]."""
    r = codes.shape[0]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).view(r, -1, 32)
    byte = words.t().contiguous().view(torch.uint8).view(r, -1, 1)
    return (v * torch.exp2(byte.float() - 127)).view(r, -1)


def _plain_grouped(s):
    b = _decode(s["b"].flatten(0, 1), s["bp"]).view(s["experts"], -1, s["k"])
    rows = torch.split(_decode(s["a"], s["ap"]), s["counts"])
    c = torch.cat([torch.matmul(x, w.t()) for x, w in zip(rows, b)])
    if s["swiglu"]:
        gate, up = c.chunk(2, 1)
        c = gate * torch.sigmoid(gate) * up
    return c.bfloat16()


def _plain_route(s):
    # 64 bits: two scores may lie closer than 32 bits can tell
    l = s["logits"].detach().double()
    t, e = l.shape
    score = torch.softmax(l, 1) if s["scores"] == "softmax" else torch.sigmoid(l)
    choice = score if s["balance"] is None else score + s["balance"].double()
    if s["groups"] > 1:
        best = choice.view(t, s["groups"], -1).sort(-1, descending=True).values[..., :s["group_top"]].sum(-1)
        keep = best.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        open_ = torch.zeros_like(best, dtype=torch.bool).scatter_(1, keep, True)
        choice = choice.masked_fill(~open_.repeat_interleave(e // s["groups"], 1), -math.inf)
    experts = choice.sort(dim=1, descending=True, stable=True).indices[:, :s["top_k"]]
    chosen = score.gather(1, experts)
    total = chosen.sum(1, keepdim=True) + 1e-20
    weights = chosen / total if s["renormalize"] else chosen
    if not s["backward"]:
        return weights.float(), experts.int()
    g = s["dweights"].double()
    if s["renormalize"]:
        g = (g - (g * weights).sum(1, keepdim=True)) / total
    d = torch.zeros_like(score).scatter_(1, experts, g)
    d = score * (d - (d * score).sum(1, keepdim=True)) if s["scores"] == "softmax" else d * score * (1 - score)
    return weights.float(), experts.int(), d.to(s["logits"].dtype)


def _plain_dispatch(s):
    flat = s["choice"].flatten()
    order = flat.sort(stable=True).indices
    position = torch.empty_like(flat)
    position[order] = torch.arange(flat.numel(), dtype=torch.int32, device=flat.device)
    count = (flat[:, None] == torch.arange(s["experts"], device=flat.device)).sum(0)
    offsets = torch.cat((count.new_zeros(1), count.cumsum(0)))
    return offsets.int(), (order // s["top_k"]).int(), position.view_as(s["choice"])


def _plain_combine(s):
    y, w, at = s["y"].detach(), s["w"].detach(), s["position"].long()
    rows = y[at].float()
    out = (rows * w[..., None]).sum(1).bfloat16()
    if not s["backward"]:
        return out
    g = s["dout"].float()[:, None]
    dy = torch.zeros_like(y)
    dy[at] = (g * w[..., None]).bfloat16()
    return out, dy, (g * rows).sum(-1)


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "quantize":
        return (_values(state["x"]), _values(state["x"].t().contiguous())) if state["colwise"] else _values(state["x"])
    if op == "gemm":
        return torch.matmul(_decode(state["a"], state["ap"]), _decode(state["b"], state["bp"]).t()).bfloat16()
    return {"grouped": _plain_grouped, "route": _plain_route, "dispatch": _plain_dispatch,
            "combine": _plain_combine}[op](state)


def _run_own(s):
    from mxfp8_block_scaled_quantize_amd import moe, mxfp4

    op = s["op"]
    if op == "quantize":
        q = mxfp4.quantize(s["x"], colwise=s["colwise"], packed=True)
        row = mxfp4.dequantize(q["q_row"], q["p_row"])
        return (row, mxfp4.dequantize(q["q_colT"], q["p_colT"])) if s["colwise"] else row
    if op == "gemm":
        return mxfp4.gemm(s["a"], s["ap"], s["b"], s["bp"])
    if op == "grouped":
        return mxfp4.grouped_gemm(s["a"], s["ap"], s["b"], s["bp"], s["offsets"], swiglu=s["swiglu"])
    if op == "route":
        weights, experts = moe.route(s["logits"], s["top_k"], scores=s["scores"], bias=s["balance"],
                                     groups=s["groups"], top_groups=s["top_groups"], group_top=s["group_top"],
                                     renormalize=s["renormalize"])
        if not s["backward"]:
            return weights, experts
        return weights.detach(), experts, torch.autograd.grad(weights, s["logits"], s["dweights"])[0]
    if op == "dispatch":
        return tuple(moe.dispatch(s["choice"], s["experts"]))
    out = moe.combine(s["y"], s["position"], s["w"])
    if not s["backward"]:
        return out
    return (out.detach(), *torch.autograd.grad(out, (s["y"], s["w"]), s["dout"]))


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "quantize":
        n, copies = case["rows"] * case["cols"], 2 if case["colwise"] else 1
        return {"bytes": 2 * n + copies * 2 * n, "flops": 0}   # the input once, each copy's values once
    if op in ("gemm", "grouped"):
        m, n, k = case["m"], case["n"], case["k"]
        rows = n * (2 if case.get("swiglu") else 1)
        # experts that can have rows at all
        b_rows = rows * min(case.get("experts", 1), m)
        return {"bytes": (m + b_rows) * k * 17 / 32 + 2 * m * n, "flops": 2 * m * rows * k}
    if op == "route":
        size = 4 if case["dtype"] == "float32" else 2
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        back = t * e * size + 4 * t * k if case["backward"] else 0
        return {"bytes": t * e * size + 8 * t * k + back, "flops": 0}
    if op == "dispatch":
        return {"bytes": 12 * case["tokens"] * case["top_k"] + 4 * (case["experts"] + 1), "flops": 0}
    t, k, h = case["tokens"], case["top_k"], case["hidden"]
    back = 2 * t * h + 2 * t * k * h + 4 * t * k if case["backward"] else 0
    return {"bytes": 2 * t * k * h + 8 * t * k + 2 * t * h + back, "flops": (6 if case["backward"] else 2) * t * k * h}


# ------------------------------------------------------------------ exact

def _exact_values(x):
    """Nearest of the eight magnitudes by the midpoints between them."""
    r, c = x.shape
    b = x.double().view(r, c // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(amax.clamp(min=2.0 ** -120))) - 2)
    table = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    middle = (table[1:] + table[:-1]) / 2
    v = b.abs() / scale
    up, down = torch.bucketize(v, middle, right=True), torch.bucketize(v, middle, right=False)
    index = torch.where(up % 2 == 0, up, down)      # they differ on a midpoint alone: the even code
    return torch.copysign(table[index] * scale, b).view(r, c)


def _exact_decode(codes, words):
    """Values in 64 bits from the codes' bits: sign, two exponent bits, one mantissa bit."""
    r = codes.shape[0]
    n = torch.stack((codes % 16, codes // 16), -1).view(r, -1, 32).to(torch.int16)
    exponent, mantissa = (n // 2) % 4, (n % 2).double() / 2
    v = torch.where(exponent == 0, mantissa, (1 + mantissa) * torch.exp2(exponent.double() - 1))
    v = torch.where(n >= 8, -v, v)
    byte = torch.stack([(words.t() >> sh) & 255 for sh in (0, 8, 16, 24)], -1).reshape(r, -1, 1)
    return (v * torch.exp2(byte.double() - 127)).view(r, -1)


def _exact_route(s):
    l = s["logits"].detach().double()
    t, e = l.shape
    if s["scores"] == "softmax":
        score = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    else:
        score = 1 / (1 + torch.exp(-l))
    left = score.clone() if s["balance"] is None else score + s["balance"].double()

    def first_best(v, n):
        v, picked, at = v.clone(), [], torch.arange(v.shape[1], device=v.device)
        for _ in range(n):
            top = v.amax(1, keepdim=True)
            i = torch.where(v == top, at, v.shape[1]).amin(1, keepdim=True)
            picked.append(i)
            v.scatter_(1, i, -math.inf)
        return torch.cat(picked, 1)

    if s["groups"] > 1:
        per = e // s["groups"]
        inside = left.view(-1, per)
        best = inside.gather(1, first_best(inside, min(s["group_top"], per))).sum(1).view(t, -1)
        shut = torch.ones_like(best, dtype=torch.bool).scatter_(1, first_best(best, s["top_groups"]), False)
        left = torch.where(shut[:, :, None], -math.inf, left.view(t, s["groups"], per)).view(t, e)
    experts = first_best(left, s["top_k"])
    picked = torch.zeros_like(score).scatter_(1, experts, 1.0)
    total = (score * picked).sum(1, keepdim=True) + 1e-20 if s["renormalize"] else torch.ones_like(score[:, :1])
    weights = (score / total).gather(1, experts)
    if not s["backward"]:
        return weights, None
    g = torch.zeros_like(score).scatter_(1, experts, s["dweights"].double())
    # dw_i / ds_j = [i = j] / total - (renormalize) s_i / total^2, i and j chosen
    ds = g / total
    if s["renormalize"]:
        ds = picked * (ds - (g * score).sum(1, keepdim=True) / total ** 2)
    if s["scores"] == "softmax":
        return weights, None, ds * score - score * (ds * score).sum(1, keepdim=True)
    return weights, None, ds * (score - score * score)


def exact(case, seed):
    op = case["op"]
    if op == "dispatch":
        return None                       # whole numbers alone
    s = prepare(case, seed)
    if op == "quantize":
        x = s["x"]
        return (_exact_values(x), _exact_values(x.t().contiguous())) if case["colwise"] else _exact_values(x)
    if op == "gemm":
        return _exact_decode(s["a"], s["ap"]) @ _exact_decode(s["b"], s["bp"]).t()
    if op == "grouped":
        a, start, parts = _exact_decode(s["a"], s["ap"]), 0, []
        rows = s["b"].shape[1]
        for e, count in enumerate(s["counts"]):
            b = _exact_decode(s["b"][e], s["bp"][:, e * rows:(e + 1) * rows])
            parts.append(a[start:start + count] @ b.t())
            start += count
        c = torch.cat(parts)
        if not case["swiglu"]:
            return c
        n = case["n"]
        return c[:, :n] / (1 + torch.exp(-c[:, :n])) * c[:, n:]
    if op == "route":
        return _exact_route(s)
    y, w = s["y"].detach().double(), s["w"].detach().double()
    t, k = w.shape
    slot = s["position"].flatten().long()
    out = torch.zeros(t, case["hidden"], dtype=torch.float64, device=y.device)
    dw, g = [], s["dout"].double()
    for j in range(k):
        rows = y[slot[j::k]]
        out += w[:, j:j + 1] * rows
        dw.append(torch.linalg.vecdot(g, rows))
    if not case["backward"]:
        return out
    dy = torch.zeros_like(y)
    dy.index_copy_(0, slot, (w.view(t, k, 1) * g.view(t, 1, -1)).view(t * k, -1))
    return out, dy, torch.stack(dw, 1)
