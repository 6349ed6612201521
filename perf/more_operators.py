"""Measured cases of the operators around a paged 4-bit (MXFP4) key-value cache.

``run`` computes an operator either in its plain form (elementary torch
operations in 32 or 64 bits) or, with ``own`` set, through this package's
public entry points.  ``exact`` evaluates the operator's definition in 64 bits
by another route.  Operators:

    tables     block tables, slots and positions of new tokens, from the requests'
               lengths, their counts of new tokens and a stack of free pages
    rotary     queries and keys turned by their positions, with the gradients
    append     keys and values into their slots of the cache as MXFP4, and back;
               the outputs are the BF16 values that codes and scales stand for
    attention  of queries over the cache, each at its place in its sequence

A page holds ``page`` tokens.  For each page and key-value head the cache has, in
this order: the keys' codes [page][D / 2], the values' codes [page / 4][D / 8]
[4 tokens][4 bytes], the keys' scale bytes [page][D / 32], the values' [D / 32]
[page].
"""

import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decoding step of 64 requests: a page now and then
        {"name": "tables-decode", "op": "tables", "requests": 64, "new": 1, "past": 4096, "page": 16, "ragged": False},
        # many prompts admitted at once, of every length
        {"name": "tables-prompts", "op": "tables", "requests": 509, "new": 2048, "past": 1024, "page": 32, "ragged": True},
        # one token each of 32 sequences far along, frequencies stretched for a long context, half of the head turned
        {"name": "rotary-decode", "op": "rotary", "tokens": 32, "heads": 32, "kv_heads": 8, "head_dim": 128, "turned": 64,
         "interleaved": True, "farthest": 131072, "factor": 8.0, "dtype": "bfloat16", "backward": False},
        # a training step's queries and keys and their gradients
        {"name": "rotary-train", "op": "rotary", "tokens": 8192, "heads": 32, "kv_heads": 8, "head_dim": 128, "turned": 128,
         "interleaved": False, "farthest": 8192, "factor": 1.0, "dtype": "bfloat16", "backward": True},
        # one token each of 64 sequences
        {"name": "append-decode", "op": "append", "tokens": 64, "kv_heads": 8, "head_dim": 128, "page": 16, "padded": False},
        # a long prompt, odd token count, some rows padding
        {"name": "append-prompt", "op": "append", "tokens": 16381, "kv_heads": 8, "head_dim": 128, "page": 32, "padded": True},
        # a few short chats, one token each: latency
        {"name": "attention-short", "op": "attention", "sequences": 4, "queries": 1, "context": 301, "heads": 16, "kv_heads": 4,
         "head_dim": 64, "page": 16, "window": 0, "ragged": False, "lse": False},
        # one decoding step of 64 sequences of every length up to 8192
        {"name": "attention-decode", "op": "attention", "sequences": 64, "queries": 1, "context": 8192, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 16, "window": 0, "ragged": False, "lse": False},
        # one token of one very long sequence
        {"name": "attention-long", "op": "attention", "sequences": 1, "queries": 1, "context": 131071, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 64, "window": 0, "ragged": False, "lse": False},
        # drafted tokens checked at once, wide heads, a sliding window
        {"name": "attention-draft", "op": "attention", "sequences": 16, "queries": 5, "context": 16384, "heads": 16,
         "kv_heads": 8, "head_dim": 256, "page": 32, "window": 4096, "ragged": True, "lse": False},
        # prompts of every length up to 4096 behind a common history or none
        {"name": "attention-prompts", "op": "attention", "sequences": 4, "queries": 4096, "context": 4608, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 16, "window": 0, "ragged": True, "lse": False},
        # a piece of 500 tokens at the end of a long document, to be joined with another piece's softmax
        {"name": "attention-piece", "op": "attention", "sequences": 1, "queries": 500, "context": 49152, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 64, "window": 0, "ragged": False, "lse": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tables", "rotary", "append", "attention", "attention"))
    if op == "tables":
        case = {"op": op, "requests": _log_int(rng, 1, 1024), "new": rng.choice((1, _log_int(rng, 2, 4096))),
                "past": _log_int(rng, 1, 16384), "page": rng.choice((16, 32, 64, 128)), "ragged": rng.random() < 0.7}
        while case["requests"] * case["new"] > 509 * 2048:
            case["requests"] = max(1, case["requests"] // 2)
        return case
    head_dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8, 8, 5))
    if op == "rotary":
        case = {"op": op, "tokens": _log_int(rng, 1, 16384), "heads": kv_heads * rng.choice((1, 2, 4, 7)),
                "kv_heads": kv_heads, "head_dim": head_dim, "turned": head_dim // rng.choice((1, 1, 2, 4)),
                "interleaved": rng.random() < 0.5, "farthest": _log_int(rng, 64, 1 << 20),
                "factor": rng.choice((1.0, 4.0, 16.0)), "dtype": rng.choice(("bfloat16", "bfloat16", "float16", "float32")),
                "backward": rng.random() < 0.5}
        while case["tokens"] * (case["heads"] + kv_heads) * head_dim * (2 if case["dtype"] == "float32" else 1) > 8192 * 40 * 128:
            case["tokens"] = max(1, case["tokens"] // 2)
        return case
    page = rng.choice((16, 16, 32, 64, 128))
    if op == "append":
        tokens = _log_int(rng, 1, 32768)
        while tokens * kv_heads * head_dim > 16381 * 8 * 128:
            tokens = max(1, tokens // 2)
        return {"op": op, "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
                "padded": rng.random() < 0.5}
    kind = rng.choice(("decode", "decode", "draft", "prompt"))
    queries = 1 if kind == "decode" else _log_int(rng, 2, 12) if kind == "draft" else _log_int(rng, 13, 4096)
    case = {"op": op, "sequences": _log_int(rng, 1, 128), "queries": queries, "context": max(queries, _log_int(rng, 16, 65536)),
            "heads": kv_heads * rng.choice((1, 2, 4, 8, 7)), "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "window": rng.choice((0, 0, 0, _log_int(rng, 32, 4096))), "ragged": kind != "decode" and rng.random() < 0.7,
            "lse": rng.random() < 0.3}
    # no more keys than the largest decoding step, no more scores than the longest piece
    while (case["sequences"] * case["context"] * kv_heads * head_dim > 64 * 8192 * 8 * 128
           or case["sequences"] * case["heads"] * case["queries"] * case["context"] * head_dim > 32 * 500 * 49152 * 128):
        if case["sequences"] > 1:
            case["sequences"] //= 2
        else:
            case["context"] = max(1, case["context"] // 2)
            case["queries"] = min(case["queries"], case["context"])
    return case


# ----------------------------------------------------------------- inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _shares(n, step, least):
    """n fractions between least and 1, the first of them 1, spread evenly."""
    return [1 - (1 - least) * ((i * step) % 1.0) for i in range(n)]


def _counts(case):
    """(tokens in the cache with the new ones, new tokens) of each request, the same for every seed."""
    n = case["requests"] if case["op"] == "tables" else case["sequences"]
    most, longest = case["new" if case["op"] == "tables" else "queries"], case["past" if case["op"] == "tables" else "context"]
    new = [max(1, round(most * f)) if case["ragged"] else most for f in _shares(n, math.sqrt(2) - 1, 0.1)]
    total = [max(1, round(longest * f)) for f in _shares(n, (math.sqrt(5) - 1) / 2, 0.25)]
    if case["op"] == "tables":
        return [t + m for t, m in zip(total, new)], new
    return [max(t, m) for t, m in zip(total, new)], new


def _encode(x):
    """E2M1 codes uint8 [.., D / 2] and E8M0 scale bytes uint8 [.., D / 32] along the last axis."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    exponent = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(min=-127)
    b = torch.ldexp(b, -exponent)
    v = b.abs()
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    v = torch.clamp(torch.round(v / step) * step, max=6.0)
    code = torch.where(v < 2, v * 2, torch.where(v < 4, v + 2, v / 2 + 4)).to(torch.uint8) + 8 * torch.signbit(b).to(torch.uint8)
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] + 16 * code[..., 1], (exponent[..., 0] + 127).to(torch.uint8)


def _cache(k, v):
    """Pages of keys and values [pages, kv heads, page, D] as the cache's bytes."""
    (kc, ks), (vc, vs) = _encode(k), _encode(v)
    vc = vc.unflatten(3, (-1, 4)).unflatten(2, (-1, 4)).transpose(3, 4)
    return torch.cat((kc.flatten(2), vc.flatten(2), ks.flatten(2), vs.transpose(2, 3).flatten(2)), 2)


def _frequencies(case):
    """Turns per position of each pair, the slow ones stretched by the factor, the fast ones kept."""
    n = case["turned"] // 2
    turns = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n) / (2 * math.pi)
    rounds = turns * 4096
    keep = ((rounds - 1) / (32 - 1)).clamp(0, 1)
    return (turns * keep + turns / case["factor"] * (1 - keep)).to(_device())


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev) * std

    def i32(values):
        return torch.tensor(values, dtype=torch.int32).to(dev)

    s = dict(case)
    op = case["op"]
    if op in ("tables", "attention"):
        total, new = _counts(case)
        order = torch.randperm(len(total), generator=host).tolist()
        total, new = [total[i] for i in order], [new[i] for i in order]
        page = case["page"]
        held = [-(-(t - m if op == "tables" else t) // page) for t, m in zip(total, new)]
        width = max(-(-t // page) for t in total) + 1
        pages = sum(-(-t // page) for t in total) + 3
        shuffled = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        starts = torch.tensor([0] + held).cumsum(0)[:-1].to(dev)
        column = torch.arange(width, device=dev)
        inside = column < torch.tensor(held, device=dev)[:, None]
        s["table"] = torch.where(inside, shuffled[(starts[:, None] + column).clamp(max=pages - 1)], -1)
    if op == "tables":
        s["free"] = torch.cat((shuffled[sum(held):], torch.full((sum(held),), -1, dtype=torch.int32, device=dev)))
        s["free_count"] = i32([pages - sum(held)])
        s["lengths"], s["counts"], s["tokens"] = i32([t - m for t, m in zip(total, new)]), i32(new), sum(new)
    elif op == "rotary":
        dtype = getattr(torch, case["dtype"])
        t, d, back = case["tokens"], case["head_dim"], case["backward"]
        s["q"] = normal(t, case["heads"], d).to(dtype).requires_grad_(back)
        s["k"] = normal(t, case["kv_heads"], d).to(dtype).requires_grad_(back)
        s["dq"], s["dk"] = normal(t, case["heads"], d).to(dtype), normal(t, case["kv_heads"], d).to(dtype)
        s["positions"] = torch.randint(0, case["farthest"], (t,), generator=g, device=dev, dtype=torch.int32)
        s["turns"] = _frequencies(case)
        s["magnitude"] = 1 + 0.1 * math.log(case["factor"])
    elif op == "append":
        t, d, page = case["tokens"], case["head_dim"], case["page"]
        # keys have some dimensions of larger spread
        spread = torch.exp2(torch.randint(-1, 3, (case["kv_heads"], d), generator=g, device=dev).float())
        s["k"] = (normal(t, case["kv_heads"], d) * spread).bfloat16()
        s["v"] = normal(t, case["kv_heads"], d).bfloat16()
        pages = -(-t // page) + 2
        s["cache"] = torch.zeros((pages, case["kv_heads"], page * (d + d // 16)), dtype=torch.uint8, device=dev)
        at = torch.randperm(pages, generator=g, device=dev).repeat_interleave(page) * page
        slots = at[:t] + torch.arange(t, device=dev) % page
        if case["padded"]:
            slots = torch.where(torch.arange(t, device=dev) % 17 == 16, -1, slots)
        s["slots"] = slots.to(torch.int32)
    else:
        d = case["head_dim"]
        k, v = (normal(pages, case["kv_heads"], page, d).bfloat16() for _ in range(2))
        s["cache"] = _cache(k, v)
        s["q"] = normal(sum(new), case["heads"], d).bfloat16()
        s["lengths"] = i32(total)
        s["offsets"] = None if case["queries"] == 1 else i32([0] + new).cumsum(0).to(torch.int32)
        s["scale"] = d ** -0.5
    return s


# ------------------------------------------------------------ plain forms

def _plain_tables(s):
    page, table, tokens = s["page"], s["table"], s["tokens"]
    count, new = s["lengths"].long(), s["counts"].long()
    held, need = (count + page - 1) // page, (count + new + page - 1) // page
    taken = (need - held).cumsum(0)
    column = torch.arange(table.shape[1], device=table.device)
    at = s["free_count"].long() - 1 - ((taken - need)[:, None] + column)
    fresh = (column >= held[:, None]) & (column < need[:, None])
    table.copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1)], table))
    offsets = torch.cat((new.new_zeros(1), new.cumsum(0)))
    row = torch.arange(tokens, device=table.device)
    request = torch.zeros(tokens + 1, dtype=torch.long, device=table.device).index_add_(0, offsets[1:], torch.ones_like(new)).cumsum(0)[:tokens]
    position = count[request] + row - offsets[request]
    slot = table[request, position // page].long() * page + position % page
    return table, offsets.int(), (count + new).int(), slot.int(), position.int(), (s["free_count"] - taken[-1:]).int()


def _turned(x, cos, sin, s):
    n = s["turned"]
    y = x.float()
    a, b = (y[..., :n:2], y[..., 1:n:2]) if s["interleaved"] else (y[..., :n // 2], y[..., n // 2:n])
    c, d = (a * cos - b * sin) * s["magnitude"], (a * sin + b * cos) * s["magnitude"]
    both = torch.stack((c, d), -1).flatten(-2) if s["interleaved"] else torch.cat((c, d), -1)
    return torch.cat((both, y[..., n:]), -1).to(x.dtype)


def _plain_rotary(s):
    angle = 2 * math.pi * s["positions"].double()[:, None, None] * s["turns"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = _turned(s["q"].detach(), cos, sin, s), _turned(s["k"].detach(), cos, sin, s)
    return out + (_turned(s["dq"], cos, -sin, s), _turned(s["dk"], cos, -sin, s)) if s["backward"] else out


def _values(x):
    """The BF16 values of the MXFP4 copy of x along its last axis."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    exponent = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(min=-127)
    scale = torch.ldexp(torch.ones_like(amax), exponent)
    v = (b / scale).abs()
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    v = torch.clamp(torch.round(v / step) * step, max=6.0)
    return torch.copysign(v * scale, b).flatten(-2).bfloat16()


def _plain_append(s):
    kept = (s["slots"] >= 0)[:, None, None]
    return tuple(torch.where(kept, _values(x), torch.zeros_like(x)) for x in (s["k"], s["v"]))


def _decoded(codes, scales):
    """fp32 values [.., D] of codes [.., D / 2] and scale bytes [.., D / 32]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2).unflatten(-1, (-1, 32))
    return (v * torch.exp2(scales.float() - 127)[..., None]).flatten(-2)


def _unpacked(pages, page, d):
    """(key codes, key scales, value codes, value scales) of the cache's bytes [.., kv heads, record], token by token."""
    half, bytes_ = page * d // 2, page * d // 32
    kc, vc, ks, vs = pages.split((half, half, bytes_, bytes_), -1)
    vc = vc.unflatten(-1, (page // 4, d // 8, 4, 4)).transpose(-3, -2).flatten(-2).flatten(-3, -2)
    return kc.unflatten(-1, (page, -1)), ks.unflatten(-1, (page, -1)), vc, vs.unflatten(-1, (-1, page)).transpose(-1, -2)


def _plain_attention(s):
    q, page, d, hkv = s["q"], s["page"], s["head_dim"], s["kv_heads"]
    dev, (t, heads), length = q.device, q.shape[:2], s["lengths"].long()
    b, r = length.numel(), heads // hkv
    offsets = torch.arange(b + 1, device=dev) if s["offsets"] is None else s["offsets"].long()
    new, most = offsets[1:] - offsets[:-1], s["queries"]
    kc, ks, vc, vs = (x.transpose(1, 2).flatten(2, 3) for x in _unpacked(s["cache"][s["table"].long().clamp(min=0)], page, d))
    k, v = _decoded(kc, ks), _decoded(vc, vs)                     # [B, kv heads, keys, D]
    row = torch.arange(most, device=dev)
    rows = q[(offsets[:-1, None] + row).clamp(max=t - 1)].float()   # padded: [B, most, heads, D]
    rows = rows.unflatten(2, (hkv, r)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = torch.matmul(rows, k.transpose(2, 3)).mul_(s["scale"]).unflatten(2, (most, r))
    at = (length - new)[:, None] + row                            # place of each query
    key = torch.arange(k.shape[2], device=dev)
    hidden = key > at[..., None]
    if s["window"]:
        hidden |= key <= at[..., None] - s["window"]
    score.masked_fill_(hidden[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (most, r)) / total.clamp(min=1e-30)
    sequence = (torch.arange(t, device=dev)[:, None] >= offsets[1:]).sum(1)
    inside = torch.arange(t, device=dev) - offsets[sequence]
    out = out[sequence, :, inside].flatten(1, 2).bfloat16()
    return (out, (top + torch.log(total))[..., 0][sequence, :, inside].flatten(1)) if s["lse"] else out


def run(state):
    if own:
        return _run_own(state)
    return {"tables": _plain_tables, "rotary": _plain_rotary, "append": _plain_append,
            "attention": _plain_attention}[state["op"]](state)


def _run_own(s):
    from mxfp8_block_scaled_quantize_amd import kvcache, rotary

    op = s["op"]
    if op == "tables":
        plan = kvcache.extend(s["table"], s["lengths"], s["counts"], s["free"], s["free_count"], s["tokens"], s["page"])
        return s["table"], plan.offsets, plan.lengths, plan.slots, plan.positions, plan.free_count
    if op == "rotary":
        q, k = rotary.rotate(s["q"], s["k"], s["positions"], s["turns"], interleaved=s["interleaved"], magnitude=s["magnitude"])
        if not s["backward"]:
            return q, k
        return (q.detach(), k.detach(), *torch.autograd.grad((q, k), (s["q"], s["k"]), (s["dq"], s["dk"])))
    if op == "append":
        kvcache.append(s["cache"], s["k"], s["v"], s["slots"])
        return kvcache.read(s["cache"], s["slots"], s["head_dim"])
    return kvcache.attention(s["q"], s["cache"], s["table"], s["lengths"], s["offsets"], scale=s["scale"], window=s["window"],
                             max_queries=s["queries"], lse=s["lse"])


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "tables":
        total, new = _counts(case)
        fresh = sum(-(-t // case["page"]) - -(-(t - m) // case["page"]) for t, m in zip(total, new))
        # lengths, counts, offsets, free pages and their numbers; a slot and a position for each token
        return {"bytes": 16 * len(total) + 8 * fresh + 8 * sum(new), "flops": 0}
    if op == "rotary":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["head_dim"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": 2 * size * n * (2 if case["backward"] else 1) + 4 * case["tokens"], "flops": 0}
    if op == "append":
        n = 2 * case["tokens"] * case["kv_heads"] * case["head_dim"]
        return {"bytes": 2 * n + 2 * n + 4 * case["tokens"], "flops": 0}   # the input once, the values once
    total, new = _counts(case)
    window = case["window"] or 1 << 40
    keys = sum(t - max(0, t - m + 1 - window) for t, m in zip(total, new))
    pairs = sum(_visible(t, window) - _visible(t - m, window) for t, m in zip(total, new))
    d = case["head_dim"]
    return {"bytes": keys * case["kv_heads"] * (d + d // 16) + 4 * sum(new) * case["heads"] * d,
            "flops": 4 * pairs * case["heads"] * d}


def _visible(n, window):
    """Keys that the first n queries of a sequence see."""
    w = min(n, window)
    return w * (w + 1) // 2 + (n - w) * w


# ------------------------------------------------------------------ exact

def _exact_values(x):
    """Nearest of the eight magnitudes by the midpoints between them."""
    b = x.double().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(amax.clamp(min=2.0 ** -120))) - 2)
    table = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    middle = (table[1:] + table[:-1]) / 2
    v = b.abs() / scale
    up, down = torch.bucketize(v, middle, right=True), torch.bucketize(v, middle, right=False)
    index = torch.where(up % 2 == 0, up, down)      # they differ on a midpoint alone: the even code
    return torch.copysign(table[index] * scale, b).flatten(-2)


def _exact_decoded(codes, scales):
    """Values in 64 bits from the codes' bits: sign, two exponent bits, one mantissa bit."""
    n = torch.stack((codes % 16, codes // 16), -1).flatten(-2).unflatten(-1, (-1, 32)).to(torch.int16)
    exponent, mantissa = (n // 2) % 4, (n % 2).double() / 2
    v = torch.where(exponent == 0, mantissa, (1 + mantissa) * torch.exp2(exponent.double() - 1))
    v = torch.where(n >= 8, -v, v)
    return (v * torch.exp2(scales.double() - 127)[..., None]).flatten(-2)


def _exact_turned(x, angle, s, sign):
    n, y = s["turned"], x.double()
    pairs = y[..., :n].unflatten(-1, (-1, 2)) if s["interleaved"] else y[..., :n].unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, s["magnitude"]), sign * angle)
    pairs = torch.view_as_real(z)
    pairs = pairs if s["interleaved"] else pairs.transpose(-1, -2)
    return torch.cat((pairs.flatten(-2), y[..., n:]), -1)


def _exact_attention(s):
    page, d, hkv, heads = s["page"], s["head_dim"], s["kv_heads"], s["heads"]
    offsets = list(range(s["sequences"] + 1)) if s["offsets"] is None else s["offsets"].tolist()
    outs, sums = [], []
    for i, length in enumerate(s["lengths"].tolist()):
        n = offsets[i + 1] - offsets[i]
        first = max(0, length - n + 1 - s["window"]) // page if s["window"] else 0
        record = s["cache"][s["table"][i, first:-(-length // page)].long()]
        key = torch.arange(first * page, length, device=record.device)
        parts = [x.transpose(0, 1).flatten(1, 2)[:, :len(key)] for x in _unpacked(record, page, d)]
        for h in range(hkv):
            k, v = _exact_decoded(parts[0][h], parts[1][h]), _exact_decoded(parts[2][h], parts[3][h])
            q = s["q"][offsets[i]:offsets[i + 1], h * (heads // hkv):(h + 1) * (heads // hkv)].double()
            at = torch.arange(length - n, length, device=q.device)[:, None]
            bias = torch.zeros((n, len(key)), dtype=torch.float64, device=q.device)
            bias[key > at] = -math.inf
            if s["window"]:
                bias[key <= at - s["window"]] = -math.inf
            score = torch.matmul(q.transpose(0, 1), k.t()) * s["scale"] + bias      # [group, n, keys]
            total = torch.logsumexp(score, -1)
            outs.append(torch.matmul(torch.exp(score - total[..., None]), v).transpose(0, 1))
            sums.append(total.transpose(0, 1))
    by = [torch.cat(outs[i * hkv:(i + 1) * hkv], 1) for i in range(s["sequences"])]
    total = [torch.cat(sums[i * hkv:(i + 1) * hkv], 1) for i in range(s["sequences"])]
    return (torch.cat(by), torch.cat(total)) if s["lse"] else torch.cat(by)


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None                       # whole numbers alone
    s = prepare(case, seed)
    if op == "append":
        return tuple(_exact_values(x) * (s["slots"] >= 0)[:, None, None] for x in (s["k"], s["v"]))
    if op == "rotary":
        turns = torch.remainder(s["positions"].double()[:, None, None] * s["turns"], 1.0)
        out = [_exact_turned(s[x].detach(), 2 * math.pi * turns, s, 1) for x in ("q", "k")]
        return tuple(out + [_exact_turned(s[x], 2 * math.pi * turns, s, -1) for x in ("dq", "dk")] if case["backward"] else out)
    return _exact_attention(s)
