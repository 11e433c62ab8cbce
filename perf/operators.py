"""The operators of a 4-bit serving step, as cases to be timed: products of a few bf16 rows with MXFP4 weights
(`gemv`), a paged MXFP4 key/value cache that is quantized as it is written and read back (`cache`), and the attention of
one or more new tokens of every sequence over that cache (`attention`).

Where `own` is false, run() computes each in its plain form, from elementary torch operations in 32 bits; where it is
true, it makes the calls that a user makes of mxfp4_act_quantizer_amd.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _gemv(name, rows, n, k, out):
    return {"name": name, "op": "gemv", "rows": rows, "n": n, "k": k, "out": out}


def _cache(name, seqs, chunk, length, heads, dim, page, factors):
    return {"name": name, "op": "cache", "seqs": seqs, "chunk": chunk, "length": length, "heads": heads, "dim": dim,
            "page": page, "factors": factors}


def _attention(name, seqs, chunk, length, q_heads, heads, dim, page, window=0, sinks=0):
    return {"name": name, "op": "attention", "seqs": seqs, "chunk": chunk, "length": length, "q_heads": q_heads,
            "heads": heads, "dim": dim, "page": page, "window": window, "sinks": sinks}


def listed():
    return [
        # one token through a linear of the narrowest DiT width: latency
        _gemv("gemv 1x1152x1152", 1, 1152, 1152, "bf16"),
        # the AdaLN modulation of two samples: six float32 shift/scale rows from one conditioning row each
        _gemv("gemv 2x6912x1152 f32", 2, 6912, 1152, "f32"),
        # a few tokens of a serving batch, a width that is no multiple of 128
        _gemv("gemv 13x8960x2240", 13, 8960, 2240, "bf16"),
        # one token through the widest linear: 320 MB of weights
        _gemv("gemv 1x49152x12288", 1, 49152, 12288, "bf16"),
        # a full serving batch of tokens
        _gemv("gemv 64x12288x4608", 64, 12288, 4608, "bf16"),
        # one new token of each of 61 sequences, written and read back
        _cache("cache 61 tokens", 61, 1, 4096, 8, 128, 16, False),
        # prompts of three lengths, the keys rotated by the per-block Kronecker transform on their way in
        _cache("cache prompts rotated", 3, 4099, 4099, 8, 128, 64, True),
        # one sequence, one new token: latency
        _attention("attention 1 token", 1, 1, 1001, 32, 8, 128, 16),
        # a serving batch: one new token of each of 48 sequences of lengths up to 16 K
        _attention("attention 48 tokens", 48, 1, 16384, 32, 8, 128, 16),
        # a chunk of a long prompt over what is cached of it
        _attention("attention chunk", 1, 2048, 16384, 32, 8, 128, 64),
        # ragged chunks, no shared heads, narrow heads
        _attention("attention ragged", 12, 257, 5001, 16, 16, 64, 32),
        # long sequences seen through a window and a few first tokens, wide heads
        _attention("attention window", 8, 5, 65537, 16, 4, 256, 128, 4096, 4),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("gemv", "gemv", "cache", "attention", "attention"))
    if op == "gemv":
        n, k = _spread(rng, 33, 49152), 32 * _spread(rng, 4, 384)
        case = _gemv("", _spread(rng, 1, 64), n, k, rng.choice(("bf16", "f32")))
    elif op == "cache":
        chunk = _spread(rng, 1, 4099)
        case = _cache("", _spread(rng, 1, max(1, min(61, 8192 // chunk))), chunk, chunk + rng.randrange(0, 2000),
                      rng.choice((1, 2, 4, 8)), rng.choice((32, 64, 96, 128, 256)), 16 * rng.randrange(1, 17),
                      rng.random() < 0.5)
    else:
        chunk = 1 if rng.random() < 0.5 else _spread(rng, 2, 1024)
        length = chunk + _spread(rng, 1, 16384)
        heads, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 256))
        group = rng.choice((1, 2, 4, 8) if dim == 256 else (1, 3, 4, 8, 16))
        # no more work, and no more cached values, than the largest listed cases have
        chunk = max(1, min(chunk, (1 << 36) // (length * heads * group * dim)))
        most = min((1 << 36) // (chunk * length * heads * group * dim), (1 << 28) // (length * heads * dim))
        seqs = _spread(rng, 1, max(1, min(48, most)))
        window = rng.choice((0, 0, _spread(rng, 16, 8192)))
        case = _attention("", seqs, chunk, length, heads * group, heads, dim, 16 * rng.randrange(1, 17), window,
                          rng.choice((0, 1, 4, 33)) if window else 0)
    del case["name"]
    return case


def _lengths(case):
    """(new rows, length) of every sequence: the largest first, the others down to about a fourth, odd ones among them."""
    n = case["seqs"]
    out = []
    for i in range(n):
        rows = max(1, case["chunk"] - (case["chunk"] * 3 * i) // (4 * n))
        out.append((rows, max(rows, case["length"] - (case["length"] * 3 * i) // (4 * n))))
    return out


def _pairs(case):
    """(visible pairs, cached positions that some row sees) over all sequences."""
    w, sinks = case["window"], case["sinks"]
    pairs = seen = 0
    for rows, length in _lengths(case):
        first = length - rows
        if not w:
            pairs += rows * first + rows * (rows + 1) // 2
            seen += length
            continue
        for p in range(first, length):
            pairs += min(p + 1, w) + min(sinks, max(0, p + 1 - w))
        lo = max(0, first + 1 - w)
        seen += length - lo + min(sinks, lo)
    return pairs, seen


def work(case):
    if case["op"] == "gemv":
        m, n, k = case["rows"], case["n"], case["k"]
        return {"bytes": n * k // 2 + n * k // 32 + 2 * m * k + m * n * (4 if case["out"] == "f32" else 2),
                "flops": 2 * m * n * k}
    values = case["heads"] * case["dim"]
    rows = sum(r for r, _ in _lengths(case))
    if case["op"] == "cache":
        # keys and values: bf16 in, codes and scales out, codes and scales in, bf16 out
        return {"bytes": 2 * rows * values * 4 + 4 * rows * values * 17 // 32,
                "flops": 2 * rows * values * (12 if case["factors"] else 2)}
    pairs, seen = _pairs(case)
    return {"bytes": 2 * 2 * rows * case["q_heads"] * case["dim"] + 2 * seen * values * 17 // 32,
            "flops": 4 * case["dim"] * case["q_heads"] * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _mx_random(gen, shape):
    """Codes (two a byte) and scales of normal values: whole blocks drawn from a pool of quantized ones."""
    pool = torch.randn((1 << 14, 1, 32), generator=gen, device=DEV)
    pool = pool * torch.exp(0.5 * torch.randn((1 << 14, 1, 1), generator=gen, device=DEV))
    codes, scales = _quantize(pool)
    pick = torch.randint(0, 1 << 14, (math.prod(shape),), generator=gen, device=DEV)
    return codes.view(-1, 16)[pick].view(*shape, 16), scales.view(-1)[pick].view(shape)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "gemv":
        m, n, k = case["rows"], case["n"], case["k"]
        x = torch.randn((m, k), generator=gen, device=DEV)
        x[:, :: max(1, k // 12)] *= 30.0  # a few outlier channels
        codes, scales = _mx_random(gen, (n, k // 32))
        return {"case": case, "x": x.bfloat16(), "qw": codes.reshape(n, k // 2), "sw": scales}

    pairs, page, dim, heads = _lengths(case), case["page"], case["dim"], case["heads"]
    seqs, rows = len(pairs), sum(r for r, _ in pairs)
    width = max(-(-length // page) for _, length in pairs)
    used = [-(-length // page) for _, length in pairs]
    pages = sum(used) + 1
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((seqs, width), dtype=torch.int32, device=DEV)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
    start = [0]
    for r, _ in pairs:
        start.append(start[-1] + r)
    state = {"case": case, "page_table": table,
             "row_start": torch.tensor(start, dtype=torch.int32, device=DEV),
             "lengths": torch.tensor([n for _, n in pairs], dtype=torch.int32, device=DEV)}
    for name in "kv":
        codes, scales = _mx_random(gen, (pages, heads, page, dim // 32))
        state[name + "q"] = codes.reshape(pages, heads, page, dim // 2)
        state[name + "s"] = scales.transpose(2, 3).contiguous()
    if case["op"] == "attention":
        q = torch.randn((rows, case["q_heads"], dim), generator=gen, device=DEV) * 1.5
        return state | {"q": q.bfloat16()}
    # keys and values are slices of one fused projection's output
    kv = torch.randn((rows, 2, heads, dim), generator=gen, device=DEV)
    kv[:, :, :, :: max(1, dim // 3)] *= 8.0
    kv = kv.bfloat16()
    state |= {"k": kv[:, 0], "v": kv[:, 1], "factors": None}
    if case["factors"]:
        # a set of five 2x2 factors for each block of 32 channels, near the identity
        eye = torch.eye(2, device=DEV)
        state["factors"] = eye + 0.2 * torch.randn((heads * dim // 32, 5, 2, 2), generator=gen, device=DEV)
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        import mxfp4_act_quantizer_amd as kq

        if op == "gemv":
            return kq.mx_gemv(state["x"], state["qw"], state["sw"], out_dtype=_out_dtype(state["case"]))
        cache = kq.MXCache(state["kq"], state["ks"], state["vq"], state["vs"])
        batch = (state["page_table"], state["row_start"], state["lengths"])
        if op == "cache":
            kq.mx_cache_write(state["k"], state["v"], cache, *batch, factors=state["factors"])
            return kq.mx_cache_read(cache, *batch, rows=state["k"].shape[0])
        return kq.mx_cache_attention(state["q"], cache, *batch, window=state["case"]["window"],
                                     sinks=state["case"]["sinks"])
    return {"gemv": _run_gemv, "cache": _run_cache, "attention": _run_attention}[op](state)


def _out_dtype(case):
    return torch.float32 if case["out"] == "f32" else torch.bfloat16


def _quantize(y):
    """MXFP4 of float32 [..., 32 b] values: packed codes [..., 16 b] and E8M0 bytes [..., b]."""
    y = y.unflatten(-1, (-1, 32))
    _, e = torch.frexp(y.abs().amax(-1, keepdim=True))
    zero = (y == 0).all(-1, keepdim=True)
    e = torch.where(zero, -127, (e - 3).clamp(min=-127))
    a = torch.ldexp(y.abs(), -e)
    # nearest on {0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even code
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * (y < 0)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _values(codes, scales):
    """float32 values [..., 32 b] of packed codes [..., 16 b] and scales [..., b]."""
    table = torch.tensor(E2M1, device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(scales.float() - 127.0).unsqueeze(-1)).flatten(-2)


def _run_gemv(state):
    w = _values(state["qw"], state["sw"])
    return (state["x"].float() @ w.t()).to(_out_dtype(state["case"]))


def _slots(state, rows):
    """Page and offset of every row: the rows of a sequence are its last positions."""
    start, page = state["row_start"].long(), state["case"]["page"]
    r = torch.arange(rows, device=start.device)
    seq = torch.searchsorted(start[1:], r, right=True)
    pos = state["lengths"].long()[seq] - start[seq + 1] + r
    return state["page_table"][seq, pos // page].long(), pos % page, seq, pos


def _run_cache(state):
    case, f = state["case"], state["factors"]
    page, off, _, _ = _slots(state, state["k"].shape[0])
    k, v = state["k"].float(), state["v"].float()
    if f is not None:
        # y = x (A1 x A2 x A3 x A4 x A5) of each block of 32
        m = f[:, 0]
        m = (m[:, :, None, :, None] * f[:, 1][:, None, :, None, :]).reshape(-1, 4, 4)
        m = (m[:, :, None, :, None] * f[:, 2][:, None, :, None, :]).reshape(-1, 8, 8)
        m = (m[:, :, None, :, None] * f[:, 3][:, None, :, None, :]).reshape(-1, 16, 16)
        m = (m[:, :, None, :, None] * f[:, 4][:, None, :, None, :]).reshape(-1, 32, 32)
        blocks = k.reshape(k.shape[0], -1, 32).transpose(0, 1).contiguous()
        k = torch.matmul(blocks, m).transpose(0, 1).reshape(k.shape)
    out = []
    for name, x in (("k", k), ("v", v)):
        codes, scales = state[name + "q"], state[name + "s"]
        codes[page, :, off], scales[page, :, :, off] = _quantize(x)
        out.append(_values(codes[page, :, off], scales[page, :, :, off]).bfloat16())
    return tuple(out)


def _run_attention(state):
    case, q = state["case"], state["q"]
    seqs, dim, heads, size = case["seqs"], case["dim"], case["heads"], case["page"]
    group = case["q_heads"] // heads
    start, lengths = state["row_start"].long(), state["lengths"].long()
    _, _, seq, pos = _slots(state, q.shape[0])
    table = state["page_table"].long()
    span = table.shape[1] * size

    def gathered(codes, scales):
        codes = codes[table].transpose(1, 2).reshape(seqs, heads, span, dim // 2)
        scales = scales[table].permute(0, 2, 1, 4, 3).reshape(seqs, heads, span, dim // 32)
        return _values(codes, scales)

    # rows padded to the longest chunk: [seqs, heads, chunk * group, dim]
    local = torch.arange(q.shape[0], device=q.device) - start[seq]
    padded = torch.zeros((seqs, case["chunk"], heads, group, dim), device=q.device)
    padded[seq, local] = q.float().view(-1, heads, group, dim)
    padded = padded.transpose(1, 2).reshape(seqs, heads, -1, dim)
    s = torch.matmul(padded, gathered(state["kq"], state["ks"]).transpose(2, 3)) * dim ** -0.5
    j = torch.arange(span, device=q.device)
    p = (lengths - (start[1:] - start[:-1]))[:, None] + torch.arange(case["chunk"], device=q.device)
    seen = (j <= p[..., None]) & (j < lengths[:, None, None])
    if case["window"]:
        seen &= (p[..., None] - j < case["window"]) | (j < case["sinks"])
    s = s.view(seqs, heads, -1, group, span).masked_fill_(~seen[:, None, :, None], -math.inf)
    s = s.view(seqs, heads, -1, span)
    # rows past a shorter chunk may see nothing: they are not read
    s = torch.exp(s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)))
    s = s.div_(s.sum(-1, keepdim=True))
    o = torch.matmul(s, gathered(state["vq"], state["vs"]))
    o = o.view(seqs, heads, -1, group, dim).transpose(1, 2)
    return o[seq, local].reshape(q.shape).bfloat16()


# ---------------------------------------------------------------------------
# 64 bits, from the definition
# ---------------------------------------------------------------------------
def _grid(codes, scales):
    """float64 values from the bits: sign, two exponent bits, one mantissa bit, and the scale's power of two."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2(e.double() - 1.0))
    power = torch.exp2(scales.double() - 127.0).repeat_interleave(32, -1)
    return torch.where(c >= 8, -mag, mag) * power


def _exact_mx(x):
    """The float64 values that MXFP4 gives float64 [..., 32 b] values."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))), torch.zeros_like(top))
    # log2 next to a power of two may land on either side of it
    e = torch.where(torch.exp2(e) > top, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= top, e + 1, e)
    unit = torch.exp2((e - 2).clamp(min=-127.0))
    a = (b / unit).abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).double()
    return (torch.sign(b) * torch.round(a / step) * step * unit).flatten(-2)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "gemv":
        x, parts = state["x"].double(), []
        for i in range(0, case["n"], 4096):
            parts.append(x @ _grid(state["qw"][i:i + 4096], state["sw"][i:i + 4096]).t())
        return torch.cat(parts, 1)
    if case["op"] == "cache":
        k, v = state["k"].double(), state["v"].double()
        if state["factors"] is not None:
            f = state["factors"].double()
            n = f.shape[0]
            y = k.reshape(-1, n, 2, 2, 2, 2, 2)
            # one factor at a time on its own axis of the block's five two-valued indices
            for i in range(5):
                y = y.movedim(2 + i, -1)
                shape = y.shape
                y = (y.reshape(shape[0], n, -1, 2, 1) * f[:, i][None, :, None]).sum(-2).reshape(shape)
                y = y.movedim(-1, 2 + i)
            k = y.reshape(k.shape)
        return tuple(_exact_mx(t) for t in (k, v))
    q, dim, heads = state["q"].double(), case["dim"], case["heads"]
    group = case["q_heads"] // heads
    out, at = torch.empty_like(q), 0
    for i, (rows, length) in enumerate(_lengths(case)):
        pos = torch.arange(length, device=q.device)
        page, off = state["page_table"][i, pos // case["page"]].long(), pos % case["page"]
        p = torch.arange(length - rows, length, device=q.device)[:, None]
        hidden = pos > p
        if case["window"]:
            hidden |= (p - pos >= case["window"]) & (pos >= case["sinks"])
        for h in range(heads):
            k = _grid(state["kq"][page, h, off], state["ks"][page, h, :, off])
            v = _grid(state["vq"][page, h, off], state["vs"][page, h, :, off])
            for g in range(h * group, (h + 1) * group):
                s = (q[at:at + rows, g] @ k.t()) / math.sqrt(dim)
                out[at:at + rows, g] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v
        at += rows
    return out
