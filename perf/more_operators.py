"""The operators of the 4-bit key/value cache: appending rotated keys and
values to its pages, reading rows back, and attention over it, for single
tokens, drafts, prompts and chunks of prompts.

Each case is a dict of plain values.  run() computes it in elementary torch
operations (own = False) or through libq4 (own = True).  A cache row is D
values of one token and head in the affine 4-bit format: codes, low nibble
first, with an fp16 scale and an fp16 zero point per 64 values; the value is
(code - zero) * scale.  Rows stand as [pages][heads][page].
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # One request's next token: the latency of a decode step.
        dict(name="append-token", op="append", T=1, Hq=16, Hkv=2, D=128, page=16, rot=128, interleaved=False, f32=True),
        # A decode batch of an odd number of requests, half of each head rotated.
        dict(name="append-batch", op="append", T=61, Hq=40, Hkv=8, D=128, page=16, rot=64, interleaved=True, f32=False),
        # Prompts, written in one call.
        dict(name="append-prompt", op="append", T=8191, Hq=40, Hkv=8, D=128, page=64, rot=128, interleaved=False,
             f32=False),
        # A few rows of a cache with small heads.
        dict(name="read-rows", op="read", n=37, Hkv=12, D=64, page=32, f32=True),
        # A prefix as values, for a program that goes on with them elsewhere.
        dict(name="read-prefix", op="read", n=20000, Hkv=8, D=128, page=64, f32=False),
        # One request's decode step on a short context.
        dict(name="attend-token", op="attend", B=1, T=1, most=300, new=1, Hq=16, Hkv=2, D=128, page=16, window=0,
             lse=False),
        # A decode batch with ragged contexts.
        dict(name="attend-batch", op="attend", B=64, T=64, most=8192, new=1, Hq=40, Hkv=8, D=128, page=16, window=0,
             lse=False),
        # Two requests on long contexts: the work has to be split along the keys.
        dict(name="attend-long", op="attend", B=2, T=2, most=131072, new=1, Hq=40, Hkv=8, D=128, page=64, window=0,
             lse=True),
        # Drafts checked: up to five new tokens of each request, a sliding window, one query head a key head.
        dict(name="attend-draft", op="attend", B=24, T=71, most=4096, new=5, Hq=12, Hkv=12, D=64, page=32, window=1000,
             lse=False),
        # Large heads, few of them.
        dict(name="attend-wide", op="attend", B=16, T=16, most=6000, new=1, Hq=8, Hkv=4, D=256, page=128, window=0,
             lse=True),
        # Prompts of three requests without a prefix: compute bound.
        dict(name="attend-prompt", op="attend", B=3, T=8191, most=0, new=8191, Hq=16, Hkv=2, D=128, page=64, window=0,
             lse=False),
        # A chunk of a prompt behind a long prefix.
        dict(name="attend-chunk", op="attend", B=1, T=512, most=33000, new=512, Hq=40, Hkv=8, D=128, page=16, window=0,
             lse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        op = rng.choice(("append", "append", "read", "attend", "attend", "attend", "attend"))
        Hkv, D, page = rng.choice((1, 2, 3, 4, 8, 12)), rng.choice((64, 128, 128, 192, 256)), rng.choice((16, 32, 64, 128, 256))
        Hq = Hkv * rng.choice((1, 2, 4, 5, 7, 8, 16))
        if op == "read":
            c = dict(op=op, n=_log(rng, 1, 20000), Hkv=Hkv, D=D, page=page, f32=rng.random() < 0.5)
        elif op == "append":
            c = dict(op=op, T=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, D=D, page=page, rot=rng.choice((D, D, D // 2, 0)),
                     interleaved=rng.random() < 0.5, f32=rng.random() < 0.5)
        else:
            kind = rng.choice(("token", "token", "draft", "prompt", "chunk"))
            c = dict(op=op, B=1, T=1, most=_log(rng, 1, 131072), new=1, Hq=Hq, Hkv=Hkv, D=D, page=page,
                     window=rng.choice((0, 0, 0, _log(rng, 16, 4096))), lse=rng.random() < 0.5)
            if kind in ("token", "draft"):
                c["B"] = c["T"] = _log(rng, 1, 200)
            if kind == "draft":
                c["new"] = rng.randint(2, 9)
                c["T"] = rng.randint(c["B"], c["B"] * c["new"])
            if kind in ("prompt", "chunk"):
                c["B"] = rng.randint(1, 6)
                c["T"] = c["new"] = _log(rng, 16, 8192)
                c["most"] = 0 if kind == "prompt" else c["most"]
                c["B"] = min(c["B"], c["T"])
        if _cost(c) <= most[op]:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 100)


def _spread(c):
    """(new tokens, context behind them) of each sequence: ragged, and a
    function of the case alone."""
    B, T, most = c["B"], c["T"], c["most"]
    if c["new"] < T or B == T:              # tokens or drafts: 1 .. new of each
        new, left = [1] * B, T - B
        b = 0
        while left > 0:
            take = min(left, c["new"] - 1, (5 * b) % c["new"] if b < B else c["new"] - 1)
            take = min(take, c["new"] - new[b % B])
            new[b % B] += take
            left -= take
            b += 1
    else:                                   # prompts: a few long ones
        share = [1.0 / (1 + b) for b in range(B)]
        new = [max(1, int(T * x / sum(share))) for x in share]
        new[0] += T - sum(new)
    behind = [most if b == 0 else int(most * (0.03 + 0.97 * ((b * 0.618033988749895) % 1.0))) for b in range(B)]
    return [(n, max(0, p - n) if most else 0) for n, p in zip(new, behind)]


def _seen(c, n, p):
    """Keys that a sequence's rows need, and (token, key) pairs."""
    if not c["window"]:
        return n + p, n * p + n * (n + 1) // 2
    w = c["window"]
    pairs = sum(min(w, p + j + 1) for j in range(n)) if n < 64 else n * p + n * (n + 1) // 2 - sum(
        max(0, p + j + 1 - w) for j in range(n))
    return min(n + p, w + n - 1), pairs


def work(case):
    c = case
    D, Hkv = c["D"], c["Hkv"]
    row = D / 2 + D / 64 * 4
    if c["op"] == "read":
        return dict(bytes=c["n"] * 2.0 * Hkv * (row + D * (4 if c["f32"] else 2)) + 4.0 * c["n"], flops=4.0 * c["n"] * Hkv * D)
    if c["op"] == "append":
        T, Hq, e = c["T"], c["Hq"], 4 if c["f32"] else 2
        # The rows are written, and read back as bf16.
        return dict(bytes=T * 2.0 * Hkv * (e * D + 2 * row + 2 * D) + T * Hq * D * (e + 2.0) + 8.0 * T + 2.0 * c["rot"],
                    flops=T * (Hq * 3.0 + 2.0 * Hkv * 20) * D)
    keys = pairs = 0
    for n, p in _spread(c):
        k, m = _seen(c, n, p)
        keys, pairs = keys + k, pairs + m
    return dict(bytes=keys * 2.0 * Hkv * row + c["T"] * c["Hq"] * (4.0 * D + (4 if c["lse"] else 0)),
                flops=4.0 * D * c["Hq"] * pairs)


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _rows(g, pages, Hkv, page, D):
    """A cache that holds normal values: a block's 64 values reach about 2.4
    standard deviations to each side."""
    shape = (pages, Hkv, page)
    nibbles = []
    for _ in range(2):
        x = torch.randn((*shape, D // 2), generator=g, device=DEV, dtype=torch.float16)
        nibbles.append(x.mul_(3.1).add_(7.5).round_().clamp_(0, 15).to(torch.uint8))
    codes = nibbles[0] | (nibbles[1] << 4)
    scales = (0.25 + 0.15 * torch.rand((*shape, D // 64), generator=g, device=DEV)).to(torch.float16)
    zeros = torch.randint(6, 10, (*shape, D // 64), generator=g, device=DEV).to(torch.float16)
    return codes, scales, zeros


def prepare(case, seed):
    c, g = case, _generator(seed)
    D, Hkv, page = c["D"], c["Hkv"], c["page"]
    s = dict(case=dict(case))
    if c["op"] == "attend":
        seqs = _spread(c)
        need = [-(-(n + p) // page) for n, p in seqs]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=DEV)  # a sequence's pages lie anywhere
        table = torch.zeros((c["B"], max(need)), dtype=torch.int32, device=DEV)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = order[at:at + m].to(torch.int32)
            at += m
        ends = [0]
        for n, _ in seqs:
            ends.append(ends[-1] + n)
        s.update(seqs=seqs, ends=ends, table=table, lens=torch.tensor([n + p for n, p in seqs], dtype=torch.int32, device=DEV),
                 offsets=torch.tensor(ends, dtype=torch.int32, device=DEV), max_q=max(n for n, _ in seqs))
        # Some heads look at few keys, others at many.
        sharp = torch.linspace(0.5, 3.0, c["Hq"], device=DEV)[None, :, None]
        s["q"] = (_randn(g, (c["T"], c["Hq"], D)) * sharp).to(torch.bfloat16)
    else:
        n = c["T"] if c["op"] == "append" else c["n"]
        pages = -(-n * 5 // (4 * page)) + 1
        s["slots"] = torch.randperm(pages * page, generator=g, device=DEV)[:n].to(torch.int32)
        if c["op"] == "append":
            kind = torch.float32 if c["f32"] else torch.bfloat16
            # A projection writes q, k and v side by side; keys have a few large channels.
            big = 1 + 4 * (torch.rand(Hkv, D, generator=g, device=DEV) < 0.05)
            qkv = _randn(g, (n, c["Hq"] + 2 * Hkv, D))
            qkv[:, c["Hq"]:c["Hq"] + Hkv] *= big
            s["qkv"] = qkv.to(kind)
            s["positions"] = (torch.arange(n, device=DEV) + int(torch.randint(0, 100000, (1,), generator=g, device=DEV))).to(torch.int32)
            s["inv_freq"] = (10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / max(c["rot"], 1))).float()
    s["k"], s["v"] = _rows(g, pages, Hkv, page, D), _rows(g, pages, Hkv, page, D)
    if own:
        _handle(s)
    return s


def _handle(s):
    import bit_weight_gemv_amd as q4
    s["cache"] = q4.KVCache(*s["k"], *s["v"])
    return s["cache"]


def run(state):
    s, c = state, state["case"]
    if own:
        import bit_weight_gemv_amd as q4
        cache = s.get("cache") or _handle(s)
        if c["op"] == "attend":
            return q4.q4_cache_attend(s["q"], cache, s["table"], s["lens"], q_offsets=s["offsets"], max_q=s["max_q"],
                                      window=c["window"], return_lse=c["lse"])
        if c["op"] == "read":
            return q4.q4_cache_read(cache, s["slots"], out_dtype=torch.float32 if c["f32"] else torch.bfloat16)
        Hq, Hkv, x = c["Hq"], c["Hkv"], s["qkv"]
        q = q4.q4_cache_append(cache, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], s["slots"], positions=s["positions"],
                               inv_freq=s["inv_freq"], interleaved=c["interleaved"], q=x[:, :Hq])
        return (q, *q4.q4_cache_read(cache, s["slots"]))
    if c["op"] == "attend":
        return _attend(s)
    if c["op"] == "read":
        kind = torch.float32 if c["f32"] else torch.bfloat16
        return tuple(_values(_at(r, s["slots"], c["page"])).to(kind) for r in (s["k"], s["v"]))
    return _append(s)


def _at(rows, slots, page):
    """The codes, scales and zeros of slots, [n, Hkv, .]."""
    p, i = slots.long() // page, slots.long() % page
    return tuple(r[p, :, i] for r in rows)


def _values(rows):
    codes, scales, zeros = rows
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    return (c - zeros.float().repeat_interleave(64, -1)) * scales.float().repeat_interleave(64, -1)


def _rotate(x, s):
    """In 64 bits: angles of far positions, and codes next to a border."""
    c, x = s["case"], x.double()
    rot = c["rot"]
    a = (s["positions"].double()[:, None] * s["inv_freq"].double())[:, None, :]
    cos, sin = torch.cos(a), torch.sin(a)
    out = x.clone()
    if c["interleaved"]:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    else:
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return out


def _pack(x):
    """Codes, scales and zeros of x [..., D] in 64 bits: the nearest level, a
    midpoint to the lower one."""
    x = x.unflatten(-1, (-1, 64))
    hi, lo = x.amax(-1).clamp(min=0), x.amin(-1).clamp(max=0)
    scales = ((hi - lo) / 15).to(torch.float16)
    step = scales.double()[..., None]
    safe = torch.where(step > 0, step, 1.0)
    half = 0.5 + torch.arange(15, device=DEV, dtype=torch.float64)
    zeros = (-lo[..., None] > half * step).sum(-1)
    codes = torch.ceil(x / safe + zeros[..., None] - 0.5).clamp(0, 15)
    codes = torch.where(step > 0, codes, 0.0)
    codes, zeros = codes.to(torch.uint8).flatten(-2), torch.where(step[..., 0] > 0, zeros, 0)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), scales, zeros.to(torch.float16)


def _append(s):
    c, x = s["case"], s["qkv"]
    Hq, Hkv, page = c["Hq"], c["Hkv"], c["page"]
    p, i = s["slots"].long() // page, s["slots"].long() % page
    for rows, new in ((s["k"], _rotate(x[:, Hq:Hq + Hkv], s)), (s["v"], x[:, Hq + Hkv:].double())):
        for r, n in zip(rows, _pack(new)):
            r[p, :, i] = n
    q = _rotate(x[:, :Hq], s).to(torch.bfloat16)
    return (q, *(_values(_at(r, s["slots"], page)).to(torch.bfloat16) for r in (s["k"], s["v"])))


def _context(s, b, rows, values):
    """Keys or values of sequence b, [Hkv, keys, D]."""
    n, p = s["seqs"][b]
    page = s["case"]["page"]
    ids = s["table"][b, :-(-(n + p) // page)].long()
    return values(tuple(r[ids].transpose(0, 1).flatten(1, 2)[:, :n + p] for r in rows))


def _attend(s):
    c = s["case"]
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    G = Hq // Hkv
    out = torch.empty((c["T"], Hq, D), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((c["T"], Hq), device=DEV)
    for b, (n, p) in enumerate(s["seqs"]):
        rows = slice(s["ends"][b], s["ends"][b + 1])
        q = s["q"][rows].float().reshape(n, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, n * G, D)
        k, v = _context(s, b, s["k"], _values), _context(s, b, s["v"], _values)
        score = torch.bmm(q, k.transpose(1, 2).contiguous()) * D ** -0.5
        at = (p + torch.arange(n, device=DEV)).repeat_interleave(G)[:, None]
        key = torch.arange(n + p, device=DEV)
        hidden = key > at
        if c["window"]:
            hidden |= key <= at - c["window"]
        score.masked_fill_(hidden, -math.inf)
        top = score.amax(-1, keepdim=True)
        score = torch.exp(score - top)
        total = score.sum(-1, keepdim=True)
        o = torch.bmm(score, v) / total
        out[rows] = o.reshape(Hkv, n, G, D).permute(1, 0, 2, 3).reshape(n, Hq, D).to(torch.bfloat16)
        lse[rows] = (top + torch.log(total)).reshape(Hkv, n, G).permute(1, 0, 2).reshape(n, Hq)
    return (out, lse) if c["lse"] else out


def _double(rows):
    """The rows' values in 64 bits."""
    codes, scales, zeros = rows
    x = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=torch.float64, device=DEV)
    x[..., 0::2] = (codes % 16).double()
    x[..., 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    x = x.view(*codes.shape[:-1], -1, 64)
    return ((x - zeros.double()[..., None]) * scales.double()[..., None]).flatten(-2)


def _packed_value(x):
    """What a block of the cache holds after x was written to it."""
    x = x.view(*x.shape[:-1], -1, 64)
    lo, hi = -torch.relu(-x).amax(-1, keepdim=True), torch.relu(x).amax(-1, keepdim=True)
    step = ((hi - lo) / 15).half().double()
    z = torch.ceil(-lo / step - 0.5).clamp(0, 15)
    value = (torch.ceil(x / step + z - 0.5).clamp(0, 15) - z) * step
    return torch.where(step > 0, value, torch.zeros_like(value)).flatten(-2)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "read":
        return tuple(_double(_at(r, s["slots"], c["page"])) for r in (s["k"], s["v"]))
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    if c["op"] == "append":
        # Each pair as a complex number times a rotation.
        x, rot = s["qkv"].double(), c["rot"]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           s["positions"].double()[:, None, None] * s["inv_freq"].double())
        first, second = ((slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"]
                         else (slice(0, rot // 2), slice(rot // 2, rot)))
        y = x.clone()
        if rot:
            w = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            y[..., first], y[..., second] = w.real, w.imag
        return y[:, :Hq], _packed_value(y[:, Hq:Hq + Hkv].contiguous()), _packed_value(x[:, Hq + Hkv:].contiguous())
    out = torch.zeros((c["T"], Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((c["T"], Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, (n, p) in enumerate(s["seqs"]):
        first, G = s["ends"][b], Hq // Hkv
        for h in range(Hkv):
            k, v = (_context(s, b, tuple(r[:, h:h + 1] for r in rows), _double)[0] for rows in (s["k"], s["v"]))
            for lo in range(0, n, 1024):
                m = min(n, lo + 1024) - lo
                keys = p + lo + m
                begin = max(0, p + lo - c["window"] + 1) if c["window"] else 0
                pos = p + lo + torch.arange(m, device=DEV)[:, None]
                at = torch.arange(begin, keys, device=DEV)[None, :]
                seen = at <= pos
                if c["window"]:
                    seen = seen & (at > pos - c["window"])
                for g in range(G):
                    q = s["q"][first + lo:first + lo + m, h * G + g].double()
                    z = torch.where(seen, (q @ k[begin:keys].t()) / math.sqrt(D), -math.inf)
                    l = torch.logsumexp(z, 1)
                    lse[first + lo:first + lo + m, h * G + g] = l
                    out[first + lo:first + lo + m, h * G + g] = torch.exp(z - l[:, None]) @ v[begin:keys]
    return (out, lse) if c["lse"] else out
