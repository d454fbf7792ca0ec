"""The operators that work beside the 4-bit projections: routing to experts,
products grouped by expert, their weighted sum, and low-rank adapters beside a
packed projection, forward and backward.

Each case is a dict of plain values.  run() computes it in elementary torch
operations (own = False) or through libq4 (own = True).  Weights are in the
NF4-style packed format: 4-bit codes, low nibble first, and an fp16 scale per
64 weights along K.
"""
import math

import torch

own = False

# The format's 16 levels (fp32).
LEVELS = (-1.0, -0.6961928009986877, -0.5250729322433472, -0.39491742849349976,
          -0.2844413220882416, -0.18477340042591095, -0.09104997664690018, 0.0,
          0.07958031445741653, 0.16093014180660248, 0.24611225724220276, 0.3379151225090027,
          0.4407097399234772, 0.5626168847084045, 0.722956657409668, 1.0)

DEV = "cuda"


def listed():
    return [
        # Routing of the one token that a decode step holds.
        dict(name="route-token", op="route", T=1, E=64, k=8, mode="topk"),
        # Routing of a batch of prompts, weights over all experts.
        dict(name="route-prompt", op="route", T=8192, E=128, k=8, mode="all"),
        # The gate/up products of one token's eight experts: the latency of a decode step.
        dict(name="experts-token", op="experts", T=1, E=64, k=8, M=1408, K=2048, swiglu=True),
        # A small decode batch through the down projections: ragged groups of a few rows.
        dict(name="experts-down-batch", op="experts", T=37, E=16, k=2, M=2048, K=1408, swiglu=False),
        # A prompt batch through the gate/up products: compute bound.
        dict(name="experts-prompt", op="experts", T=4096, E=64, k=8, M=1408, K=2048, swiglu=True),
        # The weighted sum over one token's experts.
        dict(name="combine-token", op="combine", T=1, E=64, k=8, M=2048),
        # The same for a prompt batch.
        dict(name="combine-prompt", op="combine", T=4096, E=64, k=8, M=2048),
        # One token of one request on the down shape, with its adapter.
        dict(name="lora-token", op="lora", N=1, M=2048, K=11008, r=16, L=8),
        # A decode batch in which every request brings an adapter of its own.
        dict(name="lora-batch", op="lora", N=32, M=11008, K=2048, r=16, L=24),
        # Prompts of several requests, an odd number of tokens in all.
        dict(name="lora-prompt", op="lora", N=4093, M=11008, K=2048, r=64, L=3),
        # A short training step on a square projection.
        dict(name="lora-grad-short", op="lora_grad", N=96, M=2048, K=2048, r=8, L=4),
        # A training step of 4096 tokens on the gate shape.
        dict(name="lora-grad-long", op="lora_grad", N=4096, M=11008, K=2048, r=16, L=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("route", "experts", "experts", "combine", "lora", "lora", "lora_grad"))
        if op in ("route", "experts", "combine"):
            E = rng.choice((8, 16, 60, 64, 100, 128))
            c = dict(op=op, T=_log(rng, 1, 8192 if op == "route" else 4096), E=E, k=rng.choice((1, 2, 4, 6, 8)))
            if op == "route":
                c["mode"] = rng.choice(("topk", "all"))
            else:
                c["M"] = _log(rng, 128, 5632)
            if op == "experts":
                c["K"] = 64 * rng.randint(4, 64)
                c["swiglu"] = rng.random() < 0.5
        else:
            c = dict(op=op, N=_log(rng, 1, 4096), M=_log(rng, 256, 22016), K=64 * _log(rng, 4, 172),
                     r=rng.choice((8, 16, 24, 32, 64)), L=rng.randint(1, 32))
        if _cost(c) <= most and _experts_bytes(c) <= 4 << 30:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _experts_bytes(c):
    """The plain form holds an expert's weights as 32-bit values."""
    return c["E"] * c["M"] * c["K"] * 4 * (2 if c["swiglu"] else 1) if c["op"] == "experts" else 0


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return dict(bytes=4.0 * T * E + 16.0 * T * k + 4 * (E + 1), flops=4.0 * T * E)
    if c["op"] == "combine":
        T, k, M = c["T"], c["k"], c["M"]
        return dict(bytes=2.0 * T * k * M + 8.0 * T * k + 2.0 * T * M, flops=2.0 * T * k * M)
    if c["op"] == "experts":
        T, E, k, M, K = c["T"], c["E"], c["k"], c["M"], c["K"]
        mats = 2 if c["swiglu"] else 1
        active = E * (1.0 - (1.0 - k / E) ** T)
        rows = T if c["swiglu"] else T * k
        return dict(bytes=active * mats * M * K * (0.5 + 1 / 32) + 2.0 * rows * K + 2.0 * T * k * M + 4.0 * T * k,
                    flops=2.0 * T * k * mats * M * K)
    N, M, K, r, L = c["N"], c["M"], c["K"], c["r"], c["L"]
    used = min(L, N)
    if c["op"] == "lora":
        return dict(bytes=M * K * (0.5 + 1 / 32) + 2.0 * N * (K + M) + 2.0 * used * r * (K + M) + 4.0 * N,
                    flops=2.0 * N * M * K + 2.0 * N * r * (M + K))
    return dict(bytes=M * K * (0.5 + 1 / 32) + 2.0 * N * (2 * K + M) + 2.0 * used * r * (K + M)
                + 4.0 * L * r * (K + M) + 4.0 * N,
                flops=2.0 * N * M * K + 4.0 * N * r * M + 6.0 * N * r * K)


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _packed(g, *shape):
    """Codes of normal weights are close to evenly used; a block's largest
    magnitude of 64 weights of standard deviation 0.02 lies around 0.05."""
    *lead, M, K = shape
    codes = torch.randint(0, 256, (*lead, M, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = (0.04 + 0.02 * torch.rand((*lead, M, K // 64), generator=g, device=DEV)).to(torch.float16)
    return codes, scales


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(case=dict(case))
    if c["op"] in ("route", "experts", "combine"):
        T, E, k = c["T"], c["E"], c["k"]
        # Experts are not equally popular.
        logits = torch.randn((T, E), generator=g, device=DEV) + 0.7 * torch.randn((1, E), generator=g, device=DEV)
        s["logits"] = logits
        if c["op"] != "route":
            experts, weights, offsets, rows, pos = _route(logits, k, "topk")
            s.update(weights=weights, offsets=offsets, rows=rows, pos=pos)
            # The rows that the fullest expert gets: the padded width of the plain form.
            s["most"] = int((offsets[1:] - offsets[:-1]).max())
        if c["op"] == "combine":
            s["Y"] = _normal(g, (T * k, c["M"]))
        if c["op"] == "experts":
            M, K = c["M"], c["K"]
            s["codes"], s["scales"] = _packed(g, E, M, K)
            s["up"] = _packed(g, E, M, K) if c["swiglu"] else None
            # Gate and up read the tokens; down reads one row for each token and expert.
            if c["swiglu"]:
                s["X"] = _normal(g, (T, K))
            else:
                a, b = _normal(g, (T * k, K), dtype=torch.float32), _normal(g, (T * k, K), dtype=torch.float32)
                s["X"] = (a * torch.sigmoid(a) * b).to(torch.bfloat16)
                s["rows"] = None
        return s
    N, M, K, r, L = c["N"], c["M"], c["K"], c["r"], c["L"]
    s["codes"], s["scales"] = _packed(g, M, K)
    s["X"] = _normal(g, (N, K))
    s["A"] = _normal(g, (L, r, K), K ** -0.5)
    s["B"] = _normal(g, (L, M, r), 0.02)
    s["scaling"] = 0.25 + 1.75 * torch.rand(L, generator=g, device=DEV)
    if N <= 64:  # a decode batch: one token of each request, some of them without an adapter
        ids = torch.randint(0, L, (N,), generator=g, device=DEV)
        ids = torch.where(torch.rand(N, generator=g, device=DEV) < 0.125, -1, ids) if N > 1 else ids
    else:        # prompts: runs of tokens, the lengths ragged
        cuts = torch.rand(max(2, N // 256), generator=g, device=DEV).mul(N).long()
        request = (torch.arange(N, device=DEV)[:, None] >= cuts[None, :]).sum(1)
        ids = torch.randint(0, L, (cuts.numel() + 1,), generator=g, device=DEV)[request]
    s["ids"] = ids.to(torch.int32)
    if c["op"] == "lora_grad":
        s["dY"] = _normal(g, (N, M), 1e-3)
    return s


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import bit_weight_gemv_amd as q4
        if op == "route":
            return q4.q4_route_topk(s["logits"], c["k"], c["mode"])
        if op == "experts":
            return q4.q4_gemm_grouped(s["codes"], s["scales"], s["X"], s["offsets"], rows=s["rows"], up=s["up"])
        if op == "combine":
            return q4.q4_moe_combine(s["Y"], s["weights"], s["pos"])
        args = (s["codes"], s["scales"], s["X"], s["A"], s["B"], s["scaling"], s["ids"])
        if op == "lora":
            return q4.q4_gemm_lora(*args)
        return q4.q4_gemm_lora_backward(s["dY"], *args)
    if op == "route":
        return _route(s["logits"], c["k"], c["mode"])
    if op == "experts":
        y = _grouped(s, s["codes"], s["scales"])
        if s["up"] is not None:
            y = y * torch.sigmoid(y) * _grouped(s, *s["up"])
        return y.to(torch.bfloat16)
    if op == "combine":
        return (s["Y"][s["pos"].long()].float() * s["weights"][:, :, None]).sum(1).to(torch.bfloat16)
    if op == "lora":
        return _lora(s)
    return _lora_grad(s)


def _route(logits, k, mode):
    """Top k by logit (ties to the lowest index), softmax weights, and the
    slots sorted by expert: offsets, the token at each position, and the
    position of each slot."""
    T, E = logits.shape
    top, experts = torch.sort(logits, dim=1, descending=True, stable=True)
    top, experts = top[:, :k], experts[:, :k]
    p = torch.exp(top - top[:, :1])
    total = torch.exp(logits - top[:, :1]).sum(1, keepdim=True) if mode == "all" else p.sum(1, keepdim=True)
    flat = experts.reshape(-1)
    order = torch.sort(flat, stable=True)[1]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), (flat[:, None] == torch.arange(E, device=DEV)).sum(0).cumsum(0)])
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device=DEV)
    i32 = torch.int32
    return experts.to(i32), p / total, offsets.to(i32), (order // k).to(i32), pos.reshape(T, k).to(i32)


def _dequantise(codes, scales):
    pair = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    levels = torch.tensor(LEVELS, device=DEV)
    return levels[pair] * scales.float().repeat_interleave(64, -1)


def _grouped(s, codes, scales):
    """The products of the experts' rows, each expert's rows padded to the
    fullest one's number."""
    offsets, most = s["offsets"].long(), s["most"]
    R = s["pos"].numel()
    at = offsets[:-1, None] + torch.arange(most, device=DEV)
    at = at.clamp(max=R - 1)
    x = s["X"][s["rows"].long()[at] if s["rows"] is not None else at].float()   # [E, most, K]
    y = torch.bmm(_dequantise(codes, scales), x.transpose(1, 2).contiguous())   # [E, M, most]
    p = torch.arange(R, device=DEV)
    e = torch.searchsorted(offsets[1:].contiguous(), p, right=True)
    return y[e, :, p - offsets[e]]


def _adapted(s):
    """Whether token n uses adapter a (as 0 or its scaling), [N, L, 1]."""
    hit = s["ids"][:, None] == torch.arange(s["A"].shape[0], device=DEV)
    return (hit * s["scaling"])[:, :, None]


def _lora(s):
    L, r, K = s["A"].shape
    x = s["X"].float()
    t = (x @ s["A"].float().reshape(L * r, K).t()).reshape(-1, L, r) * _adapted(s)
    b = s["B"].float().permute(0, 2, 1).reshape(L * r, -1)
    return (x @ _dequantise(s["codes"], s["scales"]).t() + t.reshape(-1, L * r) @ b).to(torch.bfloat16)


def _lora_grad(s):
    L, r, K = s["A"].shape
    M = s["B"].shape[1]
    x, dy, use = s["X"].float(), s["dY"].float(), _adapted(s)
    a, b = s["A"].float().reshape(L * r, K), s["B"].float().permute(0, 2, 1).reshape(L * r, M)
    t = ((x @ a.t()).reshape(-1, L, r) * use).reshape(-1, L * r)
    u = ((dy @ b.t()).reshape(-1, L, r) * use).reshape(-1, L * r)
    dx = dy @ _dequantise(s["codes"], s["scales"]) + u @ a
    da = (u.t() @ x).reshape(L, r, K)
    db = (t.t() @ dy).reshape(L, r, M).transpose(1, 2).contiguous()
    return dx.to(torch.bfloat16), da, db


def _values(codes, scales):
    """A packed matrix's weights in 64 bits."""
    M, K = scales.shape[0], scales.shape[1] * 64
    table = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)
    w = torch.empty((M, K), dtype=torch.float64, device=DEV)
    w[:, 0::2] = table[(codes % 16).long()]
    w[:, 1::2] = table[torch.div(codes, 16, rounding_mode="floor").long()]
    return (w.view(M, -1, 64) * scales.double()[:, :, None]).view(M, K)


def exact(case, seed):
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "route":
        l = s["logits"].double()
        chosen = torch.gather(l, 1, _route(s["logits"], c["k"], c["mode"])[0].long())
        over = l if c["mode"] == "all" else chosen
        return None, torch.exp(chosen - torch.logsumexp(over, 1, keepdim=True)), None, None, None
    if op == "combine":
        out = torch.zeros((c["T"], c["M"]), dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            out += s["weights"][:, j].double()[:, None] * s["Y"][s["pos"][:, j].long()].double()
        return out
    if op == "experts":
        cut = s["offsets"].tolist()
        y = torch.zeros((cut[-1], c["M"]), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            lo, hi = cut[e], cut[e + 1]
            if lo == hi:
                continue
            x = s["X"][s["rows"][lo:hi].long()] if s["rows"] is not None else s["X"][lo:hi]
            v = x.double() @ _values(s["codes"][e], s["scales"][e]).t()
            if s["up"] is not None:
                v = v / (1 + torch.exp(-v)) * (x.double() @ _values(s["up"][0][e], s["up"][1][e]).t())
            y[lo:hi] = v
        return y
    x, w = s["X"].double(), _values(s["codes"], s["scales"])
    dy = s["dY"].double() if op == "lora_grad" else None
    y = x @ w.t() if dy is None else dy @ w
    da, db = torch.zeros(s["A"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["B"].shape, dtype=torch.float64, device=DEV)
    for l in range(c["L"]):
        n = torch.nonzero(s["ids"] == l).flatten()
        a, b, f = s["A"][l].double(), s["B"][l].double(), s["scaling"][l].double()
        if dy is None:
            y[n] += f * (x[n] @ a.t()) @ b.t()
        else:
            u = f * (dy[n] @ b)
            y[n] += u @ a
            da[l], db[l] = u.t() @ x[n], f * (dy[n].t() @ (x[n] @ a.t()))
    return y if dy is None else (y, da, db)
