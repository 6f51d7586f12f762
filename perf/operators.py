"""The operators around dispatch and combine, with the cases they are measured on.

Five operators, each in a plain torch form (``own`` false) and as the library's
own calls (``own`` true):

  norm     moe_add_rmsnorm: residual addition, RMS norm, bf16 rows and e4m3 rows
           with an fp32 scale per 128 elements (the dispatch payload's codec)
  route    moe_topk_route: softmax over the experts, the K best of a token
  matmul   moe_expert_matmul: e4m3 rows by e4m3 weights, rows grouped by expert,
           fp32 scales per 128 elements of a row and per 128 x 128 weight block
  gate_up  moe_expert_gate_up: the same product with [gate; up] weights, then
           silu(gate) * up, coded as e4m3 rows with scales for the next product
  few      moe_few_token_layer: a whole expert layer for a few tokens

A case is a dict of plain values; ``op`` names the operator.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 128
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TINY = 2.0 ** -126          # the smallest scale of the codec


def _case(op, name=None, **kw):
    c = {"op": op}
    if name:
        c["name"] = name
    c.update(kw)
    return c


def listed():
    return [
        # one decoded token entering a layer: pure latency
        _case("norm", "norm 1 token", rows=1, hidden=7168, residual=True, fp8=True),
        # a decode batch of a whole group (32 ranks x 128 tokens)
        _case("norm", "norm decode batch", rows=4096, hidden=7168, residual=True, fp8=True),
        # a long prompt, bf16 only, no residual (the first norm of a model)
        _case("norm", "norm long prompt", rows=65536, hidden=4096, residual=False, fp8=False),
        # a small decode batch with bf16 logits, where many logits tie
        _case("route", "route small bf16", tokens=128, experts=8, top_k=2, bf16=True, renorm=True,
              masked=0.0),
        # prefill tokens of a whole group (64 ranks x 2048), some experts masked
        _case("route", "route prefill", tokens=131072, experts=256, top_k=8, bf16=False,
              renorm=False, masked=0.05),
        # a few ragged requests: odd widths, single rows, experts without rows
        _case("matmul", "matmul ragged small", experts=8, rows=37, n=1000, k=384, skew=1.0, spare=5),
        # the down product of a decode batch: 4096 tokens x top-8 over 256 experts
        _case("matmul", "matmul down decode", experts=256, rows=32768, n=7168, k=2048, skew=0.1,
              spare=0),
        # one dense product (a shared expert, an output projection) over a long prompt
        _case("matmul", "matmul dense prompt", experts=1, rows=16384, n=7168, k=4096, skew=0.0,
              spare=0),
        # gate and up of one rank's experts on a prefill batch: compute bound
        _case("gate_up", "gate_up prefill", experts=16, rows=32768, f=2048, k=7168, skew=0.3, spare=0),
        # gate and up of a small decode batch: 128 tokens x top-8 over 256 experts, ~4 rows each
        _case("gate_up", "gate_up small decode", experts=256, rows=1024, f=2048, k=4096, skew=0.3,
              spare=0),
        # a whole layer for one token
        _case("few", "few 1 token", tokens=1, experts=256, top_k=8, hidden=7168, f=2048, padded=0),
        # a whole layer for a small batch, padded by two empty tokens
        _case("few", "few 16 tokens", tokens=16, experts=64, top_k=4, hidden=4096, f=2048, padded=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "matmul", "gate_up", "few"])
    if op == "norm":
        fp8 = rng.random() < 0.6
        hidden = 128 * _log(rng, 1, 96) if fp8 else 8 * _log(rng, 1, 1536)
        rows = min(_log(rng, 1, 65536), (65536 * 4096) // hidden)
        return _case("norm", rows=rows, hidden=hidden, residual=rng.random() < 0.6, fp8=fp8)
    if op == "route":
        experts = rng.randint(2, 512)
        tokens = min(_log(rng, 1, 131072), (131072 * 256) // experts)
        return _case("route", tokens=tokens, experts=experts, top_k=min(experts, _log(rng, 1, 16)),
                     bf16=rng.random() < 0.5, renorm=rng.random() < 0.5,
                     masked=rng.choice([0.0, 0.0, 0.1, 0.6]))
    if op in ("matmul", "gate_up"):
        while True:
            experts = _log(rng, 1, 256)
            rows = _log(rng, 1, 32768)
            k = 128 * _log(rng, 1, 56)
            wide = 8 * _log(rng, 4, 896) if op == "matmul" else 128 * _log(rng, 1, 24)
            n = wide if op == "matmul" else 2 * wide
            if experts * n * k <= 1 << 32 and rows * n * k <= 1 << 39:
                break
        dim = {"n": wide} if op == "matmul" else {"f": wide}
        return _case(op, experts=experts, rows=rows, k=k, skew=rng.choice([0.0, 0.1, 0.3, 1.0]),
                     spare=rng.choice([0, 0, rng.randint(1, 200)]), **dim)
    while True:
        experts = rng.randint(2, 256)
        hidden, f = 128 * _log(rng, 2, 56), 128 * _log(rng, 1, 24)
        tokens = _log(rng, 1, 64)
        top_k = min(experts, rng.randint(1, 8))
        if experts * f * hidden <= 1 << 32 and tokens * top_k * f * hidden <= 1 << 31:
            break
    return _case("few", tokens=tokens, experts=experts, top_k=top_k, hidden=hidden, f=f,
                 padded=rng.choice([0, 0, rng.randint(0, tokens - 1)]))


# --- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _weights(g, experts, n, k):
    """e4m3 weights [E][n][k] and their scales [E][ceil(n/128)][k/128]: normal values that fill
    the format, blocks of different magnitude, products of unit size."""
    w = torch.empty((experts, n, k), dtype=F8, device=DEV)
    for e in range(experts):
        w[e] = (torch.randn((n, k), generator=g, device=DEV) * 96.0).clamp_(-F8_MAX, F8_MAX).to(F8)
    s = torch.rand((experts, -(-n // BLOCK), k // BLOCK), generator=g, device=DEV) + 0.5
    return w, s / (96.0 * math.sqrt(k))


def _counts(seed, experts, rows, skew):
    """Rows of each expert: even on average; popularity spread by `skew`; no expert takes more
    than a few times its share (plus a few rows), the rest moves on."""
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    p = np.exp(skew * r.standard_normal(experts))
    c = r.multinomial(rows, p / p.sum())
    most = 4 * (rows // experts) + 8
    over = int(np.maximum(c - most, 0).sum())
    c = np.minimum(c, most)
    while over:
        free = np.flatnonzero(c < most)
        take = free[: over]
        c[take] += 1
        over -= len(take)
    return c


def _activations(g, rows, width):
    x = torch.randn((rows, width), generator=g, device=DEV)
    # a few channels are much larger than the rest, as in trained models
    big = torch.rand((width,), generator=g, device=DEV) < 0.01
    return torch.where(big, 12.0 * x, x).to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op, "case": case}
    if op == "norm":
        rows, hidden = case["rows"], case["hidden"]
        s["x"] = _activations(g, rows, hidden)
        s["residual"] = 4.0 * _activations(g, rows, hidden) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn((hidden,), generator=g, device=DEV)).to(torch.bfloat16)
        s["residual_out"] = torch.zeros_like(s["x"]) if case["residual"] else None
        s["y"] = torch.zeros_like(s["x"])
        s["yq"] = torch.zeros((rows, hidden), dtype=F8, device=DEV) if case["fp8"] else None
        s["ys"] = torch.zeros((rows, hidden // BLOCK), device=DEV) if case["fp8"] else None
    elif op == "route":
        tokens, experts = case["tokens"], case["experts"]
        z = 2.0 * torch.randn((tokens, experts), generator=g, device=DEV)
        z[torch.rand((tokens, experts), generator=g, device=DEV) < case["masked"]] = -math.inf
        s["logits"] = z.to(torch.bfloat16) if case["bf16"] else z
        s["idx"] = torch.zeros((tokens, case["top_k"]), dtype=torch.int32, device=DEV)
        s["w"] = torch.zeros((tokens, case["top_k"]), device=DEV)
    elif op in ("matmul", "gate_up"):
        experts, rows, k = case["experts"], case["rows"], case["k"]
        n = case["n"] if op == "matmul" else 2 * case["f"]
        room = rows + case["spare"]              # rows behind the last expert stay as they are
        c = _counts(seed, experts, rows, case["skew"])
        s["most"], s["total"] = int(c.max()), rows
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(c)]).astype(np.int32)).to(DEV)
        s["x"], s["xs"] = _encode(_activations(g, room, k).float())
        s["w"], s["ws"] = _weights(g, experts, n, k)
        if op == "matmul":
            s["y"] = torch.zeros((room, n), dtype=torch.bfloat16, device=DEV)
        else:
            s["h"] = torch.zeros((room, case["f"]), dtype=F8, device=DEV)
            s["hs"] = torch.zeros((room, case["f"] // BLOCK), device=DEV)
    else:
        tokens, experts, top_k = case["tokens"], case["experts"], case["top_k"]
        hidden, f = case["hidden"], case["f"]
        s["x"] = _activations(g, tokens, hidden)
        z = torch.randn((tokens, experts), generator=g, device=DEV)
        s["w"], idx = torch.topk(torch.softmax(z, -1), top_k, dim=-1)
        s["idx"] = idx.to(torch.int32)
        if case["padded"]:                       # empty tokens of a padded batch name no expert
            s["idx"][tokens - case["padded"]:] = -1
        s["w13"], s["s13"] = _weights(g, experts, 2 * f, hidden)
        s["w2"], s["s2"] = _weights(g, experts, hidden, f)
        s["out"] = torch.zeros((tokens, hidden), dtype=torch.bfloat16, device=DEV)
    return s


# --- plain forms -------------------------------------------------------------------------------

def _encode(v):
    """fp32 rows [..][w] -> (e4m3 codes, fp32 scale per 128 elements), the dispatch payload's
    codec: scale = amax / 448 held at 2^-126 or more, 1 for a block of zeros."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)
    amax = b.abs().amax(-1)
    top = torch.full_like(amax, F8_MAX)          # tensor by tensor: a division, not a reciprocal
    small = amax < F8_MAX * TINY
    scale = torch.where(small, torch.where(amax == 0, 1.0, TINY), amax / top)
    inv = torch.where(small, torch.where(amax == 0, 0.0, 1.0 / TINY), top / amax)
    return (b * inv[..., None]).reshape(v.shape).to(F8), scale


def _decode_rows(q, s):
    return (q.float().view(*q.shape[:-1], -1, BLOCK) * s[..., None]).view(q.shape)


def _decode_weights(w, s):
    n, k = w.shape[-2:]
    rows = s.repeat_interleave(BLOCK, dim=-2)[..., :n, :]
    v = w.float()
    v.view(*w.shape[:-1], k // BLOCK, BLOCK).mul_(rows[..., None])
    return v


def _grouped(s):
    """fp32 product of every row with its expert's weights: the experts' rows side by side,
    each padded to the longest, in one batched product."""
    experts = s["w"].shape[0]
    r = torch.arange(s["total"], device=DEV)
    e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
    at = r - s["offsets"].long()[e]
    x = _decode_rows(s["x"][: s["total"]], s["xs"][: s["total"]])
    pad = torch.zeros((experts, s["most"], x.shape[1]), device=DEV)
    pad[e, at] = x
    y = torch.bmm(_decode_weights(s["w"], s["ws"]), pad.transpose(1, 2).contiguous())
    return y[e, :, at]


def _silu_mul(a):
    f = a.shape[-1] // 2
    g, u = a[..., :f], a[..., f:]
    return g / (1.0 + torch.exp(-g)) * u


def _run_plain(s):
    op, case = s["op"], s["case"]
    if op == "norm":
        v = s["x"].float()
        if s["residual"] is not None:
            v = v + s["residual"].float()
        y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
        out = {"y": y.to(torch.bfloat16)}
        if case["residual"]:
            out["residual_out"] = v.to(torch.bfloat16)
        if case["fp8"]:
            out["yq"], out["ys"] = _encode(y)
        return out
    if op == "route":
        z = s["logits"].float()
        order = torch.sort(z, dim=-1, descending=True, stable=True)
        idx = order.indices[:, : case["top_k"]]
        best = order.values[:, :1]
        p = torch.where(best == -math.inf, 0.0, torch.exp(z - best))
        p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
        w = torch.gather(p, 1, idx)
        if case["renorm"]:
            w = w / w.sum(-1, keepdim=True).clamp_min(1e-30)
        return {"idx": idx.to(torch.int32), "w": w}
    if op == "matmul":
        y = s["y"].clone()
        y[: s["total"]] = _grouped(s).to(torch.bfloat16)
        return {"y": y}
    if op == "gate_up":
        h, hs = s["h"].clone(), s["hs"].clone()
        h[: s["total"]], hs[: s["total"]] = _encode(_silu_mul(_grouped(s)))
        return {"h": h, "hs": hs}
    tokens, top_k = s["idx"].shape
    pair = s["idx"].reshape(-1).long()
    at = pair.clamp_min(0)
    x = _decode_rows(*_encode(s["x"].float())).repeat_interleave(top_k, 0)
    a = torch.bmm(_decode_weights(s["w13"].view(torch.uint8)[at].view(F8), s["s13"][at]), x[:, :, None])
    h = _decode_rows(*_encode(_silu_mul(a[:, :, 0])))
    y = torch.bmm(_decode_weights(s["w2"].view(torch.uint8)[at].view(F8), s["s2"][at]), h[:, :, None])
    y = torch.where(pair[:, None] >= 0, y[:, :, 0] * s["w"].reshape(-1, 1), 0.0)
    return {"out": y.view(tokens, top_k, -1).sum(1).to(torch.bfloat16)}


def _run_own(s):
    import combine_moe_dispatch_amd as mep
    op, case = s["op"], s["case"]
    if op == "norm":
        mep.moe_add_rmsnorm(case["rows"], case["hidden"], s["x"], s["residual"], s["weight"], 1e-6,
                            s["residual_out"], s["y"], s["yq"], s["ys"])
        out = {"y": s["y"]}
        if case["residual"]:
            out["residual_out"] = s["residual_out"]
        if case["fp8"]:
            out["yq"], out["ys"] = s["yq"], s["ys"]
        return out
    if op == "route":
        mep.moe_topk_route(case["tokens"], case["experts"], case["top_k"], s["logits"],
                           mep.MOE_BF16 if case["bf16"] else mep.MOE_FP32, case["renorm"],
                           s["idx"], s["w"])
        return {"idx": s["idx"], "w": s["w"]}
    if op == "matmul":
        mep.moe_expert_matmul(case["rows"] + case["spare"], case["experts"], case["n"], case["k"],
                              s["x"], s["xs"], s["offsets"], s["w"], s["ws"], s["y"])
        return {"y": s["y"]}
    if op == "gate_up":
        mep.moe_expert_gate_up(case["rows"] + case["spare"], case["experts"], case["f"], case["k"],
                               s["x"], s["xs"], s["offsets"], s["w"], s["ws"], s["h"], s["hs"])
        return {"h": s["h"], "hs": s["hs"]}
    size = mep.moe_few_token_workspace(case["tokens"], case["top_k"], case["hidden"], case["f"])
    space = torch.empty((size,), dtype=torch.uint8, device=DEV)
    mep.moe_few_token_layer(case["tokens"], case["experts"], case["top_k"], case["hidden"],
                            case["f"], s["x"], s["idx"], s["w"], s["w13"], s["s13"], s["w2"],
                            s["s2"], s["out"], space)
    return {"out": s["out"]}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["hidden"]
        b = n * 2 * (2 + 2 * case["residual"]) + case["hidden"] * 2
        if case["fp8"]:
            b += n + n // BLOCK * 4
        return {"bytes": b, "flops": 6 * n}
    if op == "route":
        n = case["tokens"] * case["experts"]
        return {"bytes": n * (2 if case["bf16"] else 4) + case["tokens"] * case["top_k"] * 8,
                "flops": 4 * n}
    if op in ("matmul", "gate_up"):
        experts, rows, k = case["experts"], case["rows"], case["k"]
        n = case["n"] if op == "matmul" else 2 * case["f"]
        used = experts * (1 - (1 - 1 / experts) ** rows)     # experts that have rows
        b = used * (n * k + -(-n // BLOCK) * (k // BLOCK) * 4) + rows * (k + k // BLOCK * 4)
        b += rows * n * 2 if op == "matmul" else rows * (n // 2 + n // 2 // BLOCK * 4)
        return {"bytes": b, "flops": 2.0 * rows * n * k}
    tokens, experts, top_k = case["tokens"] - case["padded"], case["experts"], case["top_k"]
    used = experts * (1 - (1 - top_k / experts) ** tokens)   # distinct experts of the batch
    one = 3 * case["f"] * case["hidden"]
    return {"bytes": max(1.0, used * one * (1 + 4 / BLOCK / BLOCK)) + case["tokens"] * case["hidden"] * 4,
            "flops": 2.0 * tokens * top_k * one}


# --- the definition in 64 bits -----------------------------------------------------------------

def _grid(v):
    """Nearest e4m3 value, ties to even, by the format's steps."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3.0)
    return (torch.round(v / step) * step).clamp(-F8_MAX, F8_MAX)


def _scales64(v):
    b = v.unflatten(-1, (-1, BLOCK)).abs().amax(-1) / F8_MAX
    return torch.where(b == 0, torch.ones_like(b), b.clamp_min(TINY))


def _codes64(v):
    return v / _scales64(v).repeat_interleave(BLOCK, -1)


def _coded64(v):
    """The values that the codec's codes and scales stand for. Its decisions are defined in fp32
    (inverse, product): bf16 inputs lie on ties too often to be decided in more bits."""
    amax = v.unflatten(-1, (-1, BLOCK)).abs().amax(-1)
    small = amax < F8_MAX * TINY
    inv = torch.where(small, 1.0 / TINY, F8_MAX / amax).float().double().repeat_interleave(BLOCK, -1)
    return _grid((v * inv).float().double()) * _scales64(v).repeat_interleave(BLOCK, -1)


def _weights64(w, s):
    v = w.double()
    for b in range(s.shape[0]):
        v[b * BLOCK: (b + 1) * BLOCK] *= s[b].double().repeat_interleave(BLOCK)
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = s["x"].double()
        if case["residual"]:
            v = v + s["residual"].double()
        y = v / torch.sqrt((v * v).sum(-1, keepdim=True) / case["hidden"] + 1e-6) * s["weight"].double()
        return {"y": y, "residual_out": v if case["residual"] else None,
                "yq": _codes64(y) if case["fp8"] else None, "ys": _scales64(y) if case["fp8"] else None}
    if op == "route":
        z = s["logits"].double()
        left, picks = z.clone(), []
        none = torch.isneginf(z).all(-1, keepdim=True)
        shift = torch.where(none, 0.0, z.amax(-1, keepdim=True))
        p = torch.exp(z - shift)
        p = p / torch.where(none, 1.0, p.sum(-1, keepdim=True))
        gone = torch.zeros_like(z, dtype=torch.bool)
        for _ in range(case["top_k"]):
            top = left.masked_fill(gone, math.nan).nan_to_num(nan=-math.inf, neginf=-1e300, posinf=1e300)
            top = top.masked_fill(gone, -math.inf)
            at = (top == top.amax(-1, keepdim=True)).int().argmax(-1, keepdim=True)
            picks.append(at)
            gone.scatter_(1, at, True)
        idx = torch.cat(picks, 1)
        w = torch.gather(p, 1, idx)
        if case["renorm"]:
            w = w / torch.where(none, 1.0, w.sum(-1, keepdim=True))
        return {"idx": idx.to(torch.int32), "w": w}
    if op in ("matmul", "gate_up"):
        width = case["n"] if op == "matmul" else case["f"]
        room = case["rows"] + case["spare"]
        y = torch.zeros((room, width), dtype=torch.float64, device=DEV)
        hs = None if op == "matmul" else torch.zeros((room, width // BLOCK), dtype=torch.float64, device=DEV)
        o = s["offsets"].tolist()
        for e in range(case["experts"]):
            if o[e] == o[e + 1]:
                continue
            x = s["x"][o[e]: o[e + 1]].double() * s["xs"][o[e]: o[e + 1]].double().repeat_interleave(BLOCK, 1)
            a = x @ _weights64(s["w"][e], s["ws"][e]).T
            if op == "matmul":
                y[o[e]: o[e + 1]] = a
            else:
                h = a[:, :width] * torch.sigmoid(a[:, :width]) * a[:, width:]
                y[o[e]: o[e + 1]], hs[o[e]: o[e + 1]] = _codes64(h), _scales64(h)
        return {"y": y} if op == "matmul" else {"h": y, "hs": hs}
    out = torch.zeros((case["tokens"], case["hidden"]), dtype=torch.float64, device=DEV)
    x = _coded64(s["x"].double())
    idx = s["idx"].tolist()
    for e in range(case["experts"]):
        hit = [(t, j) for t in range(case["tokens"]) for j in range(case["top_k"]) if idx[t][j] == e]
        if not hit:
            continue
        t = torch.tensor([a for a, _ in hit], device=DEV)
        j = torch.tensor([b for _, b in hit], device=DEV)
        a = x[t] @ _weights64(s["w13"][e], s["s13"][e]).T
        h = a[:, : case["f"]] * torch.sigmoid(a[:, : case["f"]]) * a[:, case["f"]:]
        h = _coded64(h)
        y = h @ _weights64(s["w2"][e], s["s2"][e]).T
        out.index_add_(0, t, y * s["w"][t, j].double()[:, None])
    return {"out": out}
