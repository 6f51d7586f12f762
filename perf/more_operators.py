"""The operators of an expert layer on one card, forward and backward, with the cases they are
measured on.

Five operators, each in a plain torch form (``own`` false) and as the library's own calls
(``own`` true):

  sort         moe_sort_plan, moe_sort_rows: tokens' rows copied into expert order (bf16, fp32, or
               e4m3 codes with their scales); backward, moe_unsort_rows without weights
  unsort       moe_unsort_rows: rows brought back and added up with the router's weights;
               backward, moe_unsort_rows_grad: gradients of the rows and of the weights
  route_grad   moe_topk_route_grad: gradient of the chosen experts' weights to the logits
  linear       moe_expert_linear: bf16 rows by bf16 weights, rows grouped by expert or all of one
               weight, with bias, activation and residual in the epilogue
  linear_grad  moe_activation_grad, moe_expert_linear_grad_input (with the gradient of the
               activation before it in the epilogue), moe_expert_linear_grad_weight (with the bias')

A case is a dict of plain values; ``op`` names the operator.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
BF16 = torch.bfloat16
ACTS = ["none", "relu", "gelu", "silu", "swiglu"]      # in the order of moe_activation
KINDS = {"bf16": BF16, "fp32": torch.float32, "e4m3": F8}


def _case(op, name=None, **kw):
    c = {"op": op}
    if name:
        c["name"] = name
    c.update(kw)
    return c


def listed():
    return [
        # one decoded token's coded row to its experts: pure latency
        _case("sort", "sort 1 token", tokens=1, experts=256, top_k=8, hidden=7168, dtype="e4m3", masked=0.0,
              backward=False),
        # a long prompt's rows to the experts
        _case("sort", "sort prompt", tokens=16384, experts=256, top_k=8, hidden=7168, dtype="bf16", masked=0.0,
              backward=False),
        # a training batch's gradient back to the tokens, some of them padding
        _case("sort", "sort gradient", tokens=4096, experts=64, top_k=6, hidden=4096, dtype="bf16", masked=0.1,
              backward=True),
        # a decode batch of one card: experts' rows back to the tokens
        _case("unsort", "unsort decode batch", tokens=128, experts=256, top_k=8, hidden=7168, dtype="bf16",
              masked=0.0, backward=False),
        # gradients of a training batch's rows and router weights
        _case("unsort", "unsort gradient", tokens=16384, experts=256, top_k=8, hidden=7168, dtype="bf16",
              masked=0.0, backward=True),
        # a small batch of a model with few experts
        _case("route_grad", "route gradient small", tokens=128, experts=8, top_k=2, bf16=True, renorm=True,
              masked=0.0),
        # a training batch's gradient to all logits, some experts masked
        _case("route_grad", "route gradient batch", tokens=131072, experts=256, top_k=8, bf16=False, renorm=False,
              masked=0.05),
        # the router's own product on a decode batch: few columns, a long sum, fp32 logits
        _case("linear", "linear router", experts=1, rows=128, n=256, k=7168, act="none", bias=True, residual=False,
              keep=False, fp32=True, skew=0.0, spare=0),
        # a ragged handful of rows through the experts' output product: odd widths, residual
        _case("linear", "linear ragged small", experts=8, rows=37, n=1000, k=392, act="gelu", bias=True,
              residual=True, keep=False, fp32=False, skew=1.0, spare=5),
        # the experts' gate and up products on a training batch, pre-activations kept for the gradient
        _case("linear", "linear experts", experts=16, rows=32768, n=4096, k=7168, act="swiglu", bias=False,
              residual=False, keep=True, fp32=False, skew=0.3, spare=0),
        # gradients of a small ragged batch, fp32 weight gradients
        _case("linear_grad", "linear gradient small", experts=8, rows=300, n=1000, k=384, act="gelu", before="none",
              bias=True, fp32=True, skew=1.0, spare=5),
        # gradients of the experts' down product on a training batch, through the gate and up activation
        _case("linear_grad", "linear gradient experts", experts=16, rows=32768, n=7168, k=2048, act="none",
              before="swiglu", bias=True, fp32=False, skew=0.3, spare=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "unsort", "route_grad", "linear", "linear_grad"])
    if op in ("sort", "unsort"):
        backward = rng.random() < 0.5
        kinds = ["bf16", "bf16", "fp32", "e4m3"] if op == "sort" and not backward else ["bf16", "bf16", "fp32"]
        dtype = rng.choice(kinds)
        while True:
            experts = _log(rng, 1, 1024)
            tokens, top_k = _log(rng, 1, 131072), min(experts, _log(rng, 1, 16))
            hidden = 128 * _log(rng, 1, 96) if dtype == "e4m3" else 8 * _log(rng, 1, 1536)
            if tokens * top_k * hidden * (2 if dtype == "fp32" else 1) <= 16384 * 8 * 7168:
                break
        return _case(op, tokens=tokens, experts=experts, top_k=top_k, hidden=hidden, dtype=dtype,
                     masked=rng.choice([0.0, 0.0, 0.1, 0.6]), backward=backward)
    if op == "route_grad":
        experts = rng.randint(2, 512)
        tokens = min(_log(rng, 1, 131072), (131072 * 256) // experts)
        return _case(op, tokens=tokens, experts=experts, top_k=min(experts, _log(rng, 1, 16)),
                     bf16=rng.random() < 0.5, renorm=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.1, 0.6]))
    while True:
        experts = rng.choice([1, _log(rng, 1, 256)])
        rows, n, k = _log(rng, 1, 32768), 16 * _log(rng, 1, 448), 8 * _log(rng, 1, 896)
        if experts * n * k <= 1 << 30 and rows * n * k <= 32768 * 7168 * 2048:
            break
    c = _case(op, experts=experts, rows=rows, n=n, k=k, act=rng.choice(ACTS), bias=rng.random() < 0.5,
              fp32=rng.random() < 0.5, skew=rng.choice([0.0, 0.1, 0.3, 1.0]),
              spare=rng.choice([0, 0, rng.randint(1, 200)]))
    if op == "linear":
        c.update(residual=rng.random() < 0.5, keep=rng.random() < 0.5)
    else:
        c.update(before=rng.choice(ACTS))
    return c


# --- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device=DEV)).to(BF16)


def _activations(g, rows, width):
    x = torch.randn((rows, width), generator=g, device=DEV)
    # a few channels are much larger than the rest, as in trained models
    big = torch.rand((width,), generator=g, device=DEV) < 0.01
    return torch.where(big, 12.0 * x, x).to(BF16)


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


def _choices(g, tokens, experts, top_k, masked):
    """Distinct experts of each token by a random popularity, softmax weights; some tokens are
    padding, which names no expert."""
    z = torch.randn((tokens, experts), generator=g, device=DEV)
    z += 0.5 * torch.randn((experts,), generator=g, device=DEV)
    w, idx = torch.topk(torch.softmax(z, -1), top_k, dim=-1)
    idx = idx.to(torch.int32)
    idx[torch.rand((tokens,), generator=g, device=DEV) < masked] = -1
    return idx, w


def _plan64(idx, experts):
    """(offsets, slot, source, rows in use) by a stable sort."""
    flat = idx.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.sort(key, stable=True).indices
    ids = torch.arange(experts + 1, device=idx.device)
    offsets = torch.searchsorted(key[order], ids)
    used = int(offsets[-1])
    slot = torch.full_like(flat, -1)
    slot[order[:used]] = torch.arange(used, device=idx.device)
    return offsets, slot.view(idx.shape), order, used


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op, "case": case}
    if op in ("sort", "unsort"):
        tokens, top_k, hidden, kind = case["tokens"], case["top_k"], case["hidden"], KINDS[case["dtype"]]
        rows = tokens * top_k
        s["idx"], s["w"] = _choices(g, tokens, case["experts"], top_k, case["masked"])
        if op == "sort" and not case["backward"]:
            x = _activations(g, tokens, hidden)
            if kind == F8:
                s["x"] = (40.0 * x.float()).clamp_(-448.0, 448.0).to(F8)
                s["xs"] = torch.rand((tokens, hidden // 128), generator=g, device=DEV) + 0.5
                s["rows_s"] = torch.zeros((rows, hidden // 128), device=DEV)
            else:
                s["x"] = x.to(kind)
            s["rows"] = torch.zeros((rows, hidden), dtype=kind, device=DEV)
            s["offsets"] = torch.zeros((case["experts"] + 1,), dtype=torch.int32, device=DEV)
            s["slot"] = torch.zeros((tokens, top_k), dtype=torch.int32, device=DEV)
            s["source"] = torch.zeros((rows,), dtype=torch.int32, device=DEV)
            return s
        # the plan that the forward pass left
        s["slot"] = _plan64(s["idx"], case["experts"])[1].to(torch.int32)
        s["y"] = _activations(g, rows, hidden).to(kind)
        if op == "unsort" and case["backward"]:
            s["dout"] = _randn(g, (tokens, hidden), 0.01).to(kind)
            s["dy"] = torch.zeros_like(s["y"])
            s["dw"] = torch.zeros((tokens, top_k), device=DEV)
        else:
            s["out"] = torch.zeros((tokens, hidden), dtype=kind, device=DEV)
    elif op == "route_grad":
        tokens, experts = case["tokens"], case["experts"]
        z = 2.0 * torch.randn((tokens, experts), generator=g, device=DEV)
        z[torch.rand((tokens, experts), generator=g, device=DEV) < case["masked"]] = -math.inf
        s["logits"] = z.to(BF16) if case["bf16"] else z
        order = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)
        s["idx"] = order.indices[:, : case["top_k"]].to(torch.int32).contiguous()
        s["dw"] = torch.randn((tokens, case["top_k"]), generator=g, device=DEV)
        s["dlogits"] = torch.zeros_like(s["logits"])
    else:
        experts, rows, n, k = case["experts"], case["rows"], case["n"], case["k"]
        room = rows + case["spare"]              # rows behind the last expert stay as they are
        c = _counts(seed, experts, rows, case["skew"])
        s["bounds"] = [0] + np.cumsum(c).tolist()
        s["offsets"] = None
        if experts > 1 or case["spare"]:
            s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device=DEV)
        s["x"] = _activations(g, room, k)
        s["w"] = torch.empty((experts, n, k), dtype=BF16, device=DEV)
        for e in range(experts):
            s["w"][e] = _randn(g, (n, k), k ** -0.5)
        wide = n // 2 if case["act"] == "swiglu" else n
        kind = torch.float32 if case["fp32"] else BF16
        if op == "linear":
            s["bias"] = _randn(g, (experts, n), 0.5) if case["bias"] else None
            s["residual"] = _activations(g, room, wide) if case["residual"] else None
            s["z"] = torch.zeros((room, n), dtype=BF16, device=DEV) if case["keep"] else None
            s["y"] = torch.zeros((room, wide), dtype=kind, device=DEV)
        else:
            s["dy"] = _randn(g, (room, wide), 0.01)
            s["z"] = _randn(g, (room, n)) if case["act"] != "none" else None
            s["dz"] = torch.zeros((room, n), dtype=BF16, device=DEV) if case["act"] != "none" else None
            before = case["before"]
            s["zb"] = _randn(g, (room, 2 * k if before == "swiglu" else k)) if before != "none" else None
            s["dx"] = torch.zeros((room, 2 * k if before == "swiglu" else k), dtype=BF16, device=DEV)
            s["dw"] = torch.zeros((experts, n, k), dtype=kind, device=DEV)
            s["db"] = torch.zeros((experts, n), device=DEV) if case["bias"] else None
    return s


# --- plain forms -------------------------------------------------------------------------------

def _gather(y, slot):
    """Rows of each token's choices, zeros where it names none: [tokens][top_k][hidden]."""
    v = y[slot.clamp_min(0).long()].float()
    return torch.where(slot[..., None] >= 0, v, 0.0)


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        return g / (1.0 + torch.exp(-g)) * u
    return z


def _act_grad(name, z, d):
    if name == "relu":
        return torch.where(z > 0, d, 0.0)
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return d * (cdf + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5)
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return d * p * (1.0 + z * (1.0 - p))
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        p = 1.0 / (1.0 + torch.exp(-g))
        return torch.cat([d * u * p * (1.0 + g * (1.0 - p)), d * g * p], -1)
    return d


def _run_plain(s):
    op, case = s["op"], s["case"]
    if op == "sort" and not case["backward"]:
        experts, top_k = case["experts"], case["top_k"]
        flat = s["idx"].reshape(-1)
        key = torch.where((flat >= 0) & (flat < experts), flat, experts)
        ordered, order = torch.sort(key, stable=True)
        offsets = torch.searchsorted(ordered, torch.arange(experts + 1, device=DEV, dtype=torch.int32))
        place = torch.arange(key.numel(), device=DEV)
        live = ordered < experts
        slot = torch.empty_like(place)
        slot[order] = torch.where(live, place, -1)
        out = {"offsets": offsets.to(torch.int32), "slot": slot.view(s["slot"].shape).to(torch.int32),
               "source": torch.where(live, order, s["source"]).to(torch.int32)}
        token = order // top_k
        x, old = s["x"], s["rows"]
        if x.dtype == F8:
            out["rows"] = torch.where(live[:, None], x.view(torch.uint8)[token], old.view(torch.uint8)).view(F8)
            out["scales"] = torch.where(live[:, None], s["xs"][token], s["rows_s"])
        else:
            out["rows"] = torch.where(live[:, None], x[token], old)
        return out
    if op == "sort":
        return {"out": _gather(s["y"], s["slot"]).sum(1).to(s["out"].dtype)}
    if op == "unsort" and not case["backward"]:
        return {"out": (_gather(s["y"], s["slot"]) * s["w"][..., None]).sum(1).to(s["out"].dtype)}
    if op == "unsort":
        dout = s["dout"].float()
        dw = (_gather(s["y"], s["slot"]) * dout[:, None]).sum(-1)
        dy = s["dy"].clone()
        live = s["slot"] >= 0
        dy[s["slot"][live].long()] = (s["w"][..., None] * dout[:, None]).to(dy.dtype)[live]
        return {"dy": dy, "dw": dw}
    if op == "route_grad":
        z = s["logits"].float()
        best = z.amax(-1, keepdim=True)
        p = torch.where(best == -math.inf, 0.0, torch.exp(z - best))
        p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
        at = s["idx"].long()
        if case["renorm"]:
            w = torch.gather(p, 1, at)
            w = w / w.sum(-1, keepdim=True).clamp_min(1e-30)
            dz = torch.zeros_like(z).scatter_(1, at, w * (s["dw"] - (w * s["dw"]).sum(-1, keepdim=True)))
        else:
            g = torch.zeros_like(z).scatter_(1, at, s["dw"])
            dz = p * (g - (p * g).sum(-1, keepdim=True))
        return {"dlogits": dz.to(s["dlogits"].dtype)}
    b = s["bounds"]
    if op == "linear":
        y, z = s["y"].clone(), None if s["z"] is None else s["z"].clone()
        for e in range(case["experts"]):
            r = slice(b[e], b[e + 1])
            if b[e] == b[e + 1]:
                continue
            v = torch.matmul(s["x"][r].float(), s["w"][e].float().t())
            if s["bias"] is not None:
                v = v + s["bias"][e].float()
            if z is not None:
                z[r] = v.to(BF16)
            v = _act(case["act"], v)
            if s["residual"] is not None:
                v = v + s["residual"][r].float()
            y[r] = v.to(y.dtype)
        return {"y": y} if z is None else {"y": y, "z": z}
    dx, dw = s["dx"].clone(), torch.zeros_like(s["dw"])
    db = None if s["db"] is None else torch.zeros_like(s["db"])
    dz = None if s["dz"] is None else s["dz"].clone()
    for e in range(case["experts"]):
        r = slice(b[e], b[e + 1])
        if b[e] == b[e + 1]:
            continue
        d = s["dy"][r].float()
        if dz is not None:
            dz[r] = _act_grad(case["act"], s["z"][r].float(), d).to(BF16)
            d = dz[r].float()
        dw[e] = torch.matmul(d.t(), s["x"][r].float()).to(dw.dtype)
        if db is not None:
            db[e] = d.sum(0)
        v = torch.matmul(d, s["w"][e].float())
        if s["zb"] is not None:
            v = _act_grad(case["before"], s["zb"][r].float(), v)
        dx[r] = v.to(BF16)
    out = {"dx": dx, "dw": dw}
    if db is not None:
        out["db"] = db
    if dz is not None:
        out["dz"] = dz
    return out


def _run_own(s):
    import combine_moe_dispatch_amd as mep
    op, case = s["op"], s["case"]
    kinds = {BF16: mep.MOE_BF16, torch.float32: mep.MOE_FP32, F8: mep.MOE_FP8_E4M3}
    if op in ("sort", "unsort"):
        tokens, top_k, hidden, experts = case["tokens"], case["top_k"], case["hidden"], case["experts"]
        rows, kind = tokens * top_k, kinds[KINDS[case["dtype"]]]
        if op == "sort" and not case["backward"]:
            space = torch.empty((mep.moe_sort_workspace(tokens, experts, top_k),), dtype=torch.uint8, device=DEV)
            mep.moe_sort_plan(tokens, experts, top_k, s["idx"], s["offsets"], s["slot"], s["source"], space)
            mep.moe_sort_rows(tokens, top_k, rows, hidden, kind, s["x"], s.get("xs"), s["slot"], s["rows"],
                              s.get("rows_s"))
            out = {"offsets": s["offsets"], "slot": s["slot"], "source": s["source"], "rows": s["rows"]}
            if "rows_s" in s:
                out["scales"] = s["rows_s"]
            return out
        if op == "unsort" and case["backward"]:
            mep.moe_unsort_rows_grad(tokens, top_k, rows, hidden, kind, s["dout"], s["y"], s["slot"], s["w"],
                                     s["dy"], s["dw"])
            return {"dy": s["dy"], "dw": s["dw"]}
        mep.moe_unsort_rows(tokens, top_k, rows, hidden, kind, s["y"], s["slot"],
                            s["w"] if op == "unsort" else None, s["out"])
        return {"out": s["out"]}
    if op == "route_grad":
        kind = kinds[s["logits"].dtype]
        mep.moe_topk_route_grad(case["tokens"], case["experts"], case["top_k"], s["logits"], kind, case["renorm"],
                                s["idx"], s["dw"], s["dlogits"], kind)
        return {"dlogits": s["dlogits"]}
    room, experts, n, k = case["rows"] + case["spare"], case["experts"], case["n"], case["k"]
    space = torch.empty((mep.moe_expert_linear_workspace(room, experts, n, k),), dtype=torch.uint8, device=DEV)
    act = ACTS.index(case["act"])
    if op == "linear":
        mep.moe_expert_linear(room, experts, n, k, s["x"], s["offsets"], s["w"], s["bias"], act, s["residual"],
                              s["z"], s["y"], kinds[s["y"].dtype], space)
        return {"y": s["y"]} if s["z"] is None else {"y": s["y"], "z": s["z"]}
    d = s["dy"]
    if s["dz"] is not None:
        mep.moe_activation_grad(room, experts, n, act, s["offsets"], s["z"], s["dy"], s["dz"])
        d = s["dz"]
    mep.moe_expert_linear_grad_input(room, experts, n, k, d, s["offsets"], s["w"], ACTS.index(case["before"]),
                                     s["zb"], None, s["dx"], mep.MOE_BF16, space)
    mep.moe_expert_linear_grad_weight(room, experts, n, k, d, s["x"], s["offsets"], s["dw"], kinds[s["dw"].dtype],
                                      s["db"], space)
    out = {"dx": s["dx"], "dw": s["dw"]}
    if s["db"] is not None:
        out["db"] = s["db"]
    if s["dz"] is not None:
        out["dz"] = s["dz"]
    return out


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def work(case):
    op = case["op"]
    if op in ("sort", "unsort"):
        tokens, top_k = case["tokens"], case["top_k"]
        pairs = tokens * top_k * (1 - case["masked"])
        row = case["hidden"] * {"bf16": 2, "fp32": 4, "e4m3": 1}[case["dtype"]]
        if case["dtype"] == "e4m3":
            row += case["hidden"] // 128 * 4
        if op == "sort" and not case["backward"]:
            live = tokens * (1 - case["masked"])
            return {"bytes": live * row + pairs * (row + 4) + tokens * top_k * 8 + (case["experts"] + 1) * 4,
                    "flops": 0}
        if not case["backward"] or op == "sort":
            n = pairs * case["hidden"]
            return {"bytes": pairs * row + tokens * (row + top_k * (4 if op == "sort" else 8)), "flops": 2 * n}
        return {"bytes": 2 * pairs * row + tokens * (row + top_k * 12), "flops": 3 * pairs * case["hidden"]}
    if op == "route_grad":
        size = 2 if case["bf16"] else 4
        n = case["tokens"] * case["experts"]
        read = case["tokens"] * case["top_k"] if case["renorm"] else n
        return {"bytes": (n + read) * size + case["tokens"] * case["top_k"] * 8, "flops": 5 * read}
    experts, rows, n, k = case["experts"], case["rows"], case["n"], case["k"]
    used = experts * (1 - (1 - 1 / experts) ** rows) if experts > 1 else 1.0     # experts that have rows
    wide = n // 2 if case["act"] == "swiglu" else n
    if op == "linear":
        b = used * n * (k + case["bias"]) * 2 + rows * k * 2 + rows * wide * (4 if case["fp32"] else 2)
        b += rows * (wide * 2 * case["residual"] + n * 2 * case["keep"])
        return {"bytes": b, "flops": 2.0 * rows * n * k}
    b = used * n * k * 2 + rows * (k + wide) * 2 + experts * n * (k * (4 if case["fp32"] else 2) + 4 * case["bias"])
    if case["act"] != "none":
        b += rows * n * 4                         # z read, dz written
    out = 2 * k if case["before"] == "swiglu" else k
    b += rows * out * (2 if case["before"] == "none" else 4)
    return {"bytes": b, "flops": 4.0 * rows * n * k}


# --- the definition in 64 bits -----------------------------------------------------------------

def _phi64(z):
    return torch.special.ndtr(z)


def _value64(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp_min(0)
    if name == "gelu":
        return z * _phi64(z)
    if name == "silu":
        return z * torch.sigmoid(z)
    f = z.shape[1] // 2
    return z[:, :f] * torch.sigmoid(z[:, :f]) * z[:, f:]


def _slope64(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return _phi64(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    p = torch.sigmoid(z)
    return p + z * p * (1 - p)


def _through64(name, z, d):
    """Gradient to z of sum(d * activation(z))."""
    if name != "swiglu":
        return d * _slope64(name, z)
    f = z.shape[1] // 2
    return torch.cat([d * z[:, f:] * _slope64("silu", z[:, :f]), d * _value64("silu", z[:, :f])], 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("sort", "unsort"):
        tokens, top_k = case["tokens"], case["top_k"]
        offsets, slot, order, used = _plan64(s["idx"], case["experts"])
        if op == "sort" and not case["backward"]:
            at = order[:used] // top_k
            rows = torch.zeros((tokens * top_k, case["hidden"]), dtype=torch.float64, device=DEV)
            rows[:used] = s["x"].double()[at]
            source = torch.zeros_like(order)
            source[:used] = order[:used]
            out = {"offsets": offsets.to(torch.int32), "slot": slot.to(torch.int32),
                   "source": source.to(torch.int32), "rows": rows}
            if "xs" in s:
                out["scales"] = torch.zeros((tokens * top_k, s["xs"].shape[1]), dtype=torch.float64, device=DEV)
                out["scales"][:used] = s["xs"].double()[at]
            return out
        pair = order[:used]                       # row r belongs to token pair[r] // top_k
        token = pair // top_k
        if op == "sort" or not case["backward"]:
            w = torch.ones((used,), dtype=torch.float64, device=DEV)
            if op == "unsort":
                w = s["w"].reshape(-1)[pair].double()
            out = torch.zeros((tokens, case["hidden"]), dtype=torch.float64, device=DEV)
            step = 1 << 14
            for a in range(0, used, step):
                e = min(used, a + step)
                out.index_add_(0, token[a:e], s["y"][a:e].double() * w[a:e, None])
            return {"out": out}
        dout = s["dout"].double()
        dy = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros((tokens * top_k,), dtype=torch.float64, device=DEV)
        step = 1 << 14
        for a in range(0, used, step):
            e = min(used, a + step)
            d = dout[token[a:e]]
            dy[a:e] = d * s["w"].reshape(-1)[pair[a:e]].double()[:, None]
            dw[pair[a:e]] = (d * s["y"][a:e].double()).sum(1)
        return {"dy": dy, "dw": dw.view(tokens, top_k)}
    if op == "route_grad":
        z, at, g = s["logits"].double(), s["idx"].long(), s["dw"].double()
        if case["renorm"]:                        # a softmax over the chosen logits alone
            zc = torch.gather(z, 1, at)
            w = torch.softmax(zc, 1)
            w = torch.where(torch.isneginf(zc).all(1, keepdim=True), 0.0, w)
            d = torch.zeros_like(z)
            d.scatter_(1, at, w * g - w * (w * g).sum(1, keepdim=True))
            return {"dlogits": d}
        p = torch.where(torch.isneginf(z).all(1, keepdim=True), 0.0, torch.softmax(z, 1))
        pc = torch.gather(p, 1, at)
        d = -p * (pc * g).sum(1, keepdim=True)
        d.scatter_add_(1, at, pc * g)
        return {"dlogits": d}
    b, room, n = s["bounds"], case["rows"] + case["spare"], case["n"]
    if op == "linear":
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
        z = torch.zeros((room, n), dtype=torch.float64, device=DEV)
        for e in range(case["experts"]):
            r = slice(b[e], b[e + 1])
            if b[e] < b[e + 1]:
                z[r] = s["x"][r].double() @ s["w"][e].double().T
                if case["bias"]:
                    z[r] += s["bias"][e].double()
                y[r] = _value64(case["act"], z[r])
                if case["residual"]:
                    y[r] += s["residual"][r].double()
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    out = {"dx": torch.zeros(s["dx"].shape, dtype=torch.float64, device=DEV),
           "dw": torch.zeros(s["dw"].shape, dtype=torch.float64, device=DEV)}
    if case["bias"]:
        out["db"] = torch.zeros(s["db"].shape, dtype=torch.float64, device=DEV)
    if case["act"] != "none":
        out["dz"] = torch.zeros(s["dz"].shape, dtype=torch.float64, device=DEV)
    for e in range(case["experts"]):
        r = slice(b[e], b[e + 1])
        if b[e] == b[e + 1]:
            continue
        d = s["dy"][r].double()
        if case["act"] != "none":
            out["dz"][r] = _through64(case["act"], s["z"][r].double(), d)
            d = out["dz"][r].to(BF16).double()    # the gradient that is handed on is a bf16 tensor
        out["dw"][e] = d.T @ s["x"][r].double()
        if case["bias"]:
            out["db"][e] = d.sum(0)
        v = d @ s["w"][e].double()
        out["dx"][r] = v if case["before"] == "none" else _through64(case["before"], s["zb"][r].double(), v)
    return out
