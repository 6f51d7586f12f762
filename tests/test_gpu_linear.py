"""The bf16 product of rows grouped by expert and its gradients, against their
definitions in 64 bits.

Whole numbers: with operands in -3 .. 3 every sum is a whole number below 2^24,
so fp32 results are exact whatever the order, and tests of sizes, tails and
offsets ask for equal values.  With random operands:
 * a sum of k products: the matrix instruction adds 8 products at a time at
   worst, each addition off by 2^-23 of the magnitudes; a split sum adds 32 more:
   (k / 8 + 48) 2^-23 of the sum of magnitudes;
 * activations and their slopes: under 32 roundings of 2^-24 of their largest
   intermediate; erfc's argument is off by 2 roundings, which |z phi(z)| <= 0.25
   passes on at 2 z^2 <= 2 ln(1/Phi) of the value;
 * half a step of the output's type.
"""
import math

import numpy as np
import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_moe_dispatch_amd as mep  # noqa: E402

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
KIND = {BF16: mep.MOE_BF16, F32: mep.MOE_FP32}
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
ACTS = ["none", "relu", "gelu", "silu", "swiglu"]


def gen(*key):
    g = torch.Generator(device=DEV)
    g.manual_seed(hash(key) & 0x7FFFFFFF)
    return g


def whole(g, *shape, most=3):
    return torch.randint(-most, most + 1, shape, generator=g, device=DEV).to(BF16)


def randn(g, *shape, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device=DEV)).to(BF16)


def bounds(rows, E, key=0):
    """Ragged rows per expert, some experts without any."""
    r = np.random.default_rng([13, rows, E, key])
    p = r.random(E) ** 3 * (r.random(E) < 0.8) + 1e-9
    return [0] + np.cumsum(r.multinomial(rows, p / p.sum())).tolist()


def space(rows, E, n, k):
    return torch.empty(mep.moe_expert_linear_workspace(rows, E, n, k), dtype=torch.uint8, device=DEV)


def offsets(b):
    return torch.tensor(b, dtype=torch.int32, device=DEV)


def per_row(b, rows):
    """The expert of each row."""
    return torch.repeat_interleave(torch.arange(len(b) - 1, device=DEV), torch.tensor(np.diff(b), device=DEV))


def grouped(x, w, b, fn):
    """fn(rows of x, w[e]) of every expert, rows in order."""
    return torch.cat([fn(x[b[e]:b[e + 1]].double(), w[e].double()) for e in range(len(b) - 1)])


SIZES = [  # rows, E, n, k
    (1, 1, 8, 8), (1, 1, 256, 7168), (5, 3, 24, 40), (16, 1, 136, 64), (17, 2, 264, 72), (33, 1, 1000, 392),
    (37, 8, 1000, 392), (64, 4, 128, 128), (100, 100, 64, 48), (128, 1, 256, 7168), (129, 2, 520, 1032),
    (200, 1, 8, 2048), (257, 1, 2048, 264), (300, 5, 384, 1000), (700, 3, 776, 520), (1000, 7, 8, 8),
    (1500, 300, 72, 136), (2000, 2, 1024, 512), (4100, 1, 264, 96), (2048, 4, 1024, 1024)]


@pytest.mark.parametrize("rows,E,n,k", SIZES)
def test_sizes(rows, E, n, k):
    """All three products on whole numbers: equal values, neighbours untouched."""
    say(f"[gpu] linear rows={rows} E={E} n={n} k={k}")
    g = gen(1, rows, E, n, k)
    b = bounds(rows, E)
    room = rows + 3
    x, dz, w = whole(g, room, k), whole(g, room, n), whole(g, E, n, k)
    x[rows:] = float("nan")                          # rows behind the last expert's are not read
    dz[rows:] = float("nan")
    bias, res = whole(g, E, n), whole(g, room, n)
    ws = space(room, E, n, k)
    off, e = offsets(b), per_row(b, rows)
    y = torch.full((room, n), 9.0, device=DEV)
    z = torch.full((room, n), 9.0, device=DEV, dtype=BF16)
    mep.moe_expert_linear(room, E, n, k, x, off, w, bias, 0, res, z, y, mep.MOE_FP32, ws)
    s = grouped(x, w, b, lambda a, v: a @ v.T) + bias.double()[e]
    assert torch.equal(y[:rows].double(), s + res[:rows].double()) and bool((y[rows:] == 9).all())
    assert torch.equal(z[:rows], s.to(BF16)) and bool((z[rows:] == 9).all())
    dx = torch.full((room, k), 9.0, device=DEV)
    rx = whole(g, room, k)
    mep.moe_expert_linear_grad_input(room, E, n, k, dz, off, w, 0, None, rx, dx, mep.MOE_FP32, ws)
    assert torch.equal(dx[:rows].double(), grouped(dz, w, b, lambda a, v: a @ v) + rx[:rows].double())
    assert bool((dx[rows:] == 9).all())
    dw, db = torch.full((E, n, k), 9.0, device=DEV), torch.full((E, n), 9.0, device=DEV)
    mep.moe_expert_linear_grad_weight(room, E, n, k, dz, x, off, dw, mep.MOE_FP32, db, ws)
    for i in range(E):
        d, a = dz[b[i]:b[i + 1]].double(), x[b[i]:b[i + 1]].double()
        assert torch.equal(dw[i].double(), d.T @ a), i
        assert torch.equal(db[i].double(), d.sum(0)), i
    # without the bias' gradient, in bf16: the same sums rounded
    dw2 = torch.full((E, n, k), 9.0, device=DEV, dtype=BF16)
    mep.moe_expert_linear_grad_weight(room, E, n, k, dz, x, off, dw2, mep.MOE_BF16, None, ws)
    assert torch.equal(dw2, dw.to(BF16))


@pytest.mark.parametrize("rows,n,k", [(1, 64, 64), (40, 72, 200), (500, 264, 136), (3000, 512, 256)])
def test_without_offsets(rows, n, k):
    """One expert with all rows: offsets may be left out."""
    say(f"[gpu] linear without offsets rows={rows} n={n} k={k}")
    g = gen(2, rows, n, k)
    x, dz, w, ws = whole(g, rows, k), whole(g, rows, n), whole(g, 1, n, k), space(rows, 1, n, k)
    y, dx, dw = (torch.full(s, 9.0, device=DEV) for s in ((rows, n), (rows, k), (1, n, k)))
    mep.moe_expert_linear(rows, 1, n, k, x, None, w, None, 0, None, None, y, mep.MOE_FP32, ws)
    mep.moe_expert_linear_grad_input(rows, 1, n, k, dz, None, w, 0, None, None, dx, mep.MOE_FP32, ws)
    mep.moe_expert_linear_grad_weight(rows, 1, n, k, dz, x, None, dw, mep.MOE_FP32, None, ws)
    assert torch.equal(y.double(), x.double() @ w[0].double().T)
    assert torch.equal(dx.double(), dz.double() @ w[0].double())
    assert torch.equal(dw[0].double(), dz.double().T @ x.double())


def value64(name, z):
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        return g * torch.sigmoid(g) * u
    return {"none": lambda v: v, "relu": lambda v: v.clamp_min(0), "silu": lambda v: v * torch.sigmoid(v),
            "gelu": lambda v: v * torch.special.ndtr(v)}[name](z)


def slope64(name, z):
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    return (z > 0).double() if name == "relu" else torch.ones_like(z)


def through64(name, z, d):
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        return torch.cat([d * u * slope64("silu", g), d * value64("silu", g)], -1)
    return d * slope64(name, z)


def sum_error(big, k):
    return (k / 8 + 48) * 2.0 ** -23 * big


EPI = 64 * 2.0 ** -24


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,E,n,k", [(37, 8, 1008, 392), (700, 2, 272, 520), (9, 1, 256, 4096), (300, 1, 528, 64)])
@pytest.mark.parametrize("kind", [BF16, F32], ids=["bf16", "fp32"])
def test_forward(rows, E, n, k, act, kind):
    say(f"[gpu] linear forward rows={rows} E={E} n={n} k={k} {act} {kind}")
    g = gen(3, rows, E, n, k)
    b = bounds(rows, E)
    e = per_row(b, rows)
    x, w, bias = randn(g, rows, k), randn(g, E, n, k, scale=k ** -0.5), randn(g, E, n)
    m = n // 2 if act == "swiglu" else n
    res, ws = randn(g, rows, m), space(rows, E, n, k)
    z64 = grouped(x, w, b, lambda a, v: a @ v.T) + bias.double()[e]
    err = sum_error(grouped(x.abs(), w.abs(), b, lambda a, v: a @ v.T) + bias.double()[e].abs(), k)
    want = value64(act, z64)
    # slopes are below 1.13; of silu(g) u: 1.1 |u| and 1 |g|
    if act == "swiglu":
        (eg, eu), (zg, zu) = err.chunk(2, -1), z64.chunk(2, -1)
        bound = 1.13 * (eg * (zu.abs() + eu) + eu * (zg.abs() + eg)) + EPI * (want.abs() + 1e-3)
    else:
        bound = 1.13 * err + EPI * (want.abs() + 1e-3)
    for r in (None, res):
        y = torch.empty((rows, m), device=DEV, dtype=kind)
        z = torch.empty((rows, n), device=DEV, dtype=BF16)
        mep.moe_expert_linear(rows, E, n, k, x, offsets(b), w, bias, ACTS.index(act), r, z, y, KIND[kind], ws)
        ref = want if r is None else want + r.double()
        lim = bound + 2.0 ** -24 * ref.abs()
        assert bool(((y.double() - ref).abs() <= lim + HALF[kind] * (ref.abs() + lim)).all())
        assert bool(((z.double() - z64).abs() <= err + HALF[BF16] * (z64.abs() + err)).all())
        y2 = torch.empty_like(y)                     # the result does not depend on z being kept
        mep.moe_expert_linear(rows, E, n, k, x, offsets(b), w, bias, ACTS.index(act), r, None, y2, KIND[kind], ws)
        assert torch.equal(y, y2)
    if kind == BF16:                                 # y over the residual
        mep.moe_expert_linear(rows, E, n, k, x, offsets(b), w, bias, ACTS.index(act), res, None, res, KIND[kind], ws)
        assert torch.equal(res, y)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,E,n,k", [(37, 8, 392, 1000), (700, 2, 520, 264), (9, 1, 4096, 256), (300, 1, 64, 528)])
@pytest.mark.parametrize("kind", [BF16, F32], ids=["bf16", "fp32"])
def test_grad_input(rows, E, n, k, act, kind):
    say(f"[gpu] linear gradient to the input rows={rows} E={E} n={n} k={k} {act} {kind}")
    g = gen(4, rows, E, n, k)
    b = bounds(rows, E)
    dz, w = randn(g, rows, n), randn(g, E, n, k, scale=n ** -0.5)
    m = 2 * k if act == "swiglu" else k
    z = None if act == "none" else randn(g, rows, m, scale=2.0)
    res, ws = randn(g, rows, m), space(rows, E, n, k)
    d64 = grouped(dz, w, b, lambda a, v: a @ v)
    err = sum_error(grouped(dz.abs(), w.abs(), b, lambda a, v: a @ v), n)
    if act == "none":
        want, bound = d64, err
    else:
        want = through64(act, z.double(), d64)
        each = d64.abs().repeat(1, m // k)
        most = torch.cat([1.13 * z[:, k:].abs(), z[:, :k].abs()], 1).double() if act == "swiglu" else 1.13
        bound = most * (err.repeat(1, m // k) + EPI * each) + EPI * want.abs()
    for r in (None, res):
        dx = torch.empty((rows, m), device=DEV, dtype=kind)
        mep.moe_expert_linear_grad_input(rows, E, n, k, dz, offsets(b), w, ACTS.index(act), z, r, dx, KIND[kind], ws)
        ref = want if r is None else want + r.double()
        lim = bound + 2.0 ** -24 * ref.abs()
        assert bool(((dx.double() - ref).abs() <= lim + HALF[kind] * (ref.abs() + lim)).all())
    if kind == BF16:
        mep.moe_expert_linear_grad_input(rows, E, n, k, dz, offsets(b), w, ACTS.index(act), z, res, res, KIND[kind], ws)
        assert torch.equal(res, dx)


@pytest.mark.parametrize("rows,E,n,k", [(3000, 2, 136, 264), (500, 6, 520, 200), (2500, 1, 64, 1000)])
def test_grad_weight(rows, E, n, k):
    say(f"[gpu] linear gradient to the weights rows={rows} E={E} n={n} k={k}")
    g = gen(5, rows, E, n, k)
    b = bounds(rows, E)
    dz, x, ws = randn(g, rows, n), randn(g, rows, k), space(rows, E, n, k)
    dw, db = torch.empty((E, n, k), device=DEV), torch.empty((E, n), device=DEV)
    mep.moe_expert_linear_grad_weight(rows, E, n, k, dz, x, offsets(b), dw, mep.MOE_FP32, db, ws)
    for e in range(E):
        d, a = dz[b[e]:b[e + 1]].double(), x[b[e]:b[e + 1]].double()
        t = b[e + 1] - b[e]
        assert bool(((dw[e].double() - d.T @ a).abs() <= sum_error(d.abs().T @ a.abs(), t)).all())
        assert bool(((db[e].double() - d.sum(0)).abs() <= sum_error(d.abs().sum(0), t)).all())
    again = torch.empty_like(dw)
    mep.moe_expert_linear_grad_weight(rows, E, n, k, dz, x, offsets(b), again, mep.MOE_FP32, None, ws)
    assert torch.equal(dw, again)


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("rows,E,n", [(1, 1, 16), (37, 8, 1008), (300, 3, 4096)])
def test_activation_grad(rows, E, n, act):
    say(f"[gpu] activation gradient rows={rows} E={E} n={n} {act}")
    g = gen(6, rows, E, n)
    room, m = rows + 2, n // 2 if act == "swiglu" else n
    off = offsets(bounds(rows, E))
    z, dy = randn(g, room, n, scale=3.0), randn(g, room, m)
    dz = torch.full((room, n), 9.0, device=DEV, dtype=BF16)
    mep.moe_activation_grad(room, E, n, ACTS.index(act), off, z, dy, dz)
    want = through64(act, z.double(), dy.double())
    each = dy.double().abs().repeat(1, n // m)
    if act == "swiglu":
        each = each * torch.cat([z[:, m:], z[:, :m]], 1).double().abs()
    lim = EPI * 1.13 * each
    ok = (dz.double() - want).abs() <= lim + HALF[BF16] * (want.abs() + lim)
    assert bool(ok[:rows].all()) and bool((dz[rows:] == 9).all())
    # over z; over dy where it has its shape
    z2 = z.clone()
    mep.moe_activation_grad(room, E, n, ACTS.index(act), off, z2, dy, z2)
    assert torch.equal(z2[:rows], dz[:rows]) and torch.equal(z2[rows:], z[rows:])
    if act != "swiglu":
        mep.moe_activation_grad(room, E, n, ACTS.index(act), off, z, dy, dy)
        assert torch.equal(dy[:rows], dz[:rows])


@pytest.mark.parametrize("act", ACTS[1:])
def test_activations_over_the_range(act):
    """Every finite bf16 from -200 to 200 through the forward epilogue (x = 1, w = z) and the
    slope: far tails, zero, the smallest numbers."""
    say(f"[gpu] activations over the range, {act}")
    bits = torch.arange(1 << 16, device=DEV, dtype=torch.int32).to(torch.int16)
    z = bits.view(BF16)
    z = z[torch.isfinite(z.float()) & (z.float().abs() <= 200)]
    z = torch.cat([z, torch.zeros(-z.numel() % 16, device=DEV, dtype=BF16)])
    n = z.numel() // 2 // 8 * 8
    for v in (z[:n], z[n:2 * n]):
        w = torch.zeros((1, n, 8), device=DEV, dtype=BF16)
        w[0, :, 0] = v
        x = torch.zeros((1, 8), device=DEV, dtype=BF16)
        x[0, 0] = 1
        name = act
        if act == "swiglu":                          # gate v, up 1
            up = torch.zeros_like(w)
            up[0, :, 0] = 1
            w, name = torch.cat([w, up], 1), "silu"
        N = w.shape[1]
        y = torch.empty((1, n), device=DEV)
        mep.moe_expert_linear(1, 1, N, 8, x, None, w, None, ACTS.index(act), None, None, y, mep.MOE_FP32, space(1, 1, N, 8))
        v64 = v.double()
        want = value64(name, v64)
        if name == "gelu":
            want = v64 * 0.5 * torch.special.erfc(-v64 * math.sqrt(0.5))
        # results below the normal numbers may be zero
        lim = (32 + 4 * (v64 ** 2 if name == "gelu" else 0)) * 2.0 ** -24 * want.abs() + 2.0 ** -117
        assert bool(((y[0].double() - want).abs() <= lim).all())
        if act != "swiglu":
            one = torch.ones((1, n), device=DEV, dtype=BF16)
            dz = torch.empty((1, n), device=DEV, dtype=BF16)
            mep.moe_activation_grad(1, 1, n, ACTS.index(act), None, v[None].contiguous(), one, dz)
            want = slope64(name, v64)
            assert bool(((dz[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + EPI).all())


@pytest.mark.parametrize("act", ACTS)
def test_gradients_by_differences(act):
    """The formulas in 64 bits against central differences of the layer, step 1e-5: off by some
    1e-10 of third derivatives below 1e3 and by 2^-52 / 1e-5 of a loss below 1e3; no sum lies
    so near to relu's kink.  The device's numbers against the formulas: z's rounding passes
    through a slope of at most 0.8 (gelu''(0)), then dz is rounded, then the sums of products."""
    say(f"[gpu] linear gradients by differences, {act}")
    rows, E, n, k, h = 7, 2, 16, 24, 1e-5
    g = gen(7)
    b = [0, 4, 7]
    x, w, bias = randn(g, rows, k), randn(g, E, n, k, scale=0.3), randn(g, E, n, scale=0.3)
    m = n // 2 if act == "swiglu" else n
    dy = randn(g, rows, m)
    e = per_row(b, rows)

    def sums(x, w, bias):
        return torch.cat([x[b[i]:b[i + 1]] @ w[i].T + bias[i] for i in range(E)])

    par = [x.double(), w.double(), bias.double()]
    z64 = sums(*par)
    assert float(z64.abs().min()) > 1e-4
    dz64 = through64(act, z64, dy.double())
    grads = [grouped(dz64, w, b, lambda a, v: a @ v),
             torch.stack([dz64[b[i]:b[i + 1]].T @ par[0][b[i]:b[i + 1]] for i in range(E)]),
             torch.stack([dz64[b[i]:b[i + 1]].sum(0) for i in range(E)])]
    for i, grad in enumerate(grads):
        for at in range(grad.numel()):
            ends = []
            for sign in (1, -1):
                q = list(par)
                q[i] = par[i].clone()
                q[i].view(-1)[at] += sign * h
                ends.append((value64(act, sums(*q)) * dy.double()).sum())
            assert abs(float((ends[0] - ends[1]) / (2 * h) - grad.reshape(-1)[at])) <= 1e-6
    # the device
    z, y = torch.empty((rows, n), device=DEV, dtype=BF16), torch.empty((rows, m), device=DEV)
    ws = space(rows, E, n, k)
    mep.moe_expert_linear(rows, E, n, k, x, offsets(b), w, bias, ACTS.index(act), None, z, y, mep.MOE_FP32, ws)
    dz, err = dy, 0.0 * dy.double()
    if act != "none":
        dz = torch.empty((rows, n), device=DEV, dtype=BF16)
        mep.moe_activation_grad(rows, E, n, ACTS.index(act), offsets(b), z, dy, dz)
        ez = HALF[BF16] * z64.abs() + sum_error(grouped(x.abs(), w.abs(), b, lambda a, v: a @ v.T) + bias.double()[e].abs(), k)
        each = dy.double().abs().repeat(1, n // m)
        err = 0.8 * ez * each
        if act == "swiglu":                          # d u silu'(g), d silu(g)
            (eg, eu), (zg, zu) = ez.chunk(2, -1), z64.chunk(2, -1)
            d = dy.double().abs().repeat(1, 2)
            err = d * torch.cat([0.5 * eg * (zu.abs() + eu) + 1.1 * eu, 1.1 * eg], -1)
            each = d * (1 + torch.cat([zu, zg], -1).abs() + torch.cat([eu, eg], -1))
        if act == "relu":
            err = torch.zeros_like(err)
        err = err + EPI * 1.13 * each
        err = err + HALF[BF16] * (dz64.abs() + err)
        assert bool(((dz.double() - dz64).abs() <= err).all())
    dx, dw, db = (torch.empty(s, device=DEV) for s in ((rows, k), (E, n, k), (E, n)))
    mep.moe_expert_linear_grad_input(rows, E, n, k, dz, offsets(b), w, 0, None, None, dx, mep.MOE_FP32, ws)
    mep.moe_expert_linear_grad_weight(rows, E, n, k, dz, x, offsets(b), dw, mep.MOE_FP32, db, ws)
    big = dz64.abs() + err
    off = [grouped(err, w.abs(), b, lambda a, v: a @ v) + sum_error(grouped(big, w.abs(), b, lambda a, v: a @ v), n)]
    for fn in (lambda d, a: d.T @ a, lambda d, a: d.sum(0)):
        part = [(err[b[i]:b[i + 1]], big[b[i]:b[i + 1]], x[b[i]:b[i + 1]].double().abs()) for i in range(E)]
        off.append(torch.stack([fn(p, a) + sum_error(fn(q, a), len(a)) for p, q, a in part]))
    for got, want, lim in zip((dx, dw, db), grads, off):
        assert bool(((got.double() - want).abs() <= lim).all())


def test_rows_do_not_meet():
    """NaN and infinite rows stay with themselves; masks of the type's lowest value pass."""
    say("[gpu] linear: NaN rows stay with themselves")
    rows, E, n, k = 200, 3, 264, 136
    g = gen(8)
    b = [0, 70, 70, 200]
    x, w, ws = whole(g, rows, k), whole(g, E, n, k), space(rows, E, n, k)
    clean, y = (torch.empty((rows, n), device=DEV) for _ in range(2))
    mep.moe_expert_linear(rows, E, n, k, x, offsets(b), w, None, 0, None, None, clean, mep.MOE_FP32, ws)
    bad = [0, 69, 70, 128, 199]
    x[bad] = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(BF16).min, float("nan")],
                          device=DEV, dtype=BF16)[:, None]
    mep.moe_expert_linear(rows, E, n, k, x, offsets(b), w, None, 0, None, None, y, mep.MOE_FP32, ws)
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[bad] = False
    assert torch.equal(y[keep], clean[keep]) and not bool(torch.isfinite(y[[0, 69, 70, 199]]).all())
    # expert 0's NaN rows spoil expert 0's weights alone
    dz, dw = whole(g, rows, n), torch.empty((E, n, k), device=DEV)
    x[bad[2:]] = 0
    mep.moe_expert_linear_grad_weight(rows, E, n, k, dz, x, offsets(b), dw, mep.MOE_FP32, None, ws)
    assert torch.isnan(dw[0]).any() and bool((dw[1] == 0).all())
    assert torch.equal(dw[2].double(), dz[70:].double().T @ x[70:].double())


def test_no_rows():
    say("[gpu] linear gradient to the weights without rows")
    dw, db = torch.full((2, 24, 40), 9.0, device=DEV), torch.full((2, 24), 9.0, device=DEV)
    mep.moe_expert_linear_grad_weight(0, 2, 24, 40, None, None, None, dw, mep.MOE_FP32, db)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_offsets_out_of_order():
    """Offsets that break their order stay inside the tensors."""
    say("[gpu] linear: offsets out of order stay inside")
    rows, E, n, k = 300, 4, 136, 72
    g = gen(9)
    x, dz, w, ws = whole(g, rows, k), whole(g, rows, n), whole(g, E, n, k), space(rows, E, n, k)
    guard = 64
    for off in ([0, 500, 100, 90, 400], [-5, 10, 2 ** 31 - 1, -2 ** 31, 300], [300, 200, 100, 50, 0], [0, 0, 0, 0, 2 ** 30]):
        y, dx = (torch.full((rows + guard, m), 9.0, device=DEV) for m in (n, k))
        dw = torch.full((E + 1, n, k), 9.0, device=DEV)
        mep.moe_expert_linear(rows, E, n, k, x, offsets(off), w, None, 0, None, None, y, mep.MOE_FP32, ws)
        mep.moe_expert_linear_grad_input(rows, E, n, k, dz, offsets(off), w, 0, None, None, dx, mep.MOE_FP32, ws)
        mep.moe_expert_linear_grad_weight(rows, E, n, k, dz, x, offsets(off), dw, mep.MOE_FP32, None, ws)
        torch.cuda.synchronize()
        for t in (y[rows:], dx[rows:], dw[E:]):
            assert bool((t == 9).all())



# (tile, splits, product / to the input / to the weights / in fp32, gated, rows, E, n, k): every tile with
# and without splits, long enough for its steady loop, most with a tail and ragged experts
FORMS = [
    ("128 x 128", 1, 0, 0, 2746, 3, 1328, 456), ("128 x 128", 8, 0, 0, 4287, 5, 16, 3800),
    ("128 x 128", 1, 0, 1, 4356, 3, 784, 592), ("128 x 128", 8, 0, 1, 3735, 5, 16, 3664),
    ("128 x 128", 1, 1, 0, 1536, 16, 464, 2856), ("128 x 128", 8, 1, 0, 4621, 2, 3696, 8),
    ("128 x 128", 1, 2, 0, 3752, 8, 2288, 136), ("128 x 128", 1, 3, 0, 2286, 5, 3888, 136),
    ("128 x 256", 1, 0, 0, 4009, 3, 960, 480), ("128 x 256", 8, 0, 0, 1794, 16, 144, 4776),
    ("128 x 256", 1, 0, 1, 4015, 2, 912, 464), ("128 x 256", 8, 0, 1, 2803, 1, 144, 4976),
    ("128 x 256", 1, 1, 0, 3646, 8, 464, 912), ("128 x 256", 4, 1, 0, 4219, 5, 3808, 160),
    ("128 x 256", 1, 2, 0, 2801, 5, 3760, 136), ("128 x 256", 1, 3, 0, 3056, 5, 3360, 152),
    ("128 x 256", 4, 3, 0, 3717, 1, 3440, 272), ("256 x 256", 1, 0, 0, 3800, 8, 2000, 464),
    ("256 x 256", 1, 0, 1, 4255, 3, 1680, 544), ("256 x 256", 1, 1, 0, 1607, 2, 480, 4880),
    ("256 x 256", 1, 2, 0, 3794, 8, 2752, 312), ("256 x 256", 1, 3, 0, 3635, 8, 2976, 264),
    ("32 x 128", 1, 0, 0, 8, 2, 16, 456), ("32 x 128", 8, 0, 0, 15, 2, 16, 3696),
    ("32 x 128", 1, 0, 1, 10, 2, 16, 456), ("32 x 128", 8, 0, 1, 18, 2, 16, 3664),
    ("32 x 128", 1, 1, 0, 12, 2, 464, 8), ("32 x 128", 8, 1, 0, 9, 2, 3888, 8), ("32 x 128", 1, 2, 0, 926, 2, 16, 8),
    ("32 x 128", 4, 2, 0, 3903, 2, 1136, 8), ("32 x 128", 1, 3, 0, 907, 2, 16, 8),
    ("32 x 128", 4, 3, 0, 3632, 2, 1056, 8), ("32 x 256", 1, 0, 0, 469, 16, 3904, 488),
    ("32 x 256", 1, 0, 1, 96, 16, 4048, 496), ("32 x 256", 1, 1, 0, 34, 16, 464, 4168),
    ("32 x 256", 1, 2, 0, 3941, 8, 80, 4512), ("32 x 256", 1, 3, 0, 3939, 8, 80, 4992),
    ("64 x 128", 1, 0, 0, 4172, 8, 160, 776), ("64 x 128", 8, 0, 0, 2129, 2, 16, 3808),
    ("64 x 128", 1, 0, 1, 4606, 2, 144, 728), ("64 x 128", 4, 0, 1, 3981, 2, 16, 1808),
    ("64 x 128", 1, 1, 0, 4550, 2, 752, 144), ("64 x 128", 4, 1, 0, 3858, 5, 1840, 8),
    ("64 x 128", 1, 2, 0, 3692, 8, 2128, 8), ("64 x 128", 8, 2, 0, 3896, 1, 2240, 8),
    ("64 x 128", 1, 3, 0, 2481, 5, 3488, 8), ("64 x 128", 4, 3, 0, 4476, 2, 3200, 8),
    ("few rows", 1, 2, 0, 30, 8, 2048, 1032), ("few rows", 1, 3, 0, 19, 5, 4096, 1000),
    ("few rows", 1, 2, 0, 3, 1, 4104, 4096), ("few rows", 1, 3, 0, 3, 1, 4104, 4096)]


@pytest.mark.parametrize("last", [1, 127, 128, 129, 255])
def test_last_rows(last):
    """Experts whose last rows take half a 256 x 256 tile, beside ones that take all of it, and
    weight rows alike."""
    say(f"[gpu] linear last rows {last}")
    b = [0]
    for r in (1280 + last, 1536, last, 0, 1024 + last):
        b.append(b[-1] + r)
    rows, E, sum_ = b[-1], 5, 1160
    g = gen(11, last)
    off, a = offsets(b), whole(g, rows, sum_)

    def width(kind, gated):                          # one that takes the tile, odd too
        for c in range(1800 + last // 8 * 8, 9000, 256):
            n, k = (sum_, c) if kind == 1 else (c - c % 16, sum_)
            if form_of(kind, gated, rows, E, n, k) == ("256 x 256", 1):
                return n, k
        raise AssertionError("no such width")

    n, k = width(0, 0)
    w, ws = whole(g, E, n, k), space(rows, E, n, k)
    s = grouped(a, w, b, lambda u, v: u @ v.T)
    for kind in (BF16, F32):
        y = torch.empty((rows, n), device=DEV, dtype=kind)
        mep.moe_expert_linear(rows, E, n, k, a, off, w, None, 0, None, None, y, KIND[kind], ws)
        assert torch.equal(y, s.to(kind))
    n, k = width(0, 1)
    w, ws = whole(g, E, n, k), space(rows, E, n, k)
    s = grouped(a, w, b, lambda u, v: u @ v.T)
    z, y = torch.empty((rows, n), device=DEV, dtype=BF16), torch.empty((rows, n // 2), device=DEV, dtype=BF16)
    mep.moe_expert_linear(rows, E, n, k, a, off, w, None, 4, None, z, y, mep.MOE_BF16, ws)
    want = value64("swiglu", s)
    assert torch.equal(z, s.to(BF16))
    assert bool(((y.double() - want).abs() <= (HALF[BF16] + EPI) * want.abs() + 1e-30).all())
    n, k = width(1, 0)
    w, ws = whole(g, E, n, k), space(rows, E, n, k)
    s = grouped(a, w, b, lambda u, v: u @ v)
    for kind in (BF16, F32):
        dx = torch.empty((rows, k), device=DEV, dtype=kind)
        mep.moe_expert_linear_grad_input(rows, E, n, k, a, off, w, 0, None, None, dx, KIND[kind], ws)
        assert torch.equal(dx, s.to(kind))
    n, k = width(2, 0)
    dz, ws = whole(g, rows, n), space(rows, E, n, k)
    for bias in (True, False):
        dw, db = torch.empty((E, n, k), device=DEV, dtype=BF16), torch.empty((E, n), device=DEV)
        mep.moe_expert_linear_grad_weight(rows, E, n, k, dz, a, off, dw, mep.MOE_BF16, db if bias else None, ws)
        for e in range(E):
            d, x = dz[b[e]:b[e + 1]].double(), a[b[e]:b[e + 1]].double()
            assert torch.equal(dw[e], (d.T @ x).to(BF16)), e
            assert not bias or torch.equal(db[e].double(), d.sum(0)), e


def form_of(kind, gated, rows, E, n, k):
    import ctypes
    splits = ctypes.c_int32(0)
    fn = mep._lib.moe_ops_linear_form
    fn.argtypes, fn.restype = [ctypes.c_int32] * 6 + [ctypes.POINTER(ctypes.c_int32)], ctypes.c_char_p
    return fn(kind, gated, rows, E, n, k, ctypes.byref(splits)).decode(), splits.value


@pytest.mark.parametrize("form,splits,kind,gated,rows,E,n,k", FORMS)
def test_forms(form, splits, kind, gated, rows, E, n, k):
    """Every tile and split on whole numbers, asked of the library by its name."""
    say(f"[gpu] linear form {form} splits={splits} kind={kind} gated={gated} rows={rows} E={E} n={n} k={k}")
    assert form_of(kind, gated, rows, E, n, k) == (form, splits)
    g = gen(10, kind, gated, rows, E, n, k)
    r = np.random.default_rng([17, rows, E])
    b = [0] + np.cumsum(r.multinomial(rows - 3, r.dirichlet(np.full(E, 4.0)))).tolist()
    used = b[-1]                                     # three rows behind the last expert's
    off = offsets(b)
    x, dz, w, ws = whole(g, rows, k), whole(g, rows, n), whole(g, E, n, k), space(rows, E, n, k)
    x[used:] = dz[used:] = float("nan")
    if kind == 0 and gated:
        z, y = torch.full((rows, n), 9.0, device=DEV, dtype=BF16), torch.full((rows, n // 2), 9.0, device=DEV, dtype=BF16)
        mep.moe_expert_linear(rows, E, n, k, x, off, w, None, 4, None, z, y, mep.MOE_BF16, ws)
        s = grouped(x, w, b, lambda a, v: a @ v.T)
        assert torch.equal(z[:used], s.to(BF16)) and bool((z[used:] == 9).all()) and bool((y[used:] == 9).all())
        want = value64("swiglu", s)
        assert bool(((y[:used].double() - want).abs() <= (HALF[BF16] + EPI) * want.abs() + 1e-30).all())
    elif kind == 0:
        y = torch.full((rows, n), 9.0, device=DEV)
        mep.moe_expert_linear(rows, E, n, k, x, off, w, None, 0, None, None, y, mep.MOE_FP32, ws)
        assert torch.equal(y[:used].double(), grouped(x, w, b, lambda a, v: a @ v.T)) and bool((y[used:] == 9).all())
    elif kind == 1:
        dx = torch.full((rows, k), 9.0, device=DEV)
        mep.moe_expert_linear_grad_input(rows, E, n, k, dz, off, w, 0, None, None, dx, mep.MOE_FP32, ws)
        assert torch.equal(dx[:used].double(), grouped(dz, w, b, lambda a, v: a @ v)) and bool((dx[used:] == 9).all())
    else:
        for bias in (True, False):
            out = F32 if kind == 3 else BF16
            dw, db = torch.full((E, n, k), 9.0, device=DEV, dtype=out), torch.full((E, n), 9.0, device=DEV)
            mep.moe_expert_linear_grad_weight(rows, E, n, k, dz, x, off, dw, KIND[out], db if bias else None, ws)
            for e in range(E):
                d, a = dz[b[e]:b[e + 1]].double(), x[b[e]:b[e + 1]].double()
                assert torch.equal(dw[e], (d.T @ a).to(out)), e
                assert not bias or torch.equal(db[e].double(), d.sum(0)), e
