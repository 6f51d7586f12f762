"""An expert layer on one card as a user runs it: router, routing, rows sorted by
expert, both products, rows back, a shared expert beside them, and everything
backwards; captured, on several streams, and with e4m3 rows.

Every number is checked against its formula in 64 bits, from the numbers that the
device rounded and kept before it (so that bounds do not pile up); the reference
carries a value and a bound on how far the device's may be off:
 * a rounding to bf16 adds 2^-8 of the value, one to fp32 2^-24;
 * a sum of k products adds (k / 8 + 48) 2^-23 of its magnitudes (the matrix
   instruction's and the split sums' additions), and passes on the errors of its
   factors: |a| eb + ea |b| + ea eb;
 * silu has a slope of at most 1.1, its slope one of 0.5; with their evaluation
   64 roundings of 2^-24 of values that stay below 1.1 |z| + 0.28 and 1.1;
 * a softmax over logits off by d is off by a factor of exp(2 d) and 64 roundings.
"""
import numpy as np
import pytest

from tests import ops_ref as R
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_moe_dispatch_amd as mep  # noqa: E402

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
SWIGLU, NONE = mep.MOE_ACT_SWIGLU, mep.MOE_ACT_NONE


def empty(*shape, dt=F32):
    return torch.empty(shape, dtype=dt, device=DEV)


class Layer:
    """T tokens, the last `pad` of them padding, E experts and a shared one of width F."""

    def __init__(self, T, H, E, K, F, pad=0, seed=0, renorm=True):
        self.dims, self.pad, self.renorm = (T, H, E, K, F), pad, renorm
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        r = lambda *s, by=1.0: (by * torch.randn(s, generator=g, device=DEV)).to(BF16)  # noqa: E731
        self.x, self.dout = r(T, H), r(T, H)
        self.wr = r(1, E, H, by=2 * H ** -0.5)
        self.w1, self.b1 = r(E, 2 * F, H, by=H ** -0.5), r(E, 2 * F, by=0.1)
        self.w2, self.b2 = r(E, H, F, by=F ** -0.5), r(E, H, by=0.1)
        self.s1, self.s2 = r(1, 2 * F, H, by=H ** -0.5), r(1, H, F, by=F ** -0.5)
        rows = self.rows = T * K
        self.logits, self.idx, self.w = empty(T, E), empty(T, K, dt=torch.int32), empty(T, K)
        self.off, self.slot = empty(E + 1, dt=torch.int32), empty(T, K, dt=torch.int32)
        self.xs, self.z, self.h = empty(rows, H, dt=BF16), empty(rows, 2 * F, dt=BF16), empty(rows, F, dt=BF16)
        self.y, self.routed = empty(rows, H, dt=BF16), empty(T, H, dt=BF16)
        self.zs, self.hs, self.out = empty(T, 2 * F, dt=BF16), empty(T, F, dt=BF16), empty(T, H, dt=BF16)
        self.dy, self.dw = empty(rows, H, dt=BF16), empty(T, K)
        self.dz, self.dxs = empty(rows, 2 * F, dt=BF16), empty(rows, H, dt=BF16)
        self.dzs, self.dx = empty(T, 2 * F, dt=BF16), empty(T, H, dt=BF16)
        self.dlogits = empty(T, E, dt=BF16)
        self.dw1, self.db1, self.dw2, self.db2 = (empty(*t.shape) for t in (self.w1, self.b1, self.w2, self.b2))
        self.dwr, self.ds1, self.ds2 = (empty(*t.shape) for t in (self.wr, self.s1, self.s2))
        most = max(mep.moe_sort_workspace(T, E, K), *(mep.moe_expert_linear_workspace(*s) for s in (
            (T, 1, E, H), (rows, E, 2 * F, H), (rows, E, H, F), (T, 1, 2 * F, H), (T, 1, H, F))))
        self.ws = empty(max(1, most), dt=torch.uint8)

    def run(self, stream=None):
        T, H, E, K, F = self.dims
        rows, ws, B, W = self.rows, self.ws, mep.MOE_BF16, mep.MOE_FP32
        s = dict(stream=stream)
        mep.moe_expert_linear(T, 1, E, H, self.x, None, self.wr, None, NONE, None, None, self.logits, W, ws, **s)
        mep.moe_topk_route(T, E, K, self.logits, W, self.renorm, self.idx, self.w, **s)
        if self.pad:
            self.idx[T - self.pad:] = -1
        mep.moe_sort_plan(T, E, K, self.idx, self.off, self.slot, None, ws, **s)
        mep.moe_sort_rows(T, K, rows, H, B, self.x, None, self.slot, self.xs, None, **s)
        mep.moe_expert_linear(rows, E, 2 * F, H, self.xs, self.off, self.w1, self.b1, SWIGLU, None, self.z, self.h, B, ws, **s)
        mep.moe_expert_linear(rows, E, H, F, self.h, self.off, self.w2, self.b2, NONE, None, None, self.y, B, ws, **s)
        mep.moe_unsort_rows(T, K, rows, H, B, self.y, self.slot, self.w, self.routed, **s)
        mep.moe_expert_linear(T, 1, 2 * F, H, self.x, None, self.s1, None, SWIGLU, None, self.zs, self.hs, B, ws, **s)
        mep.moe_expert_linear(T, 1, H, F, self.hs, None, self.s2, None, NONE, self.routed, None, self.out, B, ws, **s)
        # backwards
        mep.moe_unsort_rows_grad(T, K, rows, H, B, self.dout, self.y, self.slot, self.w, self.dy, self.dw, **s)
        mep.moe_expert_linear_grad_weight(rows, E, H, F, self.dy, self.h, self.off, self.dw2, W, self.db2, ws, **s)
        mep.moe_expert_linear_grad_input(rows, E, H, F, self.dy, self.off, self.w2, SWIGLU, self.z, None, self.dz, B, ws, **s)
        mep.moe_expert_linear_grad_weight(rows, E, 2 * F, H, self.dz, self.xs, self.off, self.dw1, W, self.db1, ws, **s)
        mep.moe_expert_linear_grad_input(rows, E, 2 * F, H, self.dz, self.off, self.w1, NONE, None, None, self.dxs, B, ws, **s)
        mep.moe_unsort_rows(T, K, rows, H, B, self.dxs, self.slot, None, self.dx, **s)
        mep.moe_expert_linear_grad_weight(T, 1, H, F, self.dout, self.hs, None, self.ds2, W, None, ws, **s)
        mep.moe_expert_linear_grad_input(T, 1, H, F, self.dout, None, self.s2, SWIGLU, self.zs, None, self.dzs, B, ws, **s)
        mep.moe_expert_linear_grad_weight(T, 1, 2 * F, H, self.dzs, self.x, None, self.ds1, W, None, ws, **s)
        mep.moe_expert_linear_grad_input(T, 1, 2 * F, H, self.dzs, None, self.s1, NONE, None, self.dx, self.dx, B, ws, **s)
        mep.moe_topk_route_grad(T, E, K, self.logits, W, self.renorm, self.idx, self.dw, self.dlogits, B, **s)
        mep.moe_expert_linear_grad_weight(T, 1, E, H, self.dlogits, self.x, None, self.dwr, W, None, ws, **s)
        mep.moe_expert_linear_grad_input(T, 1, E, H, self.dlogits, None, self.wr, NONE, None, self.dx, self.dx, B, ws, **s)

    NAMES = ("logits", "idx", "w", "off", "slot", "routed", "out", "dw", "dlogits", "dx", "dw1", "db1", "dw2", "db2",
             "dwr", "ds1", "ds2")
    ROWS = ("xs", "z", "h", "y", "dy", "dz", "dxs")                  # up to the last expert's

    def results(self):
        used = int(self.off[-1])
        return {n: getattr(self, n).clone() for n in self.NAMES} | {n: getattr(self, n)[:used].clone() for n in self.ROWS}

    def spoil(self):
        for n in self.NAMES + self.ROWS:
            t = getattr(self, n)
            t.fill_(float("nan") if t.is_floating_point() else -7)
        self.ws.fill_(0xFF)


def same(a, b):
    return all(torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)) for n in a)


class V:
    """A value in 64 bits and a bound on the device's distance from it."""

    def __init__(self, v, e=None):
        self.v = v.double()
        self.e = torch.zeros_like(self.v) if e is None else e

    def rounded(self, half):
        return V(self.v, self.e + half * (self.v.abs() + self.e))

    def __add__(self, o):
        return V(self.v + o.v, self.e + o.e + U * ((self.v + o.v).abs() + self.e + o.e))

    def __mul__(self, o):
        e = self.v.abs() * o.e + self.e * o.v.abs() + self.e * o.e
        return V(self.v * o.v, e + U * ((self.v * o.v).abs() + e))

    def __getitem__(self, i):
        return V(self.v[i], self.e[i])

    def t(self):
        return V(self.v.T, self.e.T)

    def flat(self):
        return V(self.v.reshape(-1), self.e.reshape(-1))


def matmul(a, b):
    """a [r][k] times b [k][c]."""
    big = (a.v.abs() + a.e) @ (b.v.abs() + b.e)
    e = a.v.abs() @ b.e + a.e @ b.v.abs() + a.e @ b.e
    return V(a.v @ b.v, e + (a.v.shape[1] / 8 + 48) * 2 * U * big)


def summed(a, terms):
    """Over the last dimension, one addition after the other."""
    return V(a.v.sum(-1), a.e.sum(-1) + terms * U * (a.v.abs() + a.e).sum(-1))


def silu(z):
    p = torch.sigmoid(z.v)
    return V(z.v * p, 1.1 * z.e + 64 * U * (z.v.abs() + z.e))


def silu_slope(z):
    p = torch.sigmoid(z.v)
    return V(p * (1 + z.v * (1 - p)), 0.5 * z.e + 64 * U * 1.1)


def halves(z):
    f = z.v.shape[1] // 2
    return z[:, :f], z[:, f:]


def join(a, b):
    return V(torch.cat([a.v, b.v], 1), torch.cat([a.e, b.e], 1))


def swiglu(z):
    g, u = halves(z)
    return silu(g) * u


def through_swiglu(z, d):
    g, u = halves(z)
    return join(d * u * silu_slope(g), d * silu(g))


def check(name, got, want, half):
    """Within the bound and a rounding; the device's own numbers, exact, for what follows."""
    want = want.rounded(half)
    far = (got.double() - want.v).abs() - want.e
    assert bool((far <= 0).all()), (name, float(far.max()))
    return V(got)


def check_layer(L):
    T, H, E, K, F = L.dims
    HB = 2.0 ** -8
    live = T - L.pad
    used = live * K
    x, dout = V(L.x), V(L.dout)
    logits = check("logits", L.logits, matmul(x, V(L.wr[0]).t()), U)
    idx = L.idx.long()
    assert bool((idx[live:] == -1).all()) and bool((idx[:live] >= 0).all())
    chosen = torch.zeros((T, E), dtype=torch.bool, device=DEV)
    chosen[:live].scatter_(1, idx[:live], True)
    assert bool((chosen[:live].sum(1) == K).all())
    best = torch.sort(L.logits[:live], dim=1, descending=True).values[:, :K]
    assert torch.equal(L.logits[:live].gather(1, idx[:live]), best)
    p = torch.softmax(logits.v.masked_fill(~chosen, float("-inf")) if L.renorm else logits.v, 1).nan_to_num(0.0)
    p = V(p, 64 * U * p)
    pick = idx.clamp(0)
    w = check("w", L.w[:live], V(p.v.gather(1, pick), p.e.gather(1, pick))[:live], 0)
    # rows by expert
    at = L.slot.long()[:live]
    order = torch.sort(idx[:live].reshape(-1), stable=True).indices
    assert torch.equal(at.reshape(-1)[order], torch.arange(used, device=DEV)) and bool((L.slot[live:] == -1).all())
    b = [0] + torch.bincount(idx[:live].reshape(-1), minlength=E).cumsum(0).tolist()
    assert L.off.tolist() == b
    token = order // K
    assert torch.equal(L.xs[:used], L.x[token])
    es = [e for e in range(E) if b[e + 1] > b[e]]
    ex = [slice(b[e], b[e + 1]) for e in es]
    xs = x[token]

    def per_expert(fn):
        parts = [fn(e, r) for e, r in zip(es, ex)]
        return V(torch.cat([q.v for q in parts]), torch.cat([q.e for q in parts]))

    def back(rows, by=None):
        """Rows at their tokens, added up; nothing at the padding."""
        v = rows[at.reshape(-1)]
        v = V(v.v.view(live, K, H).transpose(1, 2), v.e.view(live, K, H).transpose(1, 2))
        v = summed(v if by is None else v * V(by.v[:, None], by.e[:, None]), K)
        none = torch.zeros((L.pad, H), dtype=torch.float64, device=DEV)
        return V(torch.cat([v.v, none]), torch.cat([v.e, none]))

    w1, w2, b1, b2 = V(L.w1), V(L.w2), V(L.b1), V(L.b2)
    sums = per_expert(lambda e, r: matmul(xs[r], w1[e].t()) + b1[e])
    z = check("z", L.z[:used], sums, HB)
    h = check("h", L.h[:used], swiglu(sums), HB)
    y = check("y", L.y[:used], per_expert(lambda e, r: matmul(h[r], w2[e].t()) + b2[e]), HB)
    routed = check("routed", L.routed, back(y, w), HB)
    s1, s2 = V(L.s1[0]), V(L.s2[0])
    sums = matmul(x, s1.t())
    zs = check("zs", L.zs, sums, HB)
    hs = check("hs", L.hs, swiglu(sums), HB)
    check("out", L.out, matmul(hs, s2.t()) + routed, HB)
    # backwards
    dy = check("dy", L.dy[:used], dout[token] * w.flat()[order][:, None], HB)
    dw = summed(dout[token] * y, 152)[at.reshape(-1)]
    dw = check("dw", L.dw[:live], V(dw.v.view(live, K), dw.e.view(live, K)), U)
    assert not bool(L.dw[live:].any())
    dz = check("dz", L.dz[:used], through_swiglu(z, per_expert(lambda e, r: matmul(dy[r], w2[e]))), HB)
    for e, r in zip(es, ex):
        n = r.stop - r.start
        check("dw2", L.dw2[e], matmul(dy[r].t(), h[r]), U)
        check("dw1", L.dw1[e], matmul(dz[r].t(), xs[r]), U)
        check("db2", L.db2[e], summed(dy[r].t(), n), U)
        check("db1", L.db1[e], summed(dz[r].t(), n), U)
    for e in set(range(E)) - set(es):
        assert not any(bool(t[e].any()) for t in (L.dw1, L.dw2, L.db1, L.db2))
    dxs = check("dxs", L.dxs[:used], per_expert(lambda e, r: matmul(dz[r], w1[e])), HB)
    dzs = check("dzs", L.dzs, through_swiglu(zs, matmul(dout, s2)), HB)
    check("ds2", L.ds2[0], matmul(dout.t(), hs), U)
    check("ds1", L.ds1[0], matmul(dzs.t(), x), U)
    # the routing: p_e (g_e - sum p g), 64 roundings of the magnitudes
    g = torch.zeros((T, E), dtype=torch.float64, device=DEV)
    g[:live].scatter_(1, idx[:live], dw.v)
    dl = p.v * (g - (p.v * g).sum(1, keepdim=True))
    dl = V(dl, 64 * U * p.v * (g.abs() + (p.v * g.abs()).sum(1, keepdim=True)))
    passes = chosen if L.renorm else (torch.arange(T, device=DEV) < live)[:, None]
    dl = check("dlogits", L.dlogits, V(dl.v * passes, dl.e * passes), HB)
    check("dwr", L.dwr[0], matmul(dl.t(), x), U)
    # the input's gradient: from the sorted rows, the shared expert, the router, rounded at each
    dx = (matmul(dzs, s1) + back(dxs).rounded(HB)).rounded(HB)
    check("dx", L.dx, matmul(dl, V(L.wr[0])) + dx, HB)


@pytest.mark.parametrize("T,H,E,K,F,pad,renorm", [
    (1, 64, 8, 2, 32, 0, True), (5, 136, 8, 8, 40, 0, False), (40, 128, 16, 4, 72, 9, True), (300, 256, 8, 3, 136, 0, False),
    (700, 200, 24, 2, 96, 53, True), (2500, 128, 8, 2, 64, 100, True)])
def test_layer(T, H, E, K, F, pad, renorm):
    """Every number of the layer and of its gradients, from the layer's definition alone."""
    say(f"[gpu] layer T={T} H={H} E={E} K={K} F={F} pad={pad} renorm={renorm}")
    L = Layer(T, H, E, K, F, pad, seed=1, renorm=renorm)
    L.spoil()
    L.run()
    torch.cuda.synchronize()
    check_layer(L)
    first = L.results()                              # and the same bits again
    L.spoil()
    L.run()
    assert same(first, L.results())


def test_layer_by_differences():
    """The gradients' formulas against central differences of the layer in 64 bits (the
    choice of experts held), step 1e-5: off by some 1e-10 of the third derivatives and by
    2^-52 / 1e-5 of the loss; the loss and the derivatives are below 1e3."""
    say("[gpu] layer by differences")
    T, H, E, K, F = 3, 16, 8, 2, 8
    L = Layer(T, H, E, K, F, seed=2)
    L.run()
    torch.cuda.synchronize()
    check_layer(L)
    idx = L.idx.long()
    names = ("x", "wr", "w1", "b1", "w2", "b2", "s1", "s2")
    par = {n: getattr(L, n).double() for n in names}

    def loss(p):
        lo = p["x"] @ p["wr"][0].T
        w = torch.softmax(lo.gather(1, idx), 1)
        act = lambda v: torch.nn.functional.silu(v[..., :F]) * v[..., F:]  # noqa: E731
        z = torch.einsum("th,tkfh->tkf", p["x"], p["w1"][idx]) + p["b1"][idx]
        y = torch.einsum("tkf,tkhf->tkh", act(z), p["w2"][idx]) + p["b2"][idx]
        out = (w[..., None] * y).sum(1) + act(p["x"] @ p["s1"][0].T) @ p["s2"][0].T
        return (out * L.dout.double()).sum()

    # what the formulas' check above was made of, by autograd of the same loss
    leaves = {n: t.clone().requires_grad_() for n, t in par.items()}
    loss(leaves).backward()
    step = 1e-5
    for n in names:
        grad = leaves[n].grad.reshape(-1)
        size = grad.numel()
        for at in range(0, size, max(1, size // 40)):
            ends = []
            for sign in (1, -1):
                q = dict(par)
                t = par[n].clone().reshape(-1)
                t[at] += sign * step
                q[n] = t.view(par[n].shape)
                ends.append(loss(q))
            assert abs(float((ends[0] - ends[1]) / (2 * step) - grad[at])) <= 1e-6, (n, at)
    # and the device's own: at most 9 roundings on a path, each at most 2^-8 of the norm, which
    # the random matrices pass on as they do the values, within a third
    for n, got in (("x", L.dx), ("wr", L.dwr), ("w1", L.dw1), ("b1", L.db1), ("w2", L.dw2), ("b2", L.db2),
                   ("s1", L.ds1), ("s2", L.ds2)):
        want = leaves[n].grad
        assert float((got.double() - want).norm()) <= 12 * 2.0 ** -8 * float(want.norm()), n


def test_captured_layers():
    """Two layers captured into two graphs with a workspace each, replayed in turn and at once
    on two streams, between eager runs: every replay gives the eager bits."""
    say("[gpu] captured layers with gradients")
    layers = [Layer(33, 256, 16, 3, 136, 5, seed=3), Layer(1300, 128, 8, 2, 264, 0, seed=4)]
    want = []
    for L in layers:
        L.run()
        torch.cuda.synchronize()
        want.append(L.results())
    graphs = []
    for L in layers:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.run()
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for L in layers:
            L.spoil()
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for L, first in zip(layers, want):
            assert same(first, L.results())
        if rep == 1:                                 # eager work between the replays
            for L in layers:
                L.run()
            torch.cuda.synchronize()
            # new inputs reach the captured calls
            layers[0].x.neg_()
            layers[0].run()
            torch.cuda.synchronize()
            want[0] = layers[0].results()
            layers[0].spoil()


def test_layers_at_once_on_named_streams():
    say("[gpu] layers at once on named streams")
    layers = [Layer(64, 256, 16, 2, 128, 0, seed=5 + i) for i in range(3)]
    want = []
    for L in layers:
        L.run()
        torch.cuda.synchronize()
        want.append(L.results())
        L.spoil()
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        for L, s in zip(layers, streams):
            L.run(stream=s)
    torch.cuda.synchronize()
    for L, first in zip(layers, want):
        assert same(first, L.results())


@pytest.mark.parametrize("T,E,K", [(1, 16, 2), (77, 16, 3), (400, 64, 4)])
def test_e4m3_layer_is_the_groups(T, E, K):
    """Sorted e4m3 rows through the e4m3 products give the bits of a group of one rank."""
    say(f"[gpu] e4m3 layer T={T} E={E} K={K}")
    H, F = 384, 256
    g = np.random.default_rng([23, T, E])
    x = R.bf16(g.standard_normal((T, H)))
    w13, s13 = R.make_weights(g, E, 2 * F, H)
    w2, s2 = R.make_weights(g, E, H, F)
    w13, s13, w2, s2 = (torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for a in (w13, s13, w2, s2))
    idx = torch.from_numpy(np.argsort(g.random((T, E)), axis=1)[:, :K].astype(np.int32).copy()).to(DEV)
    w = torch.from_numpy(g.random((T, K)).astype(np.float32)).to(DEV)
    rows = T * K
    u8 = torch.uint8

    def products(ex, es, off):
        h, hs, ey = empty(rows, F, dt=u8), empty(rows, F // 128), empty(rows, H, dt=BF16)
        mep.moe_expert_gate_up(rows, E, F, H, ex, es, off, w13, s13, h, hs)
        mep.moe_expert_matmul(rows, E, H, F, h, hs, off, w2, s2, ey)
        return ey

    x = x.to(DEV)
    grp = mep.moe_group_create(1, E, K, H, T, mep.MOE_FP8_E4M3)
    ex, es, off = empty(rows, H, dt=u8), empty(rows, H // 128), empty(E + 1, dt=torch.int32)
    want = empty(T, H, dt=BF16)
    mep.moe_dispatch_send(grp, T, x, idx)
    mep.moe_dispatch_recv(grp, ex, es, off)
    mep.moe_combine_send(grp, products(ex, es, off))
    mep.moe_combine_recv(grp, w, want)
    assert mep.moe_group_status(grp) == mep.MOE_OK
    mep.moe_group_destroy(grp)
    # the tokens' codes, as dispatch coded them
    off2, slot = empty(E + 1, dt=torch.int32), empty(T, K, dt=torch.int32)
    ws = empty(max(1, mep.moe_sort_workspace(T, E, K)), dt=u8)
    mep.moe_sort_plan(T, E, K, idx, off2, slot, None, ws)
    first = slot[:, 0].long()
    ex2, es2, out = empty(rows, H, dt=u8), empty(rows, H // 128), empty(T, H, dt=BF16)
    mep.moe_sort_rows(T, K, rows, H, mep.MOE_FP8_E4M3, ex[first], es[first], slot, ex2, es2)
    assert torch.equal(off, off2) and torch.equal(ex, ex2) and torch.equal(es, es2)
    mep.moe_unsort_rows(T, K, rows, H, mep.MOE_BF16, products(ex2, es2, off2), slot, w, out)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
