"""Tokens sorted by expert and back, and the routing's gradient, against their
definitions (numpy, 64 bits), at the sizes, ids and masks where they can go
wrong.

Tolerances, from the arithmetic:
 * indices and copied rows: equal;
 * a weighted sum of K rows in fp32: K roundings of 2^-24 of the sum of
   magnitudes, then half a step of the output;
 * a dot product of h terms, per lane and then over lanes and waves: a lane has
   at most 128 terms, the rest is a tree and at most 16 waves: 152 roundings;
 * the routing's gradient: exponentials of four roundings, a sum of at most 1024
   terms of one sign in chunks of 16 (32 roundings), a product and a difference:
   under 64 roundings of 2^-24 of |p g| + |p| sum |p g|.
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
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
KIND = {BF16: mep.MOE_BF16, F32: mep.MOE_FP32, F8: mep.MOE_FP8_E4M3}
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def rng(*key):
    return np.random.default_rng([11, *key])


def plan_ref(idx, E):
    """(offsets, slot, source) by sorting (expert, pair)."""
    flat = idx.reshape(-1)
    live = np.flatnonzero((flat >= 0) & (flat < E))
    order = live[np.argsort(flat[live], kind="stable")]
    slot = np.full(flat.size, -1, np.int64)
    slot[order] = np.arange(order.size)
    return np.searchsorted(flat[order], np.arange(E + 1)), slot.reshape(idx.shape), order


def run_plan(idx, E, stream=None):
    T, K = idx.shape
    off, slot = dev(np.full(E + 1, -7, np.int32)), dev(np.full((T, K), -7, np.int32))
    src = dev(np.full(T * K, -7, np.int32))
    ws = torch.empty(mep.moe_sort_workspace(T, E, K), dtype=torch.uint8, device=DEV)
    mep.moe_sort_plan(T, E, K, dev(idx.astype(np.int32)), off, slot, src, ws, stream=stream)
    return off, slot, src


@pytest.mark.parametrize("T,E,K,pad", [
    (0, 8, 2, 0.0), (1, 1, 1, 0.0), (1, 256, 8, 0.0), (3, 5, 2, 0.5), (64, 8, 1, 0.0), (65, 7, 3, 0.1), (127, 1024, 64, 0.0),
    (128, 256, 8, 0.2), (700, 33, 6, 1.0), (1024, 8, 8, 0.0), (1025, 8, 8, 0.1), (5000, 513, 9, 0.0),
    (8192, 512, 4, 0.3), (16384, 1024, 8, 0.0), (131072, 256, 8, 0.05), (99991, 3, 17, 0.0), (40000, 1000, 60, 0.1)])
def test_plan(T, E, K, pad):
    say(f"[gpu] sort plan T={T} E={E} K={K} pad={pad}")
    g = rng(1, T, E, K)
    # popular and rare experts, the same expert twice among them, ids of no expert
    idx = np.minimum((E * g.random((T, K)) ** 2).astype(np.int64), E - 1)
    out = g.random((T, K)) < pad
    idx[out] = g.choice([-1, E, E + 5, -2 ** 31, 2 ** 31 - 1], size=int(out.sum()))
    off, slot, src = run_plan(idx, E)
    want_off, want_slot, order = plan_ref(idx, E)
    assert np.array_equal(off.cpu().numpy(), want_off)
    assert np.array_equal(slot.cpu().numpy(), want_slot)
    got = src.cpu().numpy()
    assert np.array_equal(got[:order.size], order) and (got[order.size:] == -7).all()


def test_plan_without_source_and_one_expert():
    say("[gpu] sort plan, all pairs of one expert, no source")
    for T in (100, 30000):
        idx = np.full((T, 3), 4, np.int32)
        off, slot = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (9, 3 * T))
        ws = torch.empty(mep.moe_sort_workspace(T, 8, 3), dtype=torch.uint8, device=DEV)
        mep.moe_sort_plan(T, 8, 3, dev(idx), off, slot, None, ws)
        assert off.tolist() == [0] * 5 + [3 * T] * 4
        assert torch.equal(slot, torch.arange(3 * T, dtype=torch.int32, device=DEV))


ROWS = [(1, 8, 1), (3, 24, 2), (1, 7168, 8), (5, 128, 3), (33, 40, 5), (17, 504, 4), (9, 512, 2), (7, 520, 64),
        (130, 1032, 6), (2, 65536, 2), (300, 2048, 4)]


def routed(T, K, E=11, pad=0.2, key=0):
    g = rng(2, T, K, key)
    idx = g.integers(0, E, size=(T, K))
    idx[g.random((T, K)) < pad] = -1
    off, slot, _ = run_plan(idx, E)
    return idx, slot, int(off[-1])


@pytest.mark.parametrize("T,H,K", ROWS)
@pytest.mark.parametrize("kind", [BF16, F32, F8], ids=["bf16", "fp32", "e4m3"])
def test_sort_rows(T, H, K, kind):
    if kind == F8 and H % 128:
        H = -(-H // 128) * 128
    say(f"[gpu] sort rows T={T} H={H} K={K} {kind}")
    _, slot, used = routed(T, K)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    size = torch.empty(0, dtype=kind).element_size()
    x = torch.randint(0, 256, (T, H * size), generator=gen, device=DEV, dtype=torch.uint8).view(kind)   # any bits: NaN too
    xs = torch.rand((T, H // 128), generator=gen, device=DEV) if kind == F8 else None
    rows = T * K + 3
    out = torch.full((rows, H * size), 0x5A, dtype=torch.uint8, device=DEV).view(kind)
    outs = torch.full((rows, H // 128), -3.0, device=DEV) if kind == F8 else None
    mep.moe_sort_rows(T, K, rows, H, KIND[kind], x, xs, slot, out, outs)
    want = torch.full((rows, H * size), 0x5A, dtype=torch.uint8, device=DEV)
    live = slot >= 0
    token = torch.arange(T, device=DEV)[:, None].expand(T, K)
    want[slot[live].long()] = x.view(torch.uint8)[token[live]]
    assert torch.equal(out.view(torch.uint8), want)
    if kind == F8:
        ws = torch.full((rows, H // 128), -3.0, device=DEV)
        ws[slot[live].long()] = xs[token[live]]
        assert torch.equal(outs, ws)
    assert int(live.sum()) == used


@pytest.mark.parametrize("T,H,K", ROWS)
@pytest.mark.parametrize("kind", [BF16, F32], ids=["bf16", "fp32"])
def test_unsort_and_gradient(T, H, K, kind):
    say(f"[gpu] unsort rows T={T} H={H} K={K} {kind}")
    _, slot, used = routed(T, K, key=1)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)
    rows = T * K
    y = torch.randn((rows, H), generator=gen, device=DEV).to(kind)
    y[used:] = float("nan")                          # rows of no pair are not read
    w = torch.rand((T, K), generator=gen, device=DEV)
    dout = torch.randn((T, H), generator=gen, device=DEV).to(kind)
    live, at = slot >= 0, slot.clamp_min(0).long()
    w64 = torch.where(live, w.double(), 0.0)
    y64 = torch.where(live[..., None], y[at].double(), 0.0)
    for weights in (w, None):
        f = w64 if weights is not None else live.double()
        out = torch.full((T, H), 9.0, device=DEV).to(kind)
        mep.moe_unsort_rows(T, K, rows, H, KIND[kind], y, slot, weights, out)
        ref, big = (y64 * f[..., None]).sum(1), (y64.abs() * f[..., None]).sum(1)
        assert bool(((out.double() - ref).abs() <= K * U * big + HALF[kind] * (ref.abs() + K * U * big)).all())
        dy, dw = torch.full_like(y, 9.0), torch.full((T, K), 9.0, device=DEV)
        mep.moe_unsort_rows_grad(T, K, rows, H, KIND[kind], dout, y, slot, weights, dy, dw)
        want = (f[..., None] * dout.double()[:, None])[live]
        got = dy[slot[live].long()].double()
        assert bool(((got - want).abs() <= (HALF[kind] + 2 * U) * want.abs()).all())
        assert bool((dy[used:] == 9.0).all())
        ref = (y64 * dout.double()[:, None]).sum(-1)
        big = (y64 * dout.double()[:, None]).abs().sum(-1)
        assert bool(((dw.double() - ref).abs() <= 152 * U * big).all())
        assert bool((dw[~live] == 0).all())
        # each gradient alone gives the same bits
        dy2, dw2 = torch.full_like(y, 9.0), torch.full((T, K), 9.0, device=DEV)
        mep.moe_unsort_rows_grad(T, K, rows, H, KIND[kind], dout, None, slot, weights, dy2, None)
        mep.moe_unsort_rows_grad(T, K, rows, H, KIND[kind], dout, y, slot, weights, None, dw2)
        assert torch.equal(dy.view(torch.uint8), dy2.view(torch.uint8)) and torch.equal(dw, dw2)


def test_unsort_gradient_by_differences():
    """out is linear in y and in the weights: with whole numbers in fp32 the differences are exact."""
    say("[gpu] unsort gradient by differences")
    T, K, H = 5, 3, 40
    g = rng(3)
    _, slot, used = routed(T, K, pad=0.3, key=2)
    y = dev(g.integers(-8, 9, size=(T * K, H)).astype(np.float32))
    w = dev(g.integers(-4, 5, size=(T, K)).astype(np.float32))
    dout = dev(g.integers(-4, 5, size=(T, H)).astype(np.float32))
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    mep.moe_unsort_rows_grad(T, K, T * K, H, mep.MOE_FP32, dout, y, slot, w, dy, dw)

    def loss(y, w):
        out = torch.empty((T, H), device=DEV)
        mep.moe_unsort_rows(T, K, T * K, H, mep.MOE_FP32, y, slot, w, out)
        return float((out * dout).double().sum())

    base = loss(y, w)
    for r in range(0, used, 2):
        y2 = y.clone()
        y2[r, (7 * r) % H] += 1
        assert loss(y2, w) - base == float(dy[r, (7 * r) % H])
    for t in range(T):
        for k in range(K):
            w2 = w.clone()
            w2[t, k] += 1
            assert loss(y, w2) - base == float(dw[t, k])


def test_unsort_is_combine():
    """The bits of dispatch and combine over a group of one rank."""
    say("[gpu] sort and unsort against a group of one rank")
    T, K, E, H = 300, 8, 64, 1024
    g = rng(4)
    idx = np.argsort(g.random((T, E)), axis=1)[:, :K].astype(np.int32)
    x, w = R.bf16(g.standard_normal((T, H))).to(DEV), dev(g.random((T, K)).astype(np.float32))
    y = R.bf16(g.standard_normal((T * K, H))).to(DEV)
    grp = mep.moe_group_create(1, E, K, H, T)
    ex, off0, want = torch.empty_like(y), torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty_like(x)
    mep.moe_dispatch_send(grp, T, x, dev(idx))
    mep.moe_dispatch_recv(grp, ex, None, off0)
    mep.moe_combine_send(grp, y)
    mep.moe_combine_recv(grp, w, want)
    assert mep.moe_group_status(grp) == mep.MOE_OK
    mep.moe_group_destroy(grp)
    off, slot, _ = run_plan(idx, E)
    rows, out = torch.empty_like(y), torch.empty_like(x)
    mep.moe_sort_rows(T, K, T * K, H, mep.MOE_BF16, x, None, slot, rows, None)
    mep.moe_unsort_rows(T, K, T * K, H, mep.MOE_BF16, y, slot, w, out)
    for a, b in ((off, off0), (rows, ex), (out, want)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_slots_outside_the_rows():
    """Hand-made slots beyond the room name no row."""
    say("[gpu] slots outside the rows")
    T, K, H = 4, 2, 128
    slot = dev(np.array([[0, 3], [7, -5], [2 ** 31 - 1, 1], [2, -2 ** 31]], np.int32))
    x = torch.ones((T, H), device=DEV)
    out = torch.zeros((5, H), device=DEV)
    mep.moe_sort_rows(T, K, 4, H, mep.MOE_FP32, x, None, slot, out, None)
    assert out[:, 0].tolist() == [1, 1, 1, 1, 0]
    back = torch.zeros((T, H), device=DEV)
    mep.moe_unsort_rows(T, K, 4, H, mep.MOE_FP32, out, slot, None, back)
    assert back[:, 5].tolist() == [2, 0, 1, 1]
    dy, dw = torch.zeros((5, H), device=DEV), torch.full((T, K), 9.0, device=DEV)
    mep.moe_unsort_rows_grad(T, K, 4, H, mep.MOE_FP32, x, out, slot, None, dy, dw)
    assert dy[:, 0].tolist() == [1, 1, 1, 1, 0]
    assert dw.tolist() == [[H, H], [0, 0], [0, H], [H, 0]]


# --- the routing's gradient ----------------------------------------------------------------------

def route_grad_ref(z, idx, dw, renorm):
    """(gradient, error scale) in 64 bits; ids outside are -1."""
    T, E = z.shape
    d, scale = np.zeros((T, E)), np.zeros((T, E))
    z = np.where(np.isnan(z), -np.inf, z)
    for t in range(T):
        ids = [(k, e) for k, e in enumerate(idx[t]) if 0 <= e < E]
        pool = z[t, [e for _, e in ids]] if renorm else z[t]
        top = pool.max() if len(pool) else -np.inf
        if top == -np.inf:
            continue

        def soft(v):
            return (v == np.inf).astype(float) if top == np.inf else np.exp(v - top)
        total = soft(pool).sum()
        p = soft(z[t]) / total
        live = [(k, e) for k, e in ids if p[e] > 0]
        G = sum(p[e] * dw[t, k] for k, e in live)
        Gabs = sum(p[e] * abs(dw[t, k]) for k, e in live)
        g, gabs = np.zeros(E), np.zeros(E)
        for k, e in live:
            g[e] += dw[t, k]
            gabs[e] += abs(dw[t, k])
        times = np.ones(E)
        if renorm:
            times = np.bincount([e for _, e in ids], minlength=E)
        d[t] = np.where((times > 0) & (p > 0), p * (g - times * G), 0)
        scale[t] = np.where(times > 0, p * (gabs + times * Gabs), 0)
    return d, scale


def check_route_grad(z, idx, dw, renorm, in_kind, out_kind):
    T, E = z.shape
    K = idx.shape[1]
    zt = dev(z.astype(np.float32)).to(in_kind)
    got = torch.full((T, E), 9.0, device=DEV).to(out_kind)
    mep.moe_topk_route_grad(T, E, K, zt, KIND[in_kind], renorm, dev(idx.astype(np.int32)),
                            dev(dw.astype(np.float32)), got, KIND[out_kind])
    want, scale = route_grad_ref(R.f64(zt), idx, dw.astype(np.float32).astype(np.float64), renorm)
    err = 64 * U * scale
    assert np.all(np.abs(R.f64(got) - want) <= err + HALF[out_kind] * (np.abs(want) + err) + 2.0 ** -126)


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (5, 2, 2), (70, 8, 2), (33, 16, 4), (9, 17, 17), (130, 64, 6), (64, 60, 8),
                                   (300, 256, 8), (20, 250, 16), (7, 256, 64), (11, 257, 8), (6, 1000, 64), (3, 1024, 20)])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kinds", [(F32, F32), (BF16, BF16), (F32, BF16)], ids=["fp32", "bf16", "fp32-bf16"])
def test_route_grad(T, E, K, renorm, kinds):
    say(f"[gpu] route gradient T={T} E={E} K={K} renorm={renorm} {kinds}")
    g = rng(5, T, E, K)
    z = 2 * g.standard_normal((T, E))
    z[g.random((T, E)) < 0.1] = -np.inf
    z = R.f64(dev(z.astype(np.float32)).to(kinds[0]))
    idx = np.argsort(-z, axis=1, kind="stable")[:, :K]
    check_route_grad(z, idx, g.standard_normal((T, K)), renorm, *kinds)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_masks(renorm):
    say(f"[gpu] route gradient: masks, infinities, padding, the same expert twice, renorm={renorm}")
    g = rng(6)
    inf, nan = np.inf, np.nan
    low = float(np.finfo(np.float32).min)
    z = np.array([[-inf] * 5, [nan] * 5, [1, -inf, nan, 2, 3], [inf, 1, inf, 0, -inf], [1, 2, 3, 4, 5], [1, 2, 3, 4, 5],
                  [-200, 0, -200, 0, 50], [low, low, low, low, low], [low, low, 0, low, -inf], [88, -88, 0, 200, -200]])
    idx = np.array([[0, 1, 2], [0, 1, 2], [4, 3, 0], [0, 2, 1], [-1, -1, -1], [4, 4, 9], [4, 1, 3], [0, 1, 2], [2, 0, 1], [3, 0, 2]])
    dw = g.standard_normal(idx.shape)
    check_route_grad(z, idx, dw, renorm, F32, F32)
    # weights of 0 pass nothing, whatever came for them
    dw[0] = dw[1] = nan
    idx[2] = [4, 1, 2]
    dw[2, 1:] = [inf, nan]
    check_route_grad(z, idx, dw, renorm, F32, F32)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("repeats", [False, True], ids=["", "repeats"])
def test_route_grad_by_differences(renorm, repeats):
    """Against differences of the 64-bit weights: central ones of step 1e-4 are off by about
    h^2 |f'''| / 6 < 1e-8 of the weights' size."""
    say(f"[gpu] route gradient by differences renorm={renorm} repeats={repeats}")
    T, E, K, h = 4, 24, 5, 1e-4
    g = rng(7)
    z = R.f64(dev(g.standard_normal((T, E)).astype(np.float32)))
    idx = np.argsort(-z, axis=1, kind="stable")[:, :K]
    if repeats:                                      # a caller's own choices may name an expert twice
        idx[:, 3] = idx[:, 1]
        idx[0] = idx[0, 0]
    dw = g.standard_normal((T, K)).astype(np.float32).astype(np.float64)

    def loss(z):
        p = np.exp(z - z.max(1, keepdims=True))
        w = np.take_along_axis(p / p.sum(1, keepdims=True), idx, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return (w * dw).sum(1)

    got = torch.empty((T, E), device=DEV)
    mep.moe_topk_route_grad(T, E, K, dev(z.astype(np.float32)), mep.MOE_FP32, renorm, dev(idx.astype(np.int32)),
                            dev(dw.astype(np.float32)), got, mep.MOE_FP32)
    check_route_grad(z, idx, dw, renorm, F32, F32)
    for e in range(E):
        step = np.zeros((T, E))
        step[:, e] = h
        diff = (loss(z + step) - loss(z - step)) / (2 * h)
        assert np.all(np.abs(R.f64(got)[:, e] - diff) <= 1e-7 + 64 * U * np.abs(dw).sum(1))


def test_route_grad_of_the_routing():
    """Ids as moe_topk_route gives them, a large batch."""
    say("[gpu] route gradient after moe_topk_route")
    T, E, K = 3000, 256, 8
    g = rng(8)
    z = 3 * g.standard_normal((T, E))
    z[g.random((T, E)) < 0.2] = -np.inf
    z[7] = -np.inf
    zt, idx, w = dev(z.astype(np.float32)), torch.empty((T, K), dtype=torch.int32, device=DEV), torch.empty((T, K), device=DEV)
    mep.moe_topk_route(T, E, K, zt, mep.MOE_FP32, True, idx, w)
    check_route_grad(z.astype(np.float32), idx.cpu().numpy(), g.standard_normal((T, K)), True, F32, F32)
