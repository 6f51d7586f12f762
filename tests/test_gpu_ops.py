"""The operators around dispatch and combine against their definitions in 64
bits (tests/ops_ref.py), at the sizes, masks and values where they can go
wrong.

Tolerances, from the arithmetic:
 * a bf16 result is off by half a step, 2^-8 |v|, plus the fp32 work before it;
 * an e4m3 code by half a step, 2^-4 |v| (2^-10 of the scale below the normal
   numbers), plus the fp32 work before it, which can move a value over a
   rounding border and adds its own size only;
 * an fp32 sum of n terms in chunks of at most c in a row, c + log2 of the
   rest roundings of 2^-24 of the sum of magnitudes;
 * moe_expert_matmul's block sums come from the e4m3 matrix instruction, which
   aligns a block's products before adding them: at most 2^-10 of the block's
   largest product each (measured: 2^-11.2 over random codes).
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def rng(*key):
    return np.random.default_rng([7, *key])


# --- norm ---------------------------------------------------------------------------------------

def norm_ref(x, r, w, eps):
    s = x + (0 if r is None else r)
    return s, s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * w


def check_norm(x, r, w, y, yq, ys, ro, eps):
    s, ref = norm_ref(R.f64(x), None if r is None else R.f64(r), R.f64(w), eps)
    rel = 2.0 ** -17          # sum of squares, its root, two products: well under 64 roundings
    if ro is not None:
        assert np.all(np.abs(R.f64(ro) - s) <= (R.BF16_HALF + 2.0 ** -22) * np.abs(s) + 2.0 ** -133)
    if y is not None:
        assert np.all(np.abs(R.f64(y) - ref) <= (R.BF16_HALF + rel) * np.abs(ref) + 2.0 ** -133)
    if yq is not None:
        scale, _ = R.block_scale(ref)
        got_s = R.f64(ys)
        assert np.all(np.abs(got_s - scale) <= rel * scale)
        got = R.rows_value(yq.view(torch.uint8).cpu().numpy(), got_s.astype(np.float32))
        sc = scale.repeat(R.BLOCK, -1)
        assert np.all(np.abs(got - ref) <= (R.E4M3_HALF + 2 * rel) * np.abs(ref) + (2.0 ** -10 + rel) * sc)


NORM_SHAPES = [(1, 8), (3, 24), (5, 128), (2, 136), (7, 1024), (9, 1032), (1, 4096), (3, 7168),
               (2, 16384), (2, 16392), (1, 65536), (513, 256), (130, 7168),
               (131, 32), (65, 40), (37, 384), (35, 504), (33, 512), (9, 520)]


@pytest.mark.parametrize("rows,hidden", NORM_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(rows, hidden, residual):
    say(f"[gpu] norm rows={rows} hidden={hidden} residual={residual}")
    g = rng(1, rows, hidden)
    x = R.bf16(g.standard_normal((rows, hidden)) * np.where(g.random(hidden) < 0.02, 20, 1)).to(DEV)
    r = R.bf16(5 * g.standard_normal((rows, hidden))).to(DEV) if residual else None
    w = R.bf16(1 + 0.3 * g.standard_normal(hidden)).to(DEV)
    fp8 = hidden % 128 == 0
    y, ro = torch.empty_like(x), torch.empty_like(x)
    yq = torch.empty((rows, hidden), dtype=torch.float8_e4m3fn, device=DEV) if fp8 else None
    ys = torch.empty((rows, hidden // 128), device=DEV) if fp8 else None
    mep.moe_add_rmsnorm(rows, hidden, x, r, w, 1e-6, ro, y, yq, ys)
    torch.cuda.synchronize()
    check_norm(x, r, w, y, yq, ys, ro, 1e-6)
    # each output alone gives the same bits
    for only in range(3 if fp8 else 2):
        o = [torch.empty_like(t) if t is not None else None for t in (ro, y, yq, ys)]
        mep.moe_add_rmsnorm(rows, hidden, x, r, w, 1e-6, o[0] if only == 0 else None,
                            o[1] if only == 1 else None, o[2] if only == 2 else None,
                            o[3] if only == 2 else None)
        torch.cuda.synchronize()
        for got, want in [((o[0], ro),), ((o[1], y),), ((o[2], yq), (o[3], ys))][only]:
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("rows,hidden", [(9000, 4096), (33000, 4096), (700000, 128)])
def test_norm_past_the_caches(rows, hidden):
    """Rows that the caches do not hold take other accesses: the same bits as in parts."""
    say(f"[gpu] norm past the caches rows={rows} hidden={hidden}")
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    x, r = (torch.randn((rows, hidden), generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2))
    w = torch.randn(hidden, generator=gen, device=DEV).to(torch.bfloat16)
    whole, parts = ([torch.empty_like(x), torch.empty_like(x), torch.empty((rows, hidden), dtype=torch.uint8, device=DEV),
                     torch.empty((rows, hidden // 128), device=DEV)] for _ in range(2))
    mep.moe_add_rmsnorm(rows, hidden, x, r, w, 1e-6, *whole)
    step = (1 << 21) // hidden
    for a in range(0, rows, step):
        n = min(step, rows - a)
        mep.moe_add_rmsnorm(n, hidden, x[a:a + n], r[a:a + n], w, 1e-6, *(t[a:a + n] for t in parts))
    torch.cuda.synchronize()
    for a, b in zip(whole, parts):
        assert torch.equal(a, b)


def test_norm_in_place_and_neighbours():
    say("[gpu] norm in place; rows behind the last")
    rows, hidden = 37, 7168
    g = rng(2)
    x0 = R.bf16(g.standard_normal((rows, hidden))).to(DEV)
    r0 = R.bf16(g.standard_normal((rows, hidden))).to(DEV)
    w = R.bf16(g.standard_normal(hidden)).to(DEV)
    y, ro = torch.empty_like(x0), torch.empty_like(x0)
    mep.moe_add_rmsnorm(rows, hidden, x0, r0, w, 1e-5, ro, y, None, None)
    x, r = x0.clone(), r0.clone()
    mep.moe_add_rmsnorm(rows, hidden, x, r, w, 1e-5, r, x, None, None)
    torch.cuda.synchronize()
    assert torch.equal(x, y) and torch.equal(r, ro)
    # fewer rows than the tensors hold: the rest stays as it was
    z = torch.full_like(x0, 3.0)
    mep.moe_add_rmsnorm(rows - 5, hidden, x0, r0, w, 1e-5, None, z, None, None)
    torch.cuda.synchronize()
    assert torch.equal(z[:-5], y[:-5]) and bool((z[-5:] == 3.0).all())


@pytest.mark.parametrize("rows,hidden", [(300, 24), (300, 128), (100, 384), (9, 1032), (5, 16392), (9000, 4096)])
def test_norm_in_place(rows, hidden):
    say(f"[gpu] norm in place rows={rows} hidden={hidden}")
    g = rng(20, rows, hidden)
    x, r, w = (R.bf16(g.standard_normal(s, dtype=np.float32)).to(DEV) for s in ((rows, hidden), (rows, hidden), hidden))
    ro, y = torch.empty_like(x), torch.empty_like(x)
    mep.moe_add_rmsnorm(rows, hidden, x, r, w, 1e-6, ro, y, None, None)
    for a, b in ((0, 1), (1, 0)):                   # residual_out and y over x and residual, both ways
        t = [x.clone(), r.clone()]
        mep.moe_add_rmsnorm(rows, hidden, t[0], t[1], w, 1e-6, t[a], t[b], None, None)
        torch.cuda.synchronize()
        assert torch.equal(t[a], ro) and torch.equal(t[b], y)


def test_norm_odd_values():
    """A NaN or an infinity stays in its row; rows and blocks of zeros; tiny blocks."""
    say("[gpu] norm odd values")
    rows, hidden = 6, 512
    g = rng(3)
    a = g.standard_normal((rows, hidden)).astype(np.float32)
    a[1, 7] = np.nan
    a[2, 9] = np.inf
    a[3] = 0
    a[4, 128:256] = 0
    x = R.bf16(a).to(DEV)
    wv = 1 + 0.1 * g.standard_normal(hidden)
    wv[256:384] *= 2.0 ** -124          # a block below the codec's smallest scale
    w = R.bf16(wv).to(DEV)
    y = torch.empty_like(x)
    yq = torch.empty((rows, hidden), dtype=torch.float8_e4m3fn, device=DEV)
    ys = torch.empty((rows, 4), device=DEV)
    mep.moe_add_rmsnorm(rows, hidden, x, None, w, 1e-6, None, y, yq, ys)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[1].float()).all())
    assert bool((y[3] == 0).all()) and bool((ys[3] == 1).all()) and bool((yq[3].float() == 0).all())
    assert float(ys[4, 1]) == 1.0 and bool((yq[4, 128:256].float() == 0).all())
    assert float(ys[0, 2]) == 2.0 ** -126
    keep = [0, 4, 5]
    _, ref = norm_ref(R.f64(x[keep]), None, R.f64(w), 1e-6)
    assert np.all(np.abs(R.f64(y[keep]) - ref) <= (R.BF16_HALF + 2.0 ** -17) * np.abs(ref) + 2.0 ** -133)


# --- routing --------------------------------------------------------------------------------------

def route_ref(z, K, renorm):
    z = np.where(np.isnan(z), -np.inf, z)
    idx = np.argsort(-z, axis=-1, kind="stable")[:, :K]
    top = z.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.where(np.isneginf(top), 0.0, np.where(z == top, 1.0, np.exp(z - top)))
    total = p.sum(-1, keepdims=True)
    w = np.take_along_axis(p, idx, -1)
    total = w.sum(-1, keepdims=True) if renorm else total
    return idx, np.where(total > 0, w / np.where(total > 0, total, 1), 0.0)


def check_route(logits, E, K, renorm):
    T = logits.shape[0]
    idx = torch.full((T + 1, K), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T + 1, K), -7.0, device=DEV)
    mep.moe_topk_route(T, E, K, logits, mep.MOE_BF16 if logits.dtype == torch.bfloat16 else mep.MOE_FP32,
                       renorm, idx, w)
    torch.cuda.synchronize()
    z = R.f64(logits)
    ri, rw = route_ref(z, K, renorm)
    assert np.array_equal(idx[:T].cpu().numpy(), ri)
    # exp: its argument (|z - top| ulps of it in fp32) and the sums of E and K terms
    top = np.nan_to_num(np.where(np.isnan(z), -np.inf, z).max(-1, keepdims=True), neginf=0, posinf=0)
    far = np.nan_to_num(np.abs(np.take_along_axis(z, ri, -1) - top), posinf=0, nan=0)
    assert np.all(np.abs(R.f64(w[:T]) - rw) <= rw * (far + 40) * 2.0 ** -23 + 2.0 ** -126)
    assert bool((idx[T] == -7).all()) and bool((w[T] == -7).all())


@pytest.mark.parametrize("E,K", [(1, 1), (2, 2), (7, 3), (8, 2), (63, 8), (64, 64), (65, 6), (128, 8),
                                 (255, 1), (256, 8), (256, 17), (257, 9), (384, 8), (1000, 64), (1024, 10)])
@pytest.mark.parametrize("bf", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(E, K, bf, renorm):
    say(f"[gpu] route E={E} K={K} bf16={bf} renorm={renorm}")
    for T in (1, 19, 130):
        g = rng(4, E, K, T)
        z = 3 * g.standard_normal((T, E))
        if T == 19:
            z = np.round(z)                                  # many equal logits
        z[g.random((T, E)) < 0.1] = -np.inf
        t = torch.from_numpy(z.astype(np.float32)).to(torch.bfloat16 if bf else torch.float32).to(DEV)
        check_route(t, E, K, renorm)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_masks(renorm):
    say(f"[gpu] route masks renorm={renorm}")
    E, K = 40, 6
    g = rng(5)
    z = g.standard_normal((12, E)).astype(np.float32)
    z[0] = -np.inf                                           # nothing left
    z[1] = np.nan
    z[2, :36] = -np.inf                                      # fewer than K left
    z[3] = np.finfo(np.float32).min                          # the type's lowest value masks nothing
    z[4, 3:] = np.finfo(np.float32).min
    z[5, 11] = np.inf
    z[6, [2, 9]] = np.inf
    z[7] = 1e30
    z[8] = 0.0
    z[9, 5] = np.nan
    z[10] = -200 + z[10]
    z[11, 0] = 150
    check_route(torch.from_numpy(z).to(DEV), E, K, renorm)


@pytest.mark.parametrize("T,E,K", [(16385, 100, 8), (16390, 128, 64), (16400, 65, 3), (1003, 16, 16), (77, 12, 5),
                                   (4099, 33, 12), (2051, 64, 16), (777, 17, 17), (1030, 256, 16), (515, 255, 8),
                                   (99, 200, 17), (33, 129, 1), (1, 64, 6)])
def test_route_many_tokens(T, E, K):
    say(f"[gpu] route T={T} E={E} K={K}")
    g = rng(17, T, E)
    z = np.round(2 * g.standard_normal((T, E))) / 2                # many ties
    z[g.random((T, E)) < 0.2] = -np.inf
    z[::97] = -np.inf
    z[5::101] = np.nan
    check_route(torch.from_numpy(z.astype(np.float32)).to(DEV), E, K, True)
    check_route(torch.from_numpy(z.astype(np.float32)).to(torch.bfloat16).to(DEV), E, K, False)


# --- products -------------------------------------------------------------------------------------

def counts_of(kind, E, rows, g):
    if kind == "even":
        c = np.full(E, rows // E)
        c[: rows % E] += 1
    elif kind == "first":
        c = np.zeros(E, int)
        c[0] = rows
    elif kind == "last":
        c = np.zeros(E, int)
        c[-1] = rows
    else:
        p = np.exp(1.5 * g.standard_normal(E))
        c = g.multinomial(rows, p / p.sum())
    return c


def grouped_inputs(g, E, n, k, counts, spare, spread=1.0):
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x, xs = R.make_rows(g, int(offsets[-1]) + spare, k, spread)
    w, ws = R.make_weights(g, E, n, k)
    return x, xs, w, ws, offsets


# rows per expert on both sides of every tile choice, one to many scale chunks
PRODUCTS = [
    # E, rows, n, k, counts, spare
    (1, 1, 8, 128, "even", 0), (1, 3, 136, 256, "even", 2), (3, 5, 256, 384, "spread", 0),
    (8, 37, 1000, 384, "spread", 5), (5, 60, 264, 1152, "last", 0), (2, 40, 512, 640, "even", 3),
    (3, 150, 248, 512, "spread", 1), (2, 180, 384, 2304, "first", 0), (2, 300, 520, 256, "even", 0),
    (1, 257, 256, 1024, "even", 7), (4, 1300, 304, 384, "spread", 0), (300, 700, 16, 128, "spread", 0),
    (1024, 900, 8, 128, "spread", 4)]


def run_matmul(x, xs, w, ws, offsets, room=None):
    E, n, k = w.shape
    rows = x.shape[0] if room is None else room
    y = torch.full((rows + 1, n), 9.0, dtype=torch.bfloat16, device=DEV)
    mep.moe_expert_matmul(rows, E, n, k, dev(x), dev(xs), dev(offsets), dev(w), dev(ws), y)
    torch.cuda.synchronize()
    return y


def check_product(y, ref, big, mags):
    tol = R.BF16_HALF * np.abs(ref) + 2.0 ** -10 * big * (1 + R.BF16_HALF) + 2.0 ** -20 * mags
    assert np.all(np.abs(y - ref) <= tol), float(np.max(np.abs(y - ref) / np.maximum(tol, 1e-300)))


@pytest.mark.parametrize("E,rows,n,k,kind,spare", PRODUCTS)
def test_matmul(E, rows, n, k, kind, spare):
    say(f"[gpu] matmul E={E} rows={rows} n={n} k={k} {kind}")
    g = rng(6, E, rows, n, k)
    ins = grouped_inputs(g, E, n, k, counts_of(kind, E, rows, g), spare)
    y = run_matmul(*ins)
    ref, big = R.product(*ins)
    check_product(R.f64(y[:rows]), ref, big, big * R.BLOCK)
    assert bool((y[rows:] == 9.0).all())


@pytest.mark.parametrize("E,rows,n,k,kind,spare", [
    (1, 97, 264, 384, "even", 0), (1, 144, 520, 256, "even", 1), (2, 250, 256, 128, "even", 0),
    (3, 390, 136, 640, "spread", 2), (5, 700, 512, 1280, "spread", 0), (4, 500, 256, 384, "last", 0)])
def test_matmul_near_128_rows(E, rows, n, k, kind, spare):
    test_matmul(E, rows, n, k, kind, spare)


def run_gate_up(x, xs, w, ws, offsets):
    E, n, k = w.shape
    f, rows = n // 2, x.shape[0]
    h = torch.full((rows + 1, f), 5, dtype=torch.uint8, device=DEV)
    hs = torch.full((rows + 1, f // 128), 9.0, device=DEV)
    mep.moe_expert_gate_up(rows, E, f, k, dev(x), dev(xs), dev(offsets), dev(w), dev(ws), h, hs)
    torch.cuda.synchronize()
    return h, hs


def check_gate_up(h, hs, x, xs, w, ws, offsets):
    f = w.shape[1] // 2
    a, big = R.product(x, xs, w, ws, offsets)
    gate, up = a[:, :f], a[:, f:]
    ref = R.silu(gate) * up
    # fp32 sums of the products: each of gate and up is off by d, silu's slope is below 1.1
    d = 2.0 ** -19 * big
    work = 1.1 * d[:, :f] * np.abs(up) + np.abs(R.silu(gate)) * d[:, f:] + 2.0 ** -19 * np.abs(ref)
    scale, _ = R.block_scale(ref)
    top = work.reshape(len(work), -1, R.BLOCK).max(-1) / 448
    assert np.all(np.abs(hs - scale) <= top + 2.0 ** -22 * scale)
    got = R.rows_value(h, hs)
    tol = (R.E4M3_HALF + 2.0 ** -18) * np.abs(ref) + 2 * work + (2.0 ** -10 * scale + top).repeat(R.BLOCK, -1)
    assert np.all(np.abs(got - ref) <= tol)


@pytest.mark.parametrize("E,rows,f,k,kind,spare", [
    (E, rows, max(128, (n + 64) // 128 * 128), k, kind, spare) for E, rows, n, k, kind, spare in PRODUCTS
    if E <= 300])
def test_gate_up(E, rows, f, k, kind, spare):
    say(f"[gpu] gate_up E={E} rows={rows} f={f} k={k} {kind}")
    g = rng(7, E, rows, f, k)
    x, xs, w, ws, offsets = grouped_inputs(g, E, 2 * f, k, counts_of(kind, E, rows, g), spare, 0.3)
    ws *= np.float32(2.0 ** -4 / np.sqrt(k / 128))          # gates of a size that silu does not saturate
    h, hs = run_gate_up(x, xs, w, ws, offsets)
    check_gate_up(h[:rows].cpu().numpy(), R.f64(hs[:rows]), x, xs, w, ws, offsets)
    assert bool((h[rows:] == 5).all()) and bool((hs[rows:] == 9.0).all())


@pytest.mark.parametrize("rows", [4, 40, 150, 600])
def test_products_odd_values(rows):
    """A NaN code stays in its row; rows and scales of zero; empty experts; nothing to do."""
    say(f"[gpu] products odd values rows={rows}")
    g = rng(8, rows)
    E, n, k = 2, 256, 384
    x, xs, w, ws, offsets = grouped_inputs(g, E, n, k, counts_of("even", E, rows, g), 0, 0.3)
    ws *= np.float32(2.0 ** -4)
    x[1] = 0                                              # zeros, also as -0
    x[1, ::2] = 0x80
    clean = run_matmul(x, xs, w, ws, offsets)
    ch, cs = run_gate_up(x, xs, w, ws, offsets)
    assert bool((clean[1] == 0).all()) and bool((cs[1] == 1).all())
    bad = x.copy()
    bad[rows - 1, 5] = 0x7F
    y = run_matmul(bad, xs, w, ws, offsets)
    h, hs = run_gate_up(bad, xs, w, ws, offsets)
    assert bool(torch.isnan(y[rows - 1].float()).all())
    assert torch.equal(y[: rows - 1], clean[: rows - 1])
    assert torch.equal(h[: rows - 1], ch[: rows - 1]) and torch.equal(hs[: rows - 1], cs[: rows - 1])
    assert bool(((h[rows - 1] & 0x7F) == 0x7F).all())
    # no expert has rows: nothing is written
    y = run_matmul(x, xs, w, ws, np.zeros_like(offsets))
    assert bool((y == 9.0).all())
    # offsets that leave the tensors are held to them
    wild = offsets.copy()
    wild[-1] = rows + 1000
    y = run_matmul(x, xs, w, ws, wild, rows)
    assert torch.equal(y[:rows], clean[:rows]) and bool((y[rows:] == 9.0).all())


# many workgroups: the tiles that the cases above are too small for
WIDE_PRODUCTS = [
    (64, 300, 1024, 256, "even", 3), (64, 400, 1024, 640, "spread", 0), (16, 500, 4096, 256, "spread", 0),
    (16, 1200, 4096, 128, "spread", 2), (16, 2400, 4096, 384, "spread", 0), (2, 709, 4416, 256, "even", 0),
    (3, 700, 4600, 128, "first", 1), (1, 64, 7168, 384, "even", 0), (40, 1800, 2048, 128, "spread", 1),
    (12, 960, 5120, 256, "even", 0), (10, 1900, 5120, 128, "spread", 3)]


@pytest.mark.parametrize("E,rows,n,k,kind,spare", WIDE_PRODUCTS)
def test_wide_matmul(E, rows, n, k, kind, spare):
    test_matmul(E, rows, n, k, kind, spare)


@pytest.mark.parametrize("E,rows,n,k,kind,spare", WIDE_PRODUCTS)
def test_wide_gate_up(E, rows, n, k, kind, spare):
    test_gate_up(E, rows, n // 256 * 128, k, kind, spare)


@pytest.mark.parametrize("rows", [2, 30, 130, 200, 300])
def test_widest_rows(rows):
    """The widest rows that the calls take: 512 blocks of 128."""
    say(f"[gpu] products of the widest rows rows={rows}")
    g = rng(14, rows)
    k = 65536
    ins = grouped_inputs(g, 1, 16, k, [rows], 0, 0.3)
    ref, big = R.product(*ins)
    check_product(R.f64(run_matmul(*ins)[:rows]), ref, big, big * R.BLOCK)
    if rows > 130:
        return
    x, xs, w, ws, offsets = grouped_inputs(g, 1, 256, k, [rows], 0, 0.3)
    ws *= np.float32(2.0 ** -4 / np.sqrt(k / 128))
    h, hs = run_gate_up(x, xs, w, ws, offsets)
    check_gate_up(h[:rows].cpu().numpy(), R.f64(hs[:rows]), x, xs, w, ws, offsets)


@pytest.mark.parametrize("rows", [3, 150])
def test_widest_outputs(rows):
    """The widest outputs that the calls take."""
    test_matmul(2, rows, 65536, 128, "even", 1)
    test_matmul(1, rows, 65528, 128, "even", 0)
    test_gate_up(2, rows, 65536, 128, "even", 1)


def test_matmul_long_offsets():
    """Rows and weights past 2^31 bytes."""
    say("[gpu] matmul past 32 bits")
    k, n, rows = 7168, 8, 310000
    x = torch.zeros((rows, k), dtype=torch.uint8, device=DEV)
    x[-1] = 0x38                                          # 1.0
    x[0] = 0x40                                           # 2.0
    xs = torch.ones((rows, k // 128), device=DEV)
    w = torch.full((1, n, k), 0x38, dtype=torch.uint8, device=DEV)
    ws = torch.ones((1, 1, k // 128), device=DEV)
    offsets = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    y = torch.empty((rows, n), dtype=torch.bfloat16, device=DEV)
    mep.moe_expert_matmul(rows, 1, n, k, x, xs, offsets, w, ws, y)
    torch.cuda.synchronize()
    assert bool((y[-1] == k).all()) and bool((y[0] == 2 * k).all()) and bool((y[1:-1] == 0).all())
    del x, xs, w, y
    E, n, k = 24, 16384, 8192                             # 3.2 GB of weights
    w = torch.zeros((E, n, k), dtype=torch.uint8, device=DEV)
    w[-1, -1] = 0x38
    ws = torch.ones((E, n // 128, k // 128), device=DEV)
    x = torch.full((4, k), 0x38, dtype=torch.uint8, device=DEV)
    xs = torch.ones((4, k // 128), device=DEV)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[-1] = 4
    y = torch.empty((4, n), dtype=torch.bfloat16, device=DEV)
    mep.moe_expert_matmul(4, E, n, k, x, xs, offsets, w, ws, y)
    torch.cuda.synchronize()
    assert bool((y[:, -1] == k).all()) and bool((y[:, :-1] == 0).all())


@pytest.mark.parametrize("E,rows,n,k", [(8, 60, 256, 256), (70, 300, 1024, 256), (6, 1200, 4096, 128),
                                        (6, 2400, 4096, 256)])
def test_offsets_out_of_order(E, rows, n, k):
    """Offsets that break their contract: any result, nothing outside it."""
    say(f"[gpu] offsets out of order E={E} rows={rows} n={n} k={k}")
    g = rng(18, E, rows)
    ins = list(grouped_inputs(g, E, n, k, counts_of("even", E, rows, g), 0))
    want = run_matmul(*ins)
    fine = run_gate_up(*ins[:4], ins[4])
    for bad in (np.linspace(rows, 0, E + 1), np.where(np.arange(E + 1) % 2, rows, 0),
                g.integers(-2 ** 31, 2 ** 31 - 1, E + 1), np.full(E + 1, -5), np.full(E + 1, rows + 99)):
        y = run_matmul(*ins[:4], bad.astype(np.int32))
        assert bool((y[rows:] == 9.0).all())
        h, hs = run_gate_up(*ins[:4], bad.astype(np.int32))
        assert bool((h[rows:] == 5).all()) and bool((hs[rows:] == 9.0).all())
    assert torch.equal(run_matmul(*ins), want)
    again = run_gate_up(*ins[:4], ins[4])
    assert all(torch.equal(a, b) for a, b in zip(fine, again))


# --- the few-token layer ----------------------------------------------------------------------------

def few_inputs(g, T, E, K, H, F):
    x = R.bf16(g.standard_normal((T, H)) * np.where(g.random(H) < 0.02, 10, 1)).to(DEV)
    w13, s13 = R.make_weights(g, E, 2 * F, H)
    w2, s2 = R.make_weights(g, E, H, F)
    s13 *= np.float32(2.0 ** 4 / np.sqrt(H))
    s2 *= np.float32(2.0 ** 4 / np.sqrt(F))
    idx = np.stack([g.permutation(E)[:K] if K <= E else g.integers(0, E, K) for _ in range(T)]).astype(np.int32)
    w = g.random((T, K)).astype(np.float32)
    return x, idx, w, w13, s13, w2, s2


def few_ref(x, idx, w, w13, s13, w2, s2):
    """(out, noise): noise is what a code of h one step away from the
    reference's can add -- the kernel's fp32 value of h may lie on the other
    side of a rounding border; counted for one value of each block of 128."""
    xv = R.coded(R.f64(x))
    T, K = idx.shape
    out, noise = np.zeros((T, w2.shape[1])), np.zeros((T, w2.shape[1]))
    F = w2.shape[2]
    for t in range(T):
        for k in range(K):
            e = idx[t, k]
            if not 0 <= e < w13.shape[0]:
                continue
            a = R.weights_value(w13[e], s13[e]) @ xv[t]
            h = R.coded((R.silu(a[:F]) * a[F:])[None])[0]
            wv = R.weights_value(w2[e], s2[e])
            out[t] += w[t, k] * (wv @ h)
            # one code per block moves by one step (2^-3 of it) at most
            step = np.abs(wv * h * 2.0 ** -3).reshape(len(wv), -1, R.BLOCK).max(-1).sum(-1)
            noise[t] += np.abs(w[t, k]) * (step + 2.0 ** -18 * np.abs(wv * h).sum(-1))
    return out, noise


def run_few(x, idx, w, w13, s13, w2, s2, ws=None):
    T, H = x.shape
    E, F, K = w13.shape[0], w2.shape[2], idx.shape[1]
    out = torch.full((T + 1, H), 9.0, dtype=torch.bfloat16, device=DEV)
    if ws is None:
        ws = torch.full((mep.moe_few_token_workspace(T, K, H, F),), 0xFF, dtype=torch.uint8, device=DEV)
    mep.moe_few_token_layer(T, E, K, H, F, x, dev(idx), dev(w), dev(w13), dev(s13), dev(w2), dev(s2),
                            out, ws)
    torch.cuda.synchronize()
    assert bool((out[T] == 9.0).all())
    return out[:T]


def check_few(out, ref, noise):
    assert np.all(np.abs(R.f64(out) - ref) <= R.BF16_HALF * np.abs(ref) + 1.01 * noise + 2.0 ** -133)


@pytest.mark.parametrize("T,E,K,H,F", [
    (1, 1, 1, 128, 128), (1, 8, 3, 384, 256), (2, 8, 8, 256, 640), (3, 300, 8, 128, 128),
    (15, 8, 2, 1152, 128), (16, 3, 3, 256, 256), (17, 4, 2, 384, 128), (32, 2, 2, 256, 128),
    (33, 5, 2, 128, 384), (64, 3, 2, 256, 128), (64, 64, 4, 128, 128), (5, 1024, 64, 128, 128),
    (64, 70, 64, 128, 128), (40, 2, 64, 128, 128), (3, 2, 2, 65536, 128), (20, 2, 2, 128, 65536),
    (6, 2, 1, 128, 65536), (18, 3, 1, 65536, 128)])
def test_few(T, E, K, H, F):
    say(f"[gpu] few T={T} E={E} K={K} H={H} F={F}")
    ins = few_inputs(rng(9, T, E, K, H, F), T, E, K, H, F)
    check_few(run_few(*ins), *few_ref(*ins))


@pytest.mark.parametrize("T", [3, 13, 16, 21, 50])
def test_few_one_expert(T):
    """Every token names the same expert, and one more each."""
    say(f"[gpu] few, one expert T={T}")
    E, K, H, F = 64, 2, 384, 256
    x, idx, w, *wts = few_inputs(rng(16, T), T, E, K, H, F)
    idx[:, 1] = 7
    idx[:, 0] = np.where(np.arange(T) % 3 == 0, 7, (np.arange(T) * 5) % E)
    check_few(run_few(x, idx, w, *wts), *few_ref(x, idx, w, *wts))


def test_few_padding_and_repeats():
    """Ids outside the experts name none; a token with none gets zeros; an
    expert named twice counts twice; what pads a batch cannot reach it."""
    say("[gpu] few padding and repeats")
    T, E, K, H, F = 19, 6, 4, 256, 128
    x, idx, w, *wts = few_inputs(rng(10), T, E, K, H, F)
    idx[0] = -1
    idx[1] = [2, 2, 5, 2]
    idx[2] = [E, -5, 3, 1 << 30]
    idx[3] = [4, -1, -1, 4]
    idx[T - 4:] = -1
    x[T - 4:] = float("nan")
    w[T - 4:] = np.nan
    w[0] = np.inf
    w[2, [0, 1, 3]] = np.nan
    out = run_few(x, idx, w, *wts)
    assert bool((out[0] == 0).all()) and bool((out[T - 4:] == 0).all())
    live = slice(1, T - 4)
    wl = w.copy()
    wl[(idx < 0) | (idx >= E)] = 0
    ref, noise = few_ref(x[live], idx[live], wl[live], *wts)
    check_few(out[live], ref, noise)
    # nobody names an expert
    out = run_few(x, np.full_like(idx, -1), w, *wts)
    assert bool((out == 0).all())
    # the same batch without its padding, and a NaN token beside others
    a = run_few(x[:8].contiguous(), idx[:8], wl[:8], *wts)
    y = x[:8].clone()
    y[5] = float("nan")
    b = run_few(y, idx[:8], wl[:8], *wts)
    keep = [0, 1, 2, 3, 4, 6, 7]
    assert torch.equal(a[keep], b[keep]) and bool(torch.isnan(b[5].float()).all())


# --- together, captured, on other streams -------------------------------------------------------------

def layer_weights(E, H, F, seed):
    g = rng(11, seed)
    w13, s13 = R.make_weights(g, E, 2 * F, H)
    w2, s2 = R.make_weights(g, E, H, F)
    return w13, (s13 * np.float32(2.0 ** 4 / np.sqrt(H))), w2, (s2 * np.float32(2.0 ** 4 / np.sqrt(F)))


class Layer:
    """norm -> route -> dispatch (e4m3) -> gate_up -> matmul -> combine, as a user runs it."""

    def __init__(self, N, T, H, E, K, F, seed=0):
        self.dims = N, T, H, E, K, F
        g = rng(12, seed)
        self.x = R.bf16(g.standard_normal((N * T, H))).to(DEV)
        self.r = R.bf16(g.standard_normal((N * T, H))).to(DEV)
        self.nw = R.bf16(1 + 0.1 * g.standard_normal(H)).to(DEV)
        self.logits = torch.from_numpy(g.standard_normal((N * T, E)).astype(np.float32)).to(DEV)
        self.host = layer_weights(E, H, F, seed)
        self.wts = [dev(a) for a in self.host]
        rows = N * T * K
        e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
        self.y, self.ro = e(N * T, H, dt=torch.bfloat16), e(N * T, H, dt=torch.bfloat16)
        self.idx, self.w = e(N * T, K, dt=torch.int32), e(N * T, K)
        self.ex, self.es = e(rows, H, dt=torch.uint8), e(rows, H // 128)
        self.off = e(E + 1, dt=torch.int32)
        self.h, self.hs = e(rows, F, dt=torch.uint8), e(rows, F // 128)
        self.ey, self.out = e(rows, H, dt=torch.bfloat16), e(N * T, H, dt=torch.bfloat16)
        self.few_out = e(N * T, H, dt=torch.bfloat16)
        self.ws = e(max(1, mep.moe_few_token_workspace(min(64, N * T), K, H, F)), dt=torch.uint8)
        self.g = mep.moe_group_create(N, E, K, H, T, mep.MOE_FP8_E4M3)

    def run(self):
        N, T, H, E, K, F = self.dims
        w13, s13, w2, s2 = self.wts
        mep.moe_add_rmsnorm(N * T, H, self.x, self.r, self.nw, 1e-6, self.ro, self.y, None, None)
        mep.moe_topk_route(N * T, E, K, self.logits, mep.MOE_FP32, True, self.idx, self.w)
        mep.moe_dispatch_send(self.g, T, self.y, self.idx)
        mep.moe_dispatch_recv(self.g, self.ex, self.es, self.off)
        mep.moe_expert_gate_up(N * T * K, E, F, H, self.ex, self.es, self.off, w13, s13, self.h, self.hs)
        mep.moe_expert_matmul(N * T * K, E, H, F, self.h, self.hs, self.off, w2, s2, self.ey)
        mep.moe_combine_send(self.g, self.ey)
        mep.moe_combine_recv(self.g, self.w, self.out)

    def run_few(self):
        N, T, H, E, K, F = self.dims
        mep.moe_few_token_layer(N * T, E, K, H, F, self.y, self.idx, self.w, *self.wts, self.few_out,
                                self.ws)

    def results(self):
        return [t.clone() for t in (self.ro, self.y, self.idx, self.w, self.ex, self.es, self.off, self.h,
                                    self.hs, self.ey, self.out)]

    def close(self):
        torch.cuda.synchronize()
        assert mep.moe_group_status(self.g) == mep.MOE_OK
        mep.moe_group_destroy(self.g)


def test_whole_layer():
    """The layer through dispatch and combine, and the few-token layer on the
    same rows, against the definition."""
    N, T, H, E, K, F = 4, 11, 384, 16, 3, 256
    say("[gpu] whole layer")
    L = Layer(N, T, H, E, K, F)
    try:
        L.run()
        L.run_few()
        torch.cuda.synchronize()
        w13, s13, w2, s2 = L.host
        idx, w = L.idx.cpu().numpy(), L.w.cpu().numpy()
        ref, noise = few_ref(L.y, idx, w, w13, s13, w2, s2)
        check_few(L.few_out, ref, noise)
        # through dispatch every expert output is rounded to bf16, and its block sums come from
        # the e4m3 instruction: at most 2^-10 of a block's largest product
        extra = np.zeros_like(ref)
        xv = R.coded(R.f64(L.y))
        for t in range(N * T):
            for k in range(K):
                e = idx[t, k]
                a = R.weights_value(w13[e], s13[e]) @ xv[t]
                h = R.coded((R.silu(a[:F]) * a[F:])[None])[0]
                p = R.weights_value(w2[e], s2[e]) * h
                extra[t] += w[t, k] * (R.BF16_HALF * np.abs(p.sum(-1)) +
                                       2.0 ** -10 * np.abs(p).reshape(H, -1, 128).max(-1).sum(-1))
        check_few(L.out, ref, noise + extra)
    finally:
        L.close()


def test_captured_layers():
    """Two layers captured into two graphs, replayed in turn and at once on
    two streams between eager runs: every replay gives the eager bits."""
    say("[gpu] captured layers")
    layers = [Layer(2, 9, 256, 8, 2, 128, 1), Layer(4, 16, 384, 16, 4, 256, 2)]
    try:
        want, few, graphs = [], [], []
        for L in layers:
            L.run()
            L.run_few()
            torch.cuda.synchronize()
            want.append(L.results())
            few.append(L.few_out.clone())
        for L in layers:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                L.run()
                L.run_few()
            graphs.append(graph)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for rep in range(4):
            for L in layers:
                for t in (L.out, L.few_out, L.ey, L.hs, L.w, L.y):
                    t.fill_(float("nan"))
                L.ws.fill_(0xFF)
            torch.cuda.synchronize()
            for s, graph in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
            torch.cuda.synchronize()
            for L, w, f in zip(layers, want, few):
                assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(L.results(), w))
                assert torch.equal(L.few_out, f)
            if rep == 1:
                for L in layers:
                    L.run()
                    L.run_few()
                torch.cuda.synchronize()
    finally:
        for L in layers:
            L.close()


def test_first_call_captured():
    """The first call of a tile size may be the captured one."""
    say("[gpu] first call captured")
    E, n, k, rows = 2, 264, 256, 240
    g = rng(15)
    ins = grouped_inputs(g, E, n, k, counts_of("even", E, rows, g), 0)
    d = [dev(a) for a in ins]
    y = torch.zeros((rows, n), dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mep.moe_expert_matmul(rows, E, n, k, d[0], d[1], d[4], d[2], d[3], y)
    want = run_matmul(*ins)[:rows]
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("E,rows,n,k", [(3, 40, 512, 640), (16, 500, 4096, 256), (16, 2400, 4096, 384)])
def test_products_captured_and_at_once(E, rows, n, k):
    """Captured products of each size, replayed on two streams at once."""
    say(f"[gpu] products captured E={E} rows={rows} n={n} k={k}")
    g = rng(19, E, rows)
    x, xs, w, ws, offsets = grouped_inputs(g, E, n, k, counts_of("spread", E, rows, g), 0)
    y = run_matmul(x, xs, w, ws, offsets)[:rows]
    h, hs = (t[:rows] for t in run_gate_up(x, xs, w, ws, offsets))
    d = [dev(a) for a in (x, xs, offsets, w, ws)]
    outs = [(torch.empty_like(y), torch.empty_like(h), torch.empty_like(hs)) for _ in range(2)]
    graphs = []
    torch.cuda.synchronize()
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mep.moe_expert_matmul(rows, E, n, k, *d, o[0])
            mep.moe_expert_gate_up(rows, E, n // 2, k, *d, o[1], o[2])
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for o in outs:
            for t in o:
                t.view(torch.uint8).fill_(0xFF)
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, (y, h, hs)))


def test_two_streams_at_once():
    """The same calls on two streams at once, each with its own outputs."""
    say("[gpu] two streams")
    g = rng(13)
    ins = few_inputs(g, 12, 16, 4, 1024, 512)
    want = run_few(*ins)
    x, idx, w, *wts = ins
    d = [x, dev(idx), dev(w)] + [dev(a) for a in wts]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(x) for _ in streams]
    ws = [torch.empty(mep.moe_few_token_workspace(12, 4, 1024, 512), dtype=torch.uint8, device=DEV)
          for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, b in zip(streams, outs, ws):
            mep.moe_few_token_layer(12, 16, 4, 1024, 512, *d, o, b, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_tensor_refusals():
    say("[gpu] tensor refusals")
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(256, dtype=torch.bfloat16, device=DEV)

    def refused(match, *a, **kw):
        with pytest.raises(mep.MoeError, match=match) as ei:
            mep.moe_add_rmsnorm(*a, **kw)
        assert ei.value.status == mep.MOE_ERR_INVALID

    refused("x dtype", 4, 256, x.float(), None, w, 1e-6, None, x, None, None)
    refused("x not contiguous", 4, 128, x[:, :128], None, w, 1e-6, None, x, None, None)
    refused("y 2048 bytes", 5, 256, torch.zeros((5, 256), dtype=torch.bfloat16, device=DEV), None, w, 1e-6,
            None, x, None, None)
    refused("weight not a device tensor", 4, 256, x, None, w.cpu(), 1e-6, None, x, None, None)
    big = torch.zeros((5, 256), dtype=torch.bfloat16, device=DEV)
    refused("invalid argument", 4, 256, big.view(-1)[1:1025].view(4, 256), None, w, 1e-6, None, x, None, None)


def test_bench_layer():
    """The bench's layer run: every operator and the few-token layer timed."""
    import argparse

    import bench
    from workloads import CONFIGS
    say("[gpu] bench layer, tiny")
    rec = bench.layer_run(CONFIGS["A"], argparse.Namespace(steps=3, warmup=1, expert_width=256))
    assert list(rec["us"]) == ["add_rmsnorm", "topk_route", "dispatch", "expert_gate_up", "expert_matmul",
                               "combine"]
    assert rec["value"] > 0 and all(t > 0 for t in rec["us"].values())
    assert list(rec["few_token_us"]) == ["1", "8", "32"]
