"""The operators at values where fp32 work can lose what the result keeps:
rows whose squares leave fp32's range, logits far below the largest, gates
where the exponential is large, sums that cancel.  Against the definitions in
64 bits; tolerances from the arithmetic, beside each test.
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


def rng(*key):
    return np.random.default_rng([11, *key])


# --- norm ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1e-31, 1e-24, 1e-6])
@pytest.mark.parametrize("rows,hidden", [(70, 24), (70, 128), (37, 384), (9, 520), (9, 1152), (9, 2048), (5, 7168),
                                         (3, 16384), (3, 32768)])
def test_norm_small_rows(rows, hidden, eps):
    """Rows down to bf16's smallest numbers, beside ordinary ones, with an eps
    as small: the squares underflow, the norm is an ordinary number.  Mean,
    root and the two products are fewer than 64 roundings of 2^-24: 2^-18; and
    2^-18 for squares that were left below the smallest normal number."""
    say(f"[gpu] norm small rows={rows} hidden={hidden} eps={eps}")
    g = rng(1, rows, hidden)
    size = np.exp2(np.resize([-133, 0, -126, -75, -63, -60, -55, -50, -45, -100, -40], rows))[:, None]
    v = g.standard_normal((rows, hidden)) * size
    v[:, 3] *= 40
    x, r, w = (R.bf16(a).to(DEV) for a in (v, 0.5 * v, 1 + 0.3 * g.standard_normal(hidden)))
    eps = float(np.float32(eps))
    for res in (None, r):
        y = torch.empty_like(x)
        fp8 = hidden % 128 == 0
        yq = torch.empty((rows, hidden), dtype=torch.uint8, device=DEV) if fp8 else None
        ys = torch.empty((rows, hidden // 128), device=DEV) if fp8 else None
        mep.moe_add_rmsnorm(rows, hidden, x, res, w, eps, None, y, yq, ys)
        torch.cuda.synchronize()
        s = R.f64(x) + (0 if res is None else R.f64(res))
        with np.errstate(invalid="ignore"):
            ref = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * R.f64(w)
        live = np.isfinite(ref).all(-1)              # a row of zeros with eps 0 has no norm
        assert live.sum() >= rows - rows // 11 - 1
        rel = 2.0 ** -17
        got = R.f64(y)
        assert np.all(np.abs(got - ref)[live] <= ((R.BF16_HALF + rel) * np.abs(ref) + 2.0 ** -133)[live])
        if fp8:
            scale, _ = R.block_scale(ref[live])
            assert np.all(np.abs(R.f64(ys)[live] - scale) <= rel * scale)
            got = R.rows_value(yq.cpu().numpy()[live], R.f64(ys)[live].astype(np.float32))
            tol = (R.E4M3_HALF + 2 * rel) * np.abs(ref[live]) + (2.0 ** -10 + rel) * scale.repeat(R.BLOCK, -1)
            assert np.all(np.abs(got - ref[live]) <= tol)


@pytest.mark.parametrize("size,scale", [(2.0 ** -60, 2.0 ** 90), (2.0 ** -130, 2.0 ** 70), (2.0 ** 40, 2.0 ** -110)])
def test_norm_far_weights(size, scale):
    """Rows and weights at opposite ends: 1/rms times the weight leaves fp32's
    range, the result does not."""
    say(f"[gpu] norm far weights {size} {scale}")
    for hidden in (128, 2048):
        g = rng(4, hidden)
        x, w = R.bf16(size * g.standard_normal((7, hidden))).to(DEV), R.bf16(scale * g.standard_normal(hidden)).to(DEV)
        y = torch.empty_like(x)
        mep.moe_add_rmsnorm(7, hidden, x, None, w, 0.0, None, y, None, None)
        torch.cuda.synchronize()
        s = R.f64(x)
        ref = s / np.sqrt((s * s).mean(-1, keepdims=True)) * R.f64(w)
        assert np.all(np.abs(R.f64(y) - ref) <= (R.BF16_HALF + 2.0 ** -17) * np.abs(ref) + 2.0 ** -133)


def test_norm_zero_rows():
    """A row of zeros is zero with any eps above 0; with eps 0 it is 0/0, NaN,
    and so are its codes; its neighbours are as ever."""
    say("[gpu] norm zero rows")
    for hidden in (128, 384, 1152, 2048, 7168):
        x = torch.ones((5, hidden), dtype=torch.bfloat16, device=DEV)
        x[1] = 0
        x[4] = 0
        w = torch.ones(hidden, dtype=torch.bfloat16, device=DEV)
        for eps in (0.0, 1e-45, 1e-20):
            y = torch.empty_like(x)
            yq = torch.empty((5, hidden), dtype=torch.uint8, device=DEV)
            ys = torch.empty((5, hidden // 128), device=DEV)
            mep.moe_add_rmsnorm(5, hidden, x, None, w, eps, None, y, yq, ys)
            torch.cuda.synchronize()
            assert bool((y[[0, 2, 3]] == 1).all()) and bool((ys[[1, 4]] == 1).all())
            for t in (1, 4):
                if eps == 0:
                    assert bool(torch.isnan(y[t].float()).all()) and bool(((yq[t] & 0x7F) == 0x7F).all())
                else:
                    assert bool((y[t] == 0).all()) and bool((yq[t] == 0).all())


# --- routing --------------------------------------------------------------------------------------

@pytest.mark.parametrize("E,K", [(8, 8), (16, 12), (50, 16), (128, 16), (256, 16), (64, 40), (200, 64), (512, 64),
                                 (1024, 64)])
@pytest.mark.parametrize("bf", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_far_weights(E, K, bf, renorm):
    """Weights of experts far below the best.  The best logit is 0, so z - best
    is exact.  In roundings of 2^-24: the exponential of a chosen expert 4 (its
    argument's and the instruction's last place); the sum of all of them, at
    most 22 additions in a row, and its terms' 2 + |z|, of which the softmax
    mean of |z| counts, at most 5 for 1024 experts; the quotient 1: below
    2^-19."""
    say(f"[gpu] route far weights E={E} K={K} bf16={bf} renorm={renorm}")
    g = rng(2, E, K)
    T = 300
    z = -85 * g.random((T, E)) ** 0.7
    z[np.arange(T), g.integers(0, E, T)] = 0
    z[:20, :] = np.where(z[:20] == 0, 0, -5.5)          # many near the best: the sum's worst
    t = torch.from_numpy(z.astype(np.float32)).to(torch.bfloat16 if bf else torch.float32).to(DEV)
    idx = torch.empty((T, K), dtype=torch.int32, device=DEV)
    w = torch.empty((T, K), device=DEV)
    mep.moe_topk_route(T, E, K, t, mep.MOE_BF16 if bf else mep.MOE_FP32, renorm, idx, w)
    torch.cuda.synchronize()
    v = R.f64(t)
    order = np.argsort(-v, axis=-1, kind="stable")[:, :K]
    assert np.array_equal(idx.cpu().numpy(), order)
    p = np.exp(v)
    ref = np.take_along_axis(p, order, -1)
    ref = ref / (ref if renorm else p).sum(-1, keepdims=True)
    assert np.all(np.abs(R.f64(w) - ref) <= 2.0 ** -19 * ref + 2.0 ** -126)


# --- the experts' activation ------------------------------------------------------------------------

def one_hot_rows(rows, k):
    """Rows of a single code 1 at place 0, scale 1."""
    x = torch.zeros((rows, k), dtype=torch.uint8, device=DEV)
    x[:, 0] = 0x38
    return x, torch.ones((rows, k // 128), device=DEV)


GATES = np.concatenate([-np.exp2(np.linspace(-6, 6.4, 40)), [0.0, -86.5, 1.0, 17.0, 88.0]])


def gate_weights(f, k):
    """Weights whose gate and up products of a one-hot row are a code times a
    scale: gate block b has the gates GATES[b] * (1 .. 15)/8, rounded to fp32
    with the scale; up is 1."""
    w = torch.zeros((2 * f, k), dtype=torch.uint8)
    w[:f, 0] = torch.arange(f).remainder(8).to(torch.uint8) + 0x38          # 1, 1.125 .. 1.875
    w[f:, 0] = 0x38
    s = torch.ones((2 * f // 128, k // 128))
    s[: f // 128, 0] = torch.from_numpy(np.resize(GATES, f // 128).astype(np.float32))
    code = 1 + np.arange(f) % 8 / 8
    gate = np.repeat(s[: f // 128, 0].double().numpy(), 128) * code
    return w[None].contiguous().to(DEV), s[None].contiguous().to(DEV), gate


@pytest.mark.parametrize("rows", [1, 200])
def test_gate_up_scales_of_large_gates(rows):
    """The scale is the block's largest |silu(gate)| / 448 in fp32.  The gate is
    a code times the scale, rounded once, which the reference rounds alike; in
    roundings of 2^-24: exponential 4, sum 1, quotient 3 at most, division by
    448 1: 9."""
    say(f"[gpu] gate_up scales of large gates rows={rows}")
    f, k = 128 * len(GATES), 128
    x, xs = one_hot_rows(rows, k)
    w, ws, gate = gate_weights(f, k)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    h = torch.empty((rows, f), dtype=torch.uint8, device=DEV)
    hs = torch.empty((rows, f // 128), device=DEV)
    mep.moe_expert_gate_up(rows, 1, f, k, x, xs, off, w, ws, h, hs)
    torch.cuda.synchronize()
    v = gate.astype(np.float32).astype(np.float64)
    ref = np.abs(v / (1 + np.exp(-v))).reshape(-1, 128)
    at = ref.argmax(-1)
    want = ref.max(-1) / 448
    g = np.abs(v.reshape(-1, 128)[np.arange(len(at)), at])
    want = np.where(want == 0, 1.0, np.maximum(want, 2.0 ** -126))
    got = R.f64(hs)
    assert np.all(got == got[:1])
    off_by = np.abs(got[0] - want) / want * 2.0 ** 24
    normal = want > 2.0 ** -120
    assert np.all(off_by[normal] <= 9), (g[normal], off_by[normal])


@pytest.mark.parametrize("rows", [1, 200])
def test_gate_up_far_gates(rows):
    """Gates to -88.5, where exp(-gate) nears fp32's largest number and its
    reciprocal is below the normal ones: silu is still an ordinary number, and
    counts where up is large.  Roundings as above, and one of h = silu * up."""
    say(f"[gpu] gate_up far gates rows={rows}")
    gates = np.float32([-20, -60, -80, -86.5, -87, -87.25, -87.5, -88, -88.25, -88.5])
    f, k = 128 * len(gates), 128
    x, xs = one_hot_rows(rows, k)
    w = torch.zeros((1, 2 * f, k), dtype=torch.uint8, device=DEV)
    w[:, :, 0] = 0x38
    ws = torch.full((1, 2 * len(gates), 1), 2.0 ** 60, device=DEV)
    ws[0, : len(gates), 0] = torch.from_numpy(gates).to(DEV)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    h = torch.empty((rows, f), dtype=torch.uint8, device=DEV)
    hs = torch.empty((rows, f // 128), device=DEV)
    mep.moe_expert_gate_up(rows, 1, f, k, x, xs, off, w, ws, h, hs)
    torch.cuda.synchronize()
    v = gates.astype(np.float64)
    want = np.abs(v / (1 + np.exp(-v))) * 2.0 ** 60 / 448
    got = R.f64(hs)
    assert np.all(got == got[:1])
    # silu below the normal numbers is rounded at 2^-149: nothing here is that small
    assert np.all(np.abs(got[0] - want) <= 10 * 2.0 ** -24 * want), got[0] / want - 1


def test_silu_alike():
    """gate_up and the few-token layer form the same h: with one expert, one
    token and one block of f they give the same bits through the same down product."""
    say("[gpu] silu alike")
    H, k = 128, 128
    for gate in (0.3, -3.0, -21.0, -60.0, 5.0):
        f = 128
        w = torch.zeros((1, 2 * f, k), dtype=torch.uint8, device=DEV)
        w[0, :f, 0] = (torch.arange(f) % 8).to(torch.uint8).to(DEV) + 0x38
        w[0, f:, 0] = 0x38
        s13 = torch.ones((1, 2, 1), device=DEV)
        s13[0, 0, 0] = gate
        x = torch.zeros((1, k), dtype=torch.bfloat16, device=DEV)
        x[0, 0] = 1.0                                      # codes as 448, scale 1/448
        q = torch.zeros((1, k), dtype=torch.uint8, device=DEV)
        q[0, 0] = 0x7E
        xs = torch.full((1, 1), 1.0 / 448, device=DEV)
        off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
        h = torch.empty((1, f), dtype=torch.uint8, device=DEV)
        hs = torch.empty((1, 1), device=DEV)
        mep.moe_expert_gate_up(1, 1, f, k, q, xs, off, w, s13, h, hs)
        # the down product of the few-token layer picks out h's codes one by one, and adds the
        # scale's last bits: w2 = 1 at (n, n), s2 = 1, so out[n] = bf16(code * scale)
        w2 = torch.zeros((1, H, f), dtype=torch.uint8, device=DEV)
        w2[0, torch.arange(f), torch.arange(f)] = 0x38
        s2 = torch.ones((1, 1, 1), device=DEV)
        out = torch.empty((1, H), dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(mep.moe_few_token_workspace(1, 1, H, f), dtype=torch.uint8, device=DEV)
        idx = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
        mep.moe_few_token_layer(1, 1, 1, H, f, x, idx, torch.ones((1, 1), device=DEV), w, s13, w2, s2, out, ws)
        torch.cuda.synchronize()
        want = (h.view(torch.float8_e4m3fn).float() * hs).to(torch.bfloat16)
        assert torch.equal(out, want), gate


# --- the product's sums -----------------------------------------------------------------------------

def product_bound(x, w):
    """Of rows x [r][k] and weights w [n][k] (values, scales 1): the product in
    64 bits and what the call may add to it.  Of every 8 consecutive products,
    seven are cut by less than 2^-13 of the largest (a code below 2^-6, the
    smallest normal one, counts as that); the other sums are fp32, 16 of 8 in a
    block and then the blocks, each addition off by 2^-23 of the magnitudes at
    most; and the result is rounded to bf16."""
    p = x[:, None, :] * w[None]
    floor = lambda v: np.where(v == 0, 0, np.maximum(np.abs(v), 2.0 ** -6))  # noqa: E731
    top = (floor(x)[:, None, :] * floor(w)[None]).reshape(*p.shape[:2], -1, 8).max(-1).sum(-1)
    ref = p.sum(-1)
    off = 7 * 2.0 ** -13 * top + (16 + x.shape[1] // 128) * 2.0 ** -23 * np.abs(p).sum(-1)
    return ref, R.BF16_HALF * (np.abs(ref) + off) + off


@pytest.mark.parametrize("kind", ["outliers", "cancelling", "subnormal", "random"])
@pytest.mark.parametrize("rows,n", [(16, 64), (300, 16384)])
def test_matmul_bound(kind, rows, n):
    """The documented bound, where one product of every 8 is far above the
    rest, where such products cancel, and among the format's smallest numbers;
    in the narrow kernel and in a tile (whose first and last rows are looked at)."""
    say(f"[gpu] matmul bound {kind} rows={rows} n={n}")
    g = rng(3, rows, n)
    k = 1024
    lut = R.LUT
    pick = lambda lo, hi, shape: (lambda v: g.choice(v, shape) * g.choice([1.0, 1.0, -1.0], shape))(  # noqa: E731
        lut[(lut >= lo) & (lut <= hi)])
    some = 24
    x, w = pick(0.5, 8, (some, k)), pick(0.5, 4, (64, k))
    if kind in ("outliers", "cancelling"):
        x[:, ::8], w[:, ::8] = pick(256, 448, (some, k // 8)), pick(256, 448, (64, k // 8))
        x[some // 2:], w[32:] = np.abs(x[some // 2:]), np.abs(w[32:])          # cuts that add up
        # products just below a multiple of what is kept beside 256 * 256
        x[::3, 1:8], w[::3, 1:8], x[::3, 0], w[::3, 0] = 3.75, 2, 256, 256
    if kind == "cancelling":
        x[:, 8::16], w[:, 8::16] = -x[:, ::16], w[:, ::16]
    if kind == "subnormal":
        x, w = pick(2.0 ** -9, 2.0 ** -5, (some, k)), pick(2.0 ** -9, 1, (64, k))
        w[:, ::8] = 256
    if kind == "random":
        x, w = pick(2.0 ** -9, 448, (some, k)), pick(2.0 ** -9, 448, (64, k))
    ref, tol = product_bound(x, w)
    codes = lambda v: torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn)  # noqa: E731
    xr = codes(np.resize(x, (rows, k))).to(DEV)
    wr = codes(np.resize(w, (n, k)))[None].contiguous().to(DEV)
    xs = torch.ones((rows, k // 128), device=DEV)
    ws = torch.ones((1, n // 128 + (n % 128 > 0), k // 128), device=DEV)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    y = torch.empty((rows, n), dtype=torch.bfloat16, device=DEV)
    mep.moe_expert_matmul(rows, 1, n, k, xr, xs, off, wr, ws, y)
    torch.cuda.synchronize()
    got = R.f64(y)
    m = min(rows, some)
    assert np.all(np.abs(got[:m, :64] - ref[:m]) <= tol[:m])
    assert np.all(np.abs(got[:m, n - 64:] - ref[:m]) <= tol[:m])
    if rows > some:
        last = rows // some * some - some
        assert np.all(np.abs(got[last: last + some, :64] - ref) <= tol)


# --- the stream that is named -------------------------------------------------------------------------

def test_named_stream():
    """Every operator runs on the stream it is given, behind what that stream
    does: inputs are written there late, by a copy behind long work."""
    say("[gpu] named stream")
    E, K, H, F, rows = 8, 2, 256, 128, 16
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    f8 = lambda *s: (20 * rand(*s)).to(torch.float8_e4m3fn)  # noqa: E731
    late = {"x": rand(rows, H).to(torch.bfloat16), "z": rand(rows, E), "q": f8(rows, H)}
    nw, xs, off = rand(H).to(torch.bfloat16), torch.ones((rows, H // 128), device=DEV), torch.tensor(
        [2 * e for e in range(E + 1)], dtype=torch.int32, device=DEV)
    w13, s13 = f8(E, 2 * F, H), torch.full((E, 2 * F // 128, H // 128), 2.0 ** -12, device=DEV)
    w2, s2 = f8(E, H, F), torch.full((E, H // 128, F // 128), 2.0 ** -12, device=DEV)
    idx0 = torch.arange(rows * K, device=DEV, dtype=torch.int32).remainder(E).view(rows, K).contiguous()
    space = torch.empty(mep.moe_few_token_workspace(rows, K, H, F), dtype=torch.uint8, device=DEV)
    big = torch.empty(1 << 28, dtype=torch.float32, device=DEV)

    def run(ins, outs, stream):
        x, z, q = ins["x"], ins["z"], ins["q"]
        y, idx, w, h, hs, p, o = outs
        mep.moe_add_rmsnorm(rows, H, x, None, nw, 1e-6, None, y, None, None, stream=stream)
        mep.moe_topk_route(rows, E, K, z, mep.MOE_FP32, True, idx, w, stream=stream)
        mep.moe_expert_gate_up(rows, E, F, H, q, xs, off, w13, s13, h, hs, stream=stream)
        mep.moe_expert_matmul(rows, E, 2 * F, H, q, xs, off, w13, s13, p, stream=stream)
        mep.moe_few_token_layer(rows, E, K, H, F, x, idx0, w, w13, s13, w2, s2, o, space, stream=stream)

    def outputs():
        e = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
        b = torch.bfloat16
        return (e(rows, H, dt=b), e(rows, K, dt=torch.int32), e(rows, K), e(rows, F, dt=torch.uint8),
                e(rows, F // 128), e(rows, 2 * F, dt=b), e(rows, H, dt=b))

    want = outputs()
    run(late, want, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        ins, got = {k: torch.zeros_like(v) for k, v in late.items()}, outputs()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(8):
                big.fill_(1.0)
            for k, v in late.items():
                ins[k].copy_(v)
        run(ins, got, handle)                          # the current stream is another one
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((want[4] > 0).any()) and bool((want[6] != 0).any())
