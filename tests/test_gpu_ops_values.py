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
