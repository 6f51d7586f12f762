"""Experts that hold nearly all rows: as many as the entry points take (2^31 - 1, 34
GB of operands), and a few rows per expert of which one has most.  Whole numbers, so
that all values are exact."""
import ctypes

import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_moe_dispatch_amd as mep  # noqa: E402

DEV = "cuda"
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_most_rows_of_an_expert():
    rows, E, n = (1 << 31) - 1, 2, 8
    b = [0, rows - 10, rows - 5]
    say(f"[gpu] linear, {b[1]} rows of one expert, n = k = {n}")
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    x = torch.empty((rows, n), dtype=BF16, device=DEV)
    for part in x.view(-1).split(1 << 28):
        part.copy_(torch.randint(-3, 4, part.shape, generator=g, device=DEV, dtype=torch.int8))
    w = torch.randint(-3, 4, (E, n, n), generator=g, device=DEV).to(BF16)
    off = torch.tensor(b, dtype=I32, device=DEV)
    ws = torch.empty(max(1, mep.moe_expert_linear_workspace(rows, E, n, n)), dtype=torch.uint8, device=DEV)
    y = torch.empty_like(x)

    def check(weights):
        for e in range(E):
            m = weights[e].float()
            for a in range(b[e], b[e + 1], 1 << 25):
                part = slice(a, min(a + (1 << 25), b[e + 1]))
                assert torch.equal(y[part], (x[part].float() @ m).to(BF16)), (e, a)
        assert bool((y[b[E]:] == 99).all())

    y.fill_(99)
    mep.moe_expert_linear(rows, E, n, n, x, off, w, None, 0, None, None, y, mep.MOE_BF16, ws)
    torch.cuda.synchronize()
    say("[gpu] the product is done")
    check(w.transpose(1, 2))
    y.fill_(99)
    mep.moe_expert_linear_grad_input(rows, E, n, n, x, off, w, 0, None, None, y, mep.MOE_BF16, ws)
    torch.cuda.synchronize()
    say("[gpu] the gradient to the input is done")
    check(w)


def test_longest_sum_of_an_expert():
    """The gradient to the weights where one of 512 experts has nearly all rows: a sum that is
    not split.  Rows of zeros but for some at both ends and between."""
    rows, E, n = (1 << 31) - 1, 512, 8
    b = [0] + [rows - 10] * (E - 1) + [rows - 5]
    say(f"[gpu] gradient to the weights, {b[1]} rows of one expert, n = k = {n}")
    g = torch.Generator(device=DEV)
    g.manual_seed(10)
    x = torch.zeros((rows, n), dtype=BF16, device=DEV)
    spots = [slice(0, 40), slice((1 << 30) - 20, (1 << 30) + 20), slice(rows - 50, rows)]
    for part in spots:
        x[part] = torch.randint(-3, 4, (x[part].shape[0], n), generator=g, device=DEV).to(BF16)
    off = torch.tensor(b, dtype=I32, device=DEV)
    ws = torch.empty(max(1, mep.moe_expert_linear_workspace(rows, E, n, n)), dtype=torch.uint8, device=DEV)
    dw, db = torch.full((E, n, n), 99.0, device=DEV), torch.full((E, n), 99.0, device=DEV)
    mep.moe_expert_linear_grad_weight(rows, E, n, n, x, x, off, dw, mep.MOE_FP32, db, ws)
    torch.cuda.synchronize()
    say("[gpu] done")
    first = torch.cat([x[spots[0]], x[spots[1]], x[rows - 50:rows - 10]]).double()
    last = x[rows - 10:rows - 5].double()
    assert torch.equal(dw[0].double(), first.T @ first) and torch.equal(db[0].double(), first.sum(0))
    assert torch.equal(dw[-1].double(), last.T @ last) and torch.equal(db[-1].double(), last.sum(0))
    assert not dw[1:-1].any() and not db[1:-1].any()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts", [[0] * 15 + [112], [110] + [0] * 14 + [1], [1] * 8 + [97] + [1] * 7])
def test_few_rows_mostly_of_one_expert(counts, kind):
    """The gradient to the weights of a few rows per expert, by their mean."""
    E, n, k, rows = len(counts), 2048, 1032, 112
    say(f"[gpu] gradient to the weights, rows {counts}, {kind}")
    mep._lib.moe_ops_linear_form.restype = ctypes.c_char_p
    form = mep._lib.moe_ops_linear_form(3 if kind == torch.float32 else 2, 0, rows, E, n, k, ctypes.byref(ctypes.c_int32(0)))
    assert form == b"few rows"
    b = [0]
    for c in counts:
        b.append(b[-1] + c)
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    x, dz = (torch.randint(-3, 4, (rows, c), generator=g, device=DEV).to(BF16) for c in (k, n))
    x[b[E]:] = dz[b[E]:] = float("nan")
    dw, db = torch.full((E, n, k), 99.0, device=DEV, dtype=kind), torch.full((E, n), 99.0, device=DEV)
    ws = torch.empty(max(1, mep.moe_expert_linear_workspace(rows, E, n, k)), dtype=torch.uint8, device=DEV)
    mep.moe_expert_linear_grad_weight(rows, E, n, k, dz, x, torch.tensor(b, dtype=I32, device=DEV), dw,
                                      mep.MOE_FP32 if kind == torch.float32 else mep.MOE_BF16, db, ws)
    for e in range(E):
        d, u = dz[b[e]:b[e + 1]].double(), x[b[e]:b[e + 1]].double()
        assert torch.equal(dw[e], (d.T @ u).to(kind)) and torch.equal(db[e].double(), d.sum(0)), e
