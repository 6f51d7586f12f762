"""What the entry points of the expert layer on one card refuse, which needs no
GPU: every check comes before any HIP call.  Sizes are paired with made-up
aligned addresses that no call may reach."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import combine_moe_dispatch_amd as mep  # noqa: E402

A = 4096        # an aligned address
B, F, Q = mep.MOE_BF16, mep.MOE_FP32, mep.MOE_FP8_E4M3


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    monkeypatch.setattr(mep, "_op_device", lambda: 0)


def refused(fn, *args):
    with pytest.raises(mep.MoeError) as ei:
        fn(*args, stream=0)
    assert ei.value.status == mep.MOE_ERR_INVALID


def cases(fn, good, bad):
    return [pytest.param(fn, {**good, **b}, id=f"{fn}-{i}") for i, b in enumerate(bad)]


PLAN = dict(tokens=2, num_experts=8, top_k=2, idx=A, offsets=A, slot=A, source=A, ws=None, nbytes=0)
SORT = dict(tokens=2, top_k=2, rows=4, hidden=256, dtype=B, x=A, xs=None, slot=A, sorted=A, ss=None)
SORTQ = {**SORT, "dtype": Q, "xs": A, "ss": A}
UNSORT = dict(tokens=2, top_k=2, rows=4, hidden=256, dtype=B, y=A, slot=A, w=A, out=A)
UGRAD = dict(tokens=2, top_k=2, rows=4, hidden=256, dtype=B, dout=A, y=A, slot=A, w=A, dy=A, dw=A)
RGRAD = dict(tokens=2, num_experts=8, top_k=2, logits=A, ldt=F, renorm=False, idx=A, dw=A, dz=A, ddt=F)
LINEAR = dict(rows=4, E=2, n=256, k=256, x=A, off=A, w=A, bias=A, act=0, res=A, z=A, y=A, ydt=B, ws=A, nbytes=1 << 30)
AGRAD = dict(rows=4, E=2, n=256, act=1, off=A, z=A, dy=A, dz=A)
GIN = dict(rows=4, E=2, n=256, k=256, dz=A, off=A, w=A, act=0, z=None, res=A, dx=A, ddt=B, ws=A, nbytes=1 << 30)
GW = dict(rows=4, E=2, n=256, k=256, dz=A, x=A, off=A, dw=A, ddt=B, db=A, ws=A, nbytes=1 << 30)
SIZES = [dict(rows=-1), dict(E=0), dict(E=1025), dict(n=0), dict(n=12), dict(n=65544), dict(k=0), dict(k=12),
         dict(k=65544)]
ROWS = [dict(tokens=-1), dict(top_k=0), dict(top_k=65), dict(rows=-1), dict(hidden=0), dict(hidden=12),
        dict(hidden=65544), dict(dtype=3), dict(slot=None), dict(slot=A + 4)]


@pytest.mark.parametrize("fn,args", (
    cases("moe_sort_plan", PLAN, [
        dict(tokens=-1), dict(num_experts=0), dict(num_experts=1025), dict(top_k=0), dict(top_k=65), dict(idx=None),
        dict(offsets=None), dict(slot=None), dict(idx=A + 4), dict(offsets=A + 8), dict(slot=A + 2),
        dict(source=A + 4), dict(ws=A + 4), dict(tokens=1 << 30), dict(tokens=100000, ws=None),
        dict(tokens=100000, ws=A, nbytes=mep.moe_sort_workspace(100000, 8, 2) - 1)])
    + cases("moe_sort_rows", SORT, ROWS + [
        dict(x=None), dict(sorted=None), dict(x=A + 8), dict(sorted=A + 2), dict(xs=A), dict(ss=A)])
    + cases("moe_sort_rows", SORTQ, [
        dict(hidden=264), dict(xs=None), dict(ss=None), dict(xs=A + 4), dict(ss=A + 4), dict(x=A + 8)])
    + cases("moe_unsort_rows", UNSORT, ROWS + [
        dict(dtype=Q), dict(y=None), dict(out=None), dict(y=A + 2), dict(w=A + 4), dict(out=A + 8)])
    + cases("moe_unsort_rows_grad", UGRAD, ROWS + [
        dict(dtype=Q), dict(dout=None), dict(y=None), dict(dy=None, dw=None), dict(dout=A + 2), dict(y=A + 8),
        dict(w=A + 4), dict(dy=A + 8), dict(dw=A + 4)])
    + cases("moe_topk_route_grad", RGRAD, [
        dict(tokens=-1), dict(num_experts=0), dict(num_experts=1025), dict(top_k=0), dict(top_k=9), dict(ldt=Q),
        dict(ddt=Q), dict(ldt=3), dict(ddt=-1), dict(logits=None), dict(idx=None), dict(dw=None), dict(dz=None),
        dict(logits=A + 4), dict(idx=A + 4), dict(dw=A + 8), dict(dz=A + 4)])
    + cases("moe_expert_linear", LINEAR, SIZES + [
        dict(act=-1), dict(act=5), dict(act=4, n=264), dict(ydt=Q), dict(ydt=3), dict(x=None), dict(off=None),
        dict(w=None), dict(y=None), dict(x=A + 8), dict(off=A + 4), dict(w=A + 2), dict(bias=A + 2), dict(res=A + 8),
        dict(z=A + 8), dict(y=A + 4), dict(ws=A + 8), dict(ydt=F, res=A, y=A), dict(k=8192, nbytes=0)])
    + cases("moe_activation_grad", AGRAD, [
        dict(rows=-1), dict(E=0), dict(E=1025), dict(n=4), dict(n=65544), dict(act=0), dict(act=5), dict(act=4, n=264),
        dict(act=4), dict(off=None), dict(z=None), dict(dy=None), dict(dz=None), dict(off=A + 4), dict(z=A + 8),
        dict(dy=A + 2), dict(dz=A + 4)])
    + cases("moe_expert_linear_grad_input", GIN, SIZES + [
        dict(act=-1), dict(act=5), dict(act=1), dict(z=A), dict(ddt=Q), dict(dz=None), dict(off=None), dict(w=None),
        dict(dx=None), dict(dz=A + 8), dict(w=A + 2), dict(res=A + 8), dict(dx=A + 4), dict(act=1, z=A + 4),
        dict(ddt=F, res=A, dx=A), dict(n=8192, nbytes=0)])
    + cases("moe_expert_linear_grad_weight", GW, SIZES + [
        dict(ddt=Q), dict(dz=None), dict(x=None), dict(off=None), dict(dw=None), dict(dz=A + 8), dict(x=A + 2),
        dict(off=A + 4), dict(dw=A + 8), dict(db=A + 4), dict(ws=A + 4),
        dict(rows=4096, nbytes=0)])))
def test_refuses(fn, args):
    refused(getattr(mep, fn), *args.values())


def test_nothing_to_do_needs_nothing():
    mep.moe_sort_rows(0, 2, 4, 256, B, None, None, None, None, None, stream=0)
    mep.moe_unsort_rows(0, 2, 4, 256, B, None, None, None, None, stream=0)
    mep.moe_unsort_rows_grad(0, 2, 4, 256, B, None, None, None, None, None, None, stream=0)
    mep.moe_topk_route_grad(0, 8, 2, None, F, False, None, None, None, F, stream=0)
    mep.moe_expert_linear(0, 2, 256, 256, None, None, None, None, 0, None, None, None, B, stream=0)
    mep.moe_activation_grad(0, 2, 256, 1, None, None, None, None, stream=0)
    mep.moe_expert_linear_grad_input(0, 2, 256, 256, None, None, None, 0, None, None, None, B, stream=0)


def test_workspaces():
    assert mep.moe_sort_workspace(1, 256, 8) == 0            # one workgroup has all pairs
    assert mep.moe_sort_workspace(131072, 256, 8) > 0
    for bad in [(-1, 8, 2), (4, 0, 2), (4, 1025, 2), (4, 8, 0), (4, 8, 65), (1 << 30, 8, 2)]:
        assert mep.moe_sort_workspace(*bad) == 0
    assert mep.moe_expert_linear_workspace(128, 1, 256, 7168) >= 2 * 128 * 256 * 4      # a split sum
    for bad in [(-1, 8, 256, 256), (4, 0, 256, 256), (4, 1025, 256, 256), (4, 8, 12, 256), (4, 8, 256, 12),
                (4, 8, 65544, 256), (4, 8, 256, 65544)]:
        assert mep.moe_expert_linear_workspace(*bad) == 0


def test_tensors_are_checked():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(mep.MoeError, match="x not a device tensor"):
        mep.moe_expert_linear(4, 1, 256, 256, x, None, A, None, 0, None, None, A, B, stream=0)
    with pytest.raises(mep.MoeError, match="dout not a device tensor"):
        mep.moe_unsort_rows_grad(2, 2, 4, 256, B, x, A, A, None, A, None, stream=0)


def test_activations_are_the_headers():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "moe_ep.h")).read()
    found = dict(re.findall(r"(MOE_ACT_\w+) = (\d)", text))
    assert found == {n: str(getattr(mep, n)) for n in dir(mep) if n.startswith("MOE_ACT_")} and len(found) == 5
    assert isinstance(mep._lib, ctypes.CDLL)


def _form(kind, gated, rows, E, n, k):
    splits = ctypes.c_int32(0)
    fn = mep._lib.moe_ops_linear_form
    fn.argtypes, fn.restype = [ctypes.c_int32] * 6 + [ctypes.POINTER(ctypes.c_int32)], ctypes.c_char_p
    return fn(kind, gated, rows, E, n, k, ctypes.byref(splits)).decode(), splits.value


@pytest.mark.parametrize("want,args", [
    (("256 x 256", 1), (0, 1, 32768, 16, 4096, 7168)), (("256 x 256", 1), (1, 0, 32768, 16, 7168, 2048)),
    (("256 x 256", 1), (2, 0, 32768, 16, 7168, 2048)), (("64 x 128", 1), (0, 0, 1000, 1, 4096, 4096)),
    (("32 x 128", 1), (0, 0, 37, 8, 1000, 392)), (("few rows", 1), (2, 0, 64, 64, 4096, 2048)),
    (("", 0), (4, 0, 4, 1, 256, 256)), (("", 0), (1, 1, 4, 1, 256, 256)), (("", 0), (0, 1, 4, 1, 264, 256)),
    (("", 0), (0, 0, 4, 1, 260, 256)), (("", 0), (0, 0, 4, 0, 256, 256))])
def test_linear_forms(want, args):
    assert _form(*args) == want


def test_workspace_serves_every_call():
    """The workspace of the sizes is at least what each call's splits take."""
    for rows, E, n, k in [(128, 1, 256, 7168), (64, 1, 4096, 4096), (2000, 8, 4096, 2048), (1, 1, 16, 65536),
                          (5000, 1, 256, 256), (3641, 1, 16, 8), (7, 3, 48, 4096)]:
        size = mep.moe_expert_linear_workspace(rows, E, n, k)
        for kind, gated, outputs in [(0, 0, rows * n), (0, 1, rows * n), (1, 0, rows * k), (2, 0, E * n * (k + 1)),
                                     (3, 0, E * n * (k + 1))]:
            _, splits = _form(kind, gated, rows, E, n, k)
            assert splits == 1 or size >= splits * outputs * 4, (rows, E, n, k, kind)
