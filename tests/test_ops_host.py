"""What the operators' entry points refuse, which needs no GPU: every check
comes before any HIP call.  Sizes are paired with made-up aligned addresses
that no call may reach."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import combine_moe_dispatch_amd as mep  # noqa: E402

A = 4096        # an aligned address


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    monkeypatch.setattr(mep, "_op_device", lambda: 0)


def refused(fn, *args):
    with pytest.raises(mep.MoeError) as ei:
        fn(*args, stream=0)
    assert ei.value.status == mep.MOE_ERR_INVALID


NORM = dict(rows=2, hidden=256, x=A, residual=A, weight=A, eps=1e-6, residual_out=A, y=A, y_q=A, y_scale=A)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(hidden=0), dict(hidden=4), dict(hidden=260), dict(hidden=65544),
    dict(hidden=264), dict(x=None), dict(weight=None), dict(x=A + 2), dict(residual=A + 8),
    dict(weight=A + 4), dict(residual_out=A + 1), dict(y=A + 2), dict(y_q=A + 8), dict(y_scale=A + 4),
    dict(y_q=None), dict(y_scale=None), dict(eps=-1.0), dict(eps=float("nan")),
    dict(residual_out=None, y=None, y_q=None, y_scale=None)])
def test_norm_refuses(bad):
    refused(mep.moe_add_rmsnorm, *{**NORM, **bad}.values())


ROUTE = dict(tokens=2, num_experts=8, top_k=2, logits=A, dtype=mep.MOE_FP32, renorm=False, idx=A, w=A)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(num_experts=0), dict(num_experts=1025), dict(top_k=0), dict(top_k=9),
    dict(num_experts=100, top_k=65), dict(dtype=mep.MOE_FP8_E4M3), dict(dtype=3), dict(logits=None),
    dict(idx=None), dict(w=None), dict(logits=A + 4), dict(idx=A + 4), dict(w=A + 8)])
def test_route_refuses(bad):
    refused(mep.moe_topk_route, *{**ROUTE, **bad}.values())


MATMUL = dict(rows=4, experts=2, n=256, k=256, x=A, xs=A, offsets=A, w=A, ws=A, y=A)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(experts=0), dict(experts=1025), dict(n=0), dict(n=4), dict(n=12),
    dict(n=65544), dict(k=0), dict(k=64), dict(k=200), dict(k=65664), dict(x=None), dict(xs=None),
    dict(offsets=None), dict(w=None), dict(ws=None), dict(y=None), dict(x=A + 8), dict(xs=A + 4),
    dict(offsets=A + 4), dict(w=A + 1), dict(ws=A + 4), dict(y=A + 2)])
def test_matmul_refuses(bad):
    refused(mep.moe_expert_matmul, *{**MATMUL, **bad}.values())


GATE_UP = dict(rows=4, experts=2, f=256, k=256, x=A, xs=A, offsets=A, w=A, ws=A, h=A, hs=A)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(experts=0), dict(f=0), dict(f=64), dict(f=136), dict(f=65664), dict(k=130),
    dict(x=None), dict(h=None), dict(hs=None), dict(h=A + 8), dict(hs=A + 4), dict(w=A + 2)])
def test_gate_up_refuses(bad):
    refused(mep.moe_expert_gate_up, *{**GATE_UP, **bad}.values())


FEW = dict(tokens=4, experts=8, top_k=2, hidden=256, f=256, x=A, idx=A, w=A, w13=A, s13=A, w2=A, s2=A,
           out=A, ws=A, nbytes=1 << 20)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(tokens=65), dict(experts=0), dict(experts=1025), dict(top_k=0),
    dict(top_k=65), dict(hidden=64), dict(hidden=200), dict(f=0), dict(f=130), dict(x=None),
    dict(idx=None), dict(w=None), dict(w13=None), dict(s13=None), dict(w2=None), dict(s2=None),
    dict(out=None), dict(ws=None), dict(ws=A + 8), dict(out=A + 8), dict(nbytes=0),
    dict(nbytes=mep.moe_few_token_workspace(4, 2, 256, 256) - 1)])
def test_few_tokens_refuses(bad):
    refused(mep.moe_few_token_layer, *{**FEW, **bad}.values())


def test_workspace_sizes():
    assert mep.moe_few_token_workspace(1, 8, 7168, 2048) > 0
    for bad in [(0, 8, 256, 256), (65, 8, 256, 256), (1, 0, 256, 256), (1, 65, 256, 256),
                (1, 8, 100, 256), (1, 8, 256, 100), (-1, 8, 256, 256)]:
        assert mep.moe_few_token_workspace(*bad) == 0
    small = mep.moe_few_token_workspace(1, 1, 128, 128)
    assert small <= mep.moe_few_token_workspace(64, 64, 65536, 65536)


def test_nothing_to_do_needs_nothing():
    mep.moe_add_rmsnorm(0, 256, None, None, None, 1e-6, None, A, None, None, stream=0)
    mep.moe_topk_route(0, 8, 2, None, mep.MOE_BF16, True, None, None, stream=0)
    mep.moe_expert_matmul(0, 2, 256, 256, None, None, None, None, None, None, stream=0)
    mep.moe_expert_gate_up(0, 2, 256, 256, None, None, None, None, None, None, None, stream=0)
    mep.moe_few_token_layer(0, 8, 2, 256, 256, None, None, None, None, None, None, None, None, None,
                            stream=0)


def test_tensors_are_checked():
    """A host tensor is refused by name before its address is used."""
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    with pytest.raises(mep.MoeError, match="x not a device tensor"):
        mep.moe_add_rmsnorm(2, 256, x, None, A, 1e-6, None, A, None, None, stream=0)


def test_addresses_of_any_int_type():
    """An int subclass is an address, as the four calls take it."""
    class Address(int):
        pass

    args = {**NORM, "x": Address(A), "weight": Address(A + 2)}
    refused(mep.moe_add_rmsnorm, *args.values())                 # by the library: misaligned
    assert mep._op_arg(Address(A), "call", "x", 1 << 40, 2, (), 0) == A


def _form(name, *sizes):
    fn = getattr(mep._lib, name)
    fn.argtypes, fn.restype = [ctypes.c_int32] * len(sizes), ctypes.c_char_p
    return fn(*sizes).decode()


@pytest.mark.parametrize("want,T,E,K,H,F", [
    # up to four tokens; up to 2.5 columns per expert with 256 MB of weights; up to a third with more
    ("direct", 4, 1, 1, 4096, 2048), ("direct", 10, 8, 2, 4096, 2048), ("coded", 11, 8, 2, 4096, 2048),
    ("coded", 16, 64, 4, 4096, 2048), ("direct", 5, 64, 4, 4096, 2048), ("coded", 6, 64, 4, 4096, 2048),
    ("direct", 10, 256, 8, 7168, 2048), ("coded", 11, 256, 8, 7168, 2048), ("coded", 17, 1024, 1, 4096, 128),
    ("direct split", 10, 187, 6, 384, 2432), ("coded split", 61, 177, 5, 384, 1024)])
def test_few_token_forms(want, T, E, K, H, F):
    assert _form("moe_ops_few_token_form", T, E, K, H, F) == want


@pytest.mark.parametrize("want,gate_up,rows,E,n", [
    ("narrow", 0, 64, 1, 5760), ("32 deep", 0, 64, 1, 5824), ("32 deep", 1, 1, 1, 256), ("32", 0, 1024, 256, 4096),
    ("32", 1, 1024, 256, 4096), ("64", 0, 2000, 64, 7168), ("128", 0, 6144, 64, 7168), ("256", 0, 6208, 64, 7168),
    ("128", 1, 32768, 256, 4096), ("64", 1, 2000, 2, 1536)])
def test_product_forms(want, gate_up, rows, E, n):
    assert _form("moe_ops_product_form", gate_up, rows, E, n) == want


def test_forms_of_no_call():
    for sizes in ((0, 0, 1, 256), (0, 4, 0, 256), (1, 4, 1025, 256), (0, 4, 1, 0), (0, -1, 1, 256)):
        assert _form("moe_ops_product_form", *sizes) == ""
    for sizes in ((0, 8, 2, 256, 256), (65, 8, 2, 256, 256), (4, 0, 2, 256, 256), (4, 8, 0, 256, 256),
                  (4, 8, 2, 0, 256), (4, 8, 2, 256, 64)):
        assert _form("moe_ops_few_token_form", *sizes) == ""
