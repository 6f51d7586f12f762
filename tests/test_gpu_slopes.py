"""The activations' slopes over their range, of moe_activation_grad and in the epilogue of
moe_expert_linear_grad_input, relative to themselves: every bf16 pre-activation from -12 to 12.

A slope is a sum of two parts, gelu' = Phi + z phi and silu' = p + z p (1 - p), that differ in
sign below zero and cancel only near -0.75 and -1.28.  Each part is formed of numbers that are
good to a few 2^-24 of themselves: Phi and phi, or p and 1 - p (for z > 0 off by 2^-24 of p <= 1,
which z passes on at most 12 times).  So fp32 results are held to 64 * 2^-24 of the parts'
magnitudes, whose sum is 1.6 times the slope or less from -2 down, and bf16 ones to half a step
of the type more.  What is below the normal numbers may be zero."""
import ctypes
import math

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
K = 512


def pre_activations():
    bits = torch.arange(1 << 16, device=DEV, dtype=torch.int32).to(torch.int16)
    z = bits.view(BF16)
    z = z[torch.isfinite(z.float()) & (z.float().abs() <= 12)]
    return torch.cat([z, torch.zeros(-z.numel() % K, device=DEV, dtype=BF16)]).view(-1, K)


def slope(act, z):
    """(slope, magnitudes of its parts) in 64 bits."""
    z = z.double()
    if act == "relu":
        return (z > 0).double(), (z > 0).double()
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
        rest = z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return cdf + rest, cdf + rest.abs()
    p = torch.sigmoid(z)
    q = torch.sigmoid(-z)
    return p + z * p * q, p + (z * p * q).abs()


def through(act, z, d):
    """(gradient to z of sum(d * act(z)), magnitudes of its parts)."""
    if act != "swiglu":
        s, parts = slope(act, z)
        return d * s, d.abs() * parts
    gate, up = z[:, :K].double(), z[:, K:].double()
    s, parts = slope("silu", gate)
    value = gate * torch.sigmoid(gate)
    return torch.cat([d * up * s, d * value], 1), torch.cat([(d * up).abs() * parts, (d * value).abs()], 1)


def check(got, want, parts):
    lim = HALF[got.dtype] * want.abs() + 64 * 2.0 ** -24 * parts + 2.0 ** -117
    far = (got.double() - want).abs() - lim
    i = int(far.argmax())
    assert bool((far <= 0).all()), f"{got.reshape(-1)[i].item()} for {want.reshape(-1)[i].item()}"


def case(act):
    z = pre_activations()
    if act == "swiglu":
        g = torch.Generator(device=DEV)
        g.manual_seed(3)
        z = torch.cat([z, torch.randn(z.shape, generator=g, device=DEV).to(BF16)], 1)
    return z.contiguous()


@pytest.mark.parametrize("d", [1.0, -0.375, 3.0])
@pytest.mark.parametrize("act", ACTS[1:])
def test_activation_grad(act, d):
    say(f"[gpu] slopes, {act}, gradient {d}")
    z = case(act)
    dy = torch.full((z.shape[0], K), d, device=DEV, dtype=BF16)
    dz = torch.empty_like(z)
    mep.moe_activation_grad(z.shape[0], 1, z.shape[1], ACTS.index(act), None, z, dy, dz)
    check(dz, *through(act, z, dy.double()))


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("n,split", [(8, False), (4096, True)])
@pytest.mark.parametrize("act", ACTS[1:])
def test_grad_input(act, n, split, kind):
    """A sum of one product, d * 1."""
    z = case(act)
    rows = z.shape[0]
    say(f"[gpu] slopes of the gradient to the input, {act}, {rows} rows, n={n}, {kind}")
    splits = ctypes.c_int(0)
    mep._lib.moe_ops_linear_form(1, 0, rows, 1, n, K, ctypes.byref(splits))
    assert (splits.value > 1) == split
    d = torch.tensor([1.0, -0.375, 3.0], device=DEV)[torch.arange(rows, device=DEV) % 3]
    dz = torch.zeros((rows, n), device=DEV, dtype=BF16)
    dz[:, n - 3] = d.to(BF16)
    w = torch.zeros((1, n, K), device=DEV, dtype=BF16)
    w[:, n - 3] = 1
    space = torch.empty(mep.moe_expert_linear_workspace(rows, 1, n, K), dtype=torch.uint8, device=DEV)
    dx = torch.empty(z.shape, device=DEV, dtype=kind)
    mep.moe_expert_linear_grad_input(rows, 1, n, K, dz, None, w, ACTS.index(act), z, None, dx, KIND[kind], space)
    check(dx, *through(act, z, d.double()[:, None]))
