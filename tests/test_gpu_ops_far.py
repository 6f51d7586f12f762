"""The operators on tensors beyond 2^32 bytes: rows, weights and outputs at the
far end are those of a call on that end alone, or of the 64-bit reference."""
import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_moe_dispatch_amd as mep  # noqa: E402
from tests.test_gpu_ops_tiles import check_gate_up, check_matmul, codes  # noqa: E402

DEV = "cuda"


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("rows,hidden", [(40000, 65536), (180000, 16384), (17500000, 128)])
def test_norm_far_rows(rows, hidden):
    say(f"[gpu] norm far rows={rows} hidden={hidden}")
    g = generator(1)
    x = torch.empty((rows, hidden), dtype=torch.bfloat16, device=DEV)
    for part in x.view(-1).split(1 << 28):
        part.normal_(generator=g)
    assert x.numel() * 2 > 1 << 32
    w = torch.randn(hidden, generator=g, device=DEV).to(torch.bfloat16)
    y, ro = torch.empty_like(x), torch.empty_like(x)
    yq = torch.empty((rows, hidden), dtype=torch.uint8, device=DEV)
    ys = torch.empty((rows, hidden // 128), device=DEV)
    mep.moe_add_rmsnorm(rows, hidden, x, x, w, 1e-6, ro, y, yq, ys)
    for a in (0, rows // 2 - 8, rows - 16):
        n = 16
        part = [t[a:a + n].clone() for t in (ro, y, yq, ys)]
        want = [torch.empty_like(t) for t in part]
        mep.moe_add_rmsnorm(n, hidden, x[a:a + n], x[a:a + n], w, 1e-6, *want)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(part, want))


@pytest.mark.parametrize("tokens,E,K,bf", [(1100000, 1024, 10, False), (2200000, 512, 8, False), (4300000, 255, 8, False),
                                           (10000000, 256, 8, True), (70000000, 16, 2, False), (17500000, 63, 20, False)])
def test_route_far_tokens(tokens, E, K, bf):
    say(f"[gpu] route far tokens={tokens} E={E} K={K} bf16={bf}")
    g = generator(2)
    z = torch.empty((tokens, E), dtype=torch.bfloat16 if bf else torch.float32, device=DEV)
    for part in z.view(-1).split(1 << 28):
        part.normal_(generator=g)
    assert z.numel() * z.element_size() > 1 << 32
    idx = torch.empty((tokens, K), dtype=torch.int32, device=DEV)
    w = torch.empty((tokens, K), device=DEV)
    kind = mep.MOE_BF16 if bf else mep.MOE_FP32
    mep.moe_topk_route(tokens, E, K, z, kind, True, idx, w)
    for a in (0, tokens // 2 // 16 * 16, tokens - 160):
        n = 160
        zi = z[a:a + n].clone()
        wi, ww = torch.empty((n, K), dtype=torch.int32, device=DEV), torch.empty((n, K), device=DEV)
        mep.moe_topk_route(n, E, K, zi, kind, True, wi, ww)
        torch.cuda.synchronize()
        assert torch.equal(idx[a:a + n], wi) and torch.equal(w[a:a + n], ww)


def test_products_far_rows():
    say("[gpu] products far rows")
    check_matmul("256", 1, [610000], 256, 7168, some=24)
    check_gate_up("128", 1, [610000], 128, 7168, some=24)
    # results beyond 2^32 bytes
    check_matmul("256", 1, [40000], 65536, 128, some=24)
    check_gate_up("128", 1, [70000], 65536, 128, some=24)


def test_products_far_weights():
    say("[gpu] products far weights")
    check_matmul("32", 40, [2] + [0] * 38 + [50], 16384, 8192)
    check_gate_up("32", 40, [2] + [0] * 38 + [50], 8192, 8192)
    check_matmul("256", 40, [0] * 39 + [5000], 16384, 8192, some=24)


@pytest.mark.parametrize("T", [3, 20])
def test_few_far_weights(T):
    """The last experts of 300, w13 of 5 GB, against a layer that has only the
    named ones, in the same order."""
    say(f"[gpu] few far weights T={T}")
    E, K, H, F = 300, 4, 8192, 1024
    g = generator(3)
    w13, w2 = codes(g, E, 2 * F, H), codes(g, E, H, F)
    s13 = torch.rand((E, 2 * F // 128, H // 128), generator=g, device=DEV) * 2.0 ** -14
    s2 = torch.rand((E, H // 128, F // 128), generator=g, device=DEV) * 2.0 ** -14
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    named = torch.tensor([0, 1, 255, 256, 257, 298, 299], device=DEV)
    pick = torch.stack([torch.randperm(len(named), generator=g, device=DEV)[:K] for _ in range(T)])
    w = torch.rand((T, K), generator=g, device=DEV)
    outs = []
    for ids, sel in ((named[pick], slice(None)), (pick, named)):
        wts = [t[sel].contiguous() for t in (w13.view(torch.uint8), s13, w2.view(torch.uint8), s2)]
        ws = torch.empty(mep.moe_few_token_workspace(T, K, H, F), dtype=torch.uint8, device=DEV)
        out = torch.empty_like(x)
        mep.moe_few_token_layer(T, wts[0].shape[0], K, H, F, x, ids.to(torch.int32).contiguous(), w, *wts, out, ws)
        outs.append(out)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(outs[0].float()).all()) and torch.equal(*outs)
