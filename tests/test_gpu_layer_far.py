"""The expert layer's operators on tensors beyond 2^32 bytes: rows, pairs, weights
and outputs at the far end are those of a call on that end alone, or exact whole
numbers."""
import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_moe_dispatch_amd as mep  # noqa: E402

DEV = "cuda"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
FAR = 1 << 32


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def whole(g, *shape, most=3):
    """Whole numbers -most .. most, made in parts."""
    t = torch.empty(shape, dtype=BF16, device=DEV)
    for part in t.view(-1).split(1 << 28):
        part.copy_(torch.randint(-most, most + 1, part.shape, generator=g, device=DEV, dtype=torch.int8))
    return t


def space(rows, E, n, k):
    return torch.empty(max(1, mep.moe_expert_linear_workspace(rows, E, n, k)), dtype=torch.uint8, device=DEV)


def test_plan_far_pairs():
    """1.2e9 pairs: 4.8 GB of ids, of slots, of sources."""
    T, E, K = 100_000_000, 40, 12
    say(f"[gpu] sort plan far T={T} E={E} K={K}")
    g = generator(1)
    idx = torch.empty((T, K), dtype=I32, device=DEV)
    for part in idx.view(-1).split(1 << 28):
        part.copy_(torch.randint(-1, E, part.shape, generator=g, device=DEV, dtype=torch.int8))
    assert idx.numel() * 4 > FAR
    slot, source, off = torch.empty_like(idx), torch.empty(T * K, dtype=I32, device=DEV), torch.empty(E + 1, dtype=I32, device=DEV)
    ws = torch.empty(max(1, mep.moe_sort_workspace(T, E, K)), dtype=torch.uint8, device=DEV)
    mep.moe_sort_plan(T, E, K, idx, off, slot, source, ws)
    count = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    for part in idx.view(-1).split(1 << 26):
        count += torch.bincount(part + 1, minlength=E + 1)
    assert torch.equal(off[1:].long(), count[1:].cumsum(0)) and int(off[0]) == 0
    used = int(off[-1])
    at = 0
    for part, rows in zip(idx.view(-1).split(1 << 26), slot.view(-1).split(1 << 26)):
        live = part >= 0
        assert bool((rows[~live] == -1).all())
        r = rows[live].long()
        pair = torch.arange(at, at + part.numel(), device=DEV)[live]
        e = part[live].long()
        assert torch.equal(source[r].long(), pair)                  # each row has its pair ...
        assert bool(((r >= off[e]) & (r < off[e + 1])).all())       # ... among its expert's
        at += part.numel()
    for a in range(0, used - 1, 1 << 26):                           # in the pairs' order
        s = source[a:min(used, a + (1 << 26) + 1)]
        down = torch.nonzero(s[1:] <= s[:-1]).view(-1) + a + 1
        assert bool(torch.isin(down, off.long()).all())


def test_rows_far():
    """Sorted rows of 9.8 GB, by more than 2^32 elements, and back."""
    T, K, H = 300_000, 2, 8192
    say(f"[gpu] sorted rows far T={T} K={K} H={H}")
    g = generator(2)
    x = whole(g, T, H)
    rows = T * K
    assert x.numel() * 2 > FAR and rows * H > FAR
    slot = torch.randperm(rows, generator=g, device=DEV).to(I32).view(T, K)
    out = torch.empty((rows, H), dtype=BF16, device=DEV)
    mep.moe_sort_rows(T, K, rows, H, mep.MOE_BF16, x, None, slot, out, None)
    for t in (0, T // 2, T - 512):
        part = slice(t, t + 512)
        assert torch.equal(out[slot[part].long()], x[part][:, None].expand(512, K, H))
    w = torch.randint(1, 4, (T, K), generator=g, device=DEV).float()
    back = torch.empty_like(x)
    mep.moe_unsort_rows(T, K, rows, H, mep.MOE_BF16, out, slot, w, back)
    for t in (0, T // 2, T - 512):
        part = slice(t, t + 512)
        assert torch.equal(back[part], (w[part].sum(1, keepdim=True) * x[part].float()).to(BF16))
    dw = torch.empty((T, K), device=DEV)
    dy = torch.empty_like(out)
    mep.moe_unsort_rows_grad(T, K, rows, H, mep.MOE_BF16, back, out, slot, w, dy, dw)
    for t in (0, T // 2, T - 512):
        part = slice(t, t + 512)
        b = back[part].float()
        assert torch.equal(dy[slot[part].long()], (w[part][..., None] * b[:, None]).to(BF16))
        assert torch.equal(dw[part], (b * x[part].float()).sum(1, keepdim=True).expand(512, K))


@pytest.mark.parametrize("T,E,K,bf", [(4_300_000, 255, 8, False), (17_000_000, 64, 6, False), (10_000_000, 256, 8, True),
                                      (70_000_000, 16, 2, False)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_far(T, E, K, bf, renorm):
    say(f"[gpu] route gradient far T={T} E={E} K={K} bf16={bf} renorm={renorm}")
    g = generator(3)
    z = torch.empty((T, E), dtype=BF16 if bf else F32, device=DEV)
    for part in z.view(-1).split(1 << 28):
        part.normal_(generator=g)
    assert z.numel() * z.element_size() > FAR
    kind = mep.MOE_BF16 if bf else mep.MOE_FP32
    idx = torch.randint(0, E, (T, K), generator=g, device=DEV, dtype=I32)
    dw = torch.randn((T, K), generator=g, device=DEV)
    dz = torch.empty_like(z)
    mep.moe_topk_route_grad(T, E, K, z, kind, renorm, idx, dw, dz, kind)
    n = 160
    for a in (0, T // 2 // 16 * 16, T - n):
        part = [t[a:a + n].clone() for t in (z, idx, dw)]
        want = torch.empty((n, E), dtype=z.dtype, device=DEV)
        mep.moe_topk_route_grad(n, E, K, part[0], kind, renorm, part[1], part[2], want, kind)
        assert torch.equal(dz[a:a + n], want)


def test_activation_grad_far():
    rows, n = 70_000, 65536
    say(f"[gpu] activation gradient far rows={rows} n={n}")
    g = generator(4)
    z, dy = whole(g, rows, n), whole(g, rows, n // 2)
    dz = torch.empty_like(z)
    assert z.numel() > FAR
    mep.moe_activation_grad(rows, 1, n, mep.MOE_ACT_SWIGLU, None, z, dy, dz)
    for a in (0, rows // 2, rows - 16):
        part = slice(a, a + 16)
        want = torch.empty((16, n), dtype=BF16, device=DEV)
        mep.moe_activation_grad(16, 1, n, mep.MOE_ACT_SWIGLU, None, z[part], dy[part], want)
        assert torch.equal(dz[part], want)


@pytest.mark.parametrize("rows,n,k", [(610_000, 64, 4096), (610_000, 4096, 64), (40_000, 65536, 64), (70_000, 64, 65536)])
def test_linear_far_rows(rows, n, k):
    """Rows of the operands or of the results beyond 2^32 bytes, in ragged experts."""
    say(f"[gpu] linear far rows={rows} n={n} k={k}")
    g = generator(5)
    E = 3
    b = [0, rows // 3 + 5, rows // 2 + 1, rows - 7]
    off = torch.tensor(b, dtype=I32, device=DEV)
    x, dz, w = whole(g, rows, k), whole(g, rows, n), whole(g, E, n, k)
    ws = space(rows, E, n, k)
    y = torch.full((rows, n), 9.0, device=DEV)
    mep.moe_expert_linear(rows, E, n, k, x, off, w, None, 0, None, None, y, mep.MOE_FP32, ws)
    ends = [(e, slice(a, a + 40)) for e in range(E) for a in (b[e], b[e + 1] - 40)]
    for e, part in ends:
        assert torch.equal(y[part].double(), x[part].double() @ w[e].double().T), e
    assert bool((y[rows - 7:] == 9).all())
    del y
    dx = torch.full((rows, k), 9.0, device=DEV)
    mep.moe_expert_linear_grad_input(rows, E, n, k, dz, off, w, 0, None, None, dx, mep.MOE_FP32, ws)
    for e, part in ends:
        assert torch.equal(dx[part].double(), dz[part].double() @ w[e].double()), e
    assert bool((dx[rows - 7:] == 9).all())
    del dx
    # sums of 300 000 products of at most 9 in magnitude: below 2^24 with ease
    dw, db = torch.empty((E, n, k), device=DEV), torch.empty((E, n), device=DEV)
    mep.moe_expert_linear_grad_weight(rows, E, n, k, dz, x, off, dw, mep.MOE_FP32, db, ws)
    for e in range(E):
        some = torch.linspace(0, n - 1, min(n, 64), device=DEV).long()
        want = torch.zeros((some.numel(), k), dtype=torch.float64, device=DEV)
        total = torch.zeros(n, dtype=torch.float64, device=DEV)
        for a in range(b[e], b[e + 1], 20_000):
            part = slice(a, min(b[e + 1], a + 20_000))
            want += dz[part][:, some].double().T @ x[part].double()
            total += dz[part].double().sum(0)
        assert torch.equal(dw[e][some].double(), want) and torch.equal(db[e].double(), total), e


@pytest.mark.parametrize("rows", [[2] + [0] * 38 + [50], [300] * 40])
def test_linear_far_weights(rows):
    """Weights of 10.7 GB, their gradient of 21.5 GB."""
    E, n, k = 40, 16384, 8192
    say(f"[gpu] linear far weights rows={sum(rows)}")
    g = generator(6)
    b = [0]
    for r in rows:
        b.append(b[-1] + r)
    R = b[-1]
    off = torch.tensor(b, dtype=I32, device=DEV)
    x, dz, w, ws = whole(g, R, k), whole(g, R, n), whole(g, E, n, k, most=1), space(R, E, n, k)
    y, dx = torch.empty((R, n), device=DEV), torch.empty((R, k), device=DEV)
    mep.moe_expert_linear(R, E, n, k, x, off, w, None, 0, None, None, y, mep.MOE_FP32, ws)
    mep.moe_expert_linear_grad_input(R, E, n, k, dz, off, w, 0, None, None, dx, mep.MOE_FP32, ws)
    for e in (0, E - 1):
        part = slice(b[e], b[e + 1])
        assert torch.equal(y[part].double(), x[part].double() @ w[e].double().T), e
        assert torch.equal(dx[part].double(), dz[part].double() @ w[e].double()), e
    dw = torch.full((E, n, k), 9.0, device=DEV)
    mep.moe_expert_linear_grad_weight(R, E, n, k, dz, x, off, dw, mep.MOE_FP32, None, ws)
    for e in (0, 1, 20, E - 2, E - 1):
        part = slice(b[e], b[e + 1])
        assert torch.equal(dw[e].double(), dz[part].double().T @ x[part].double()), e
