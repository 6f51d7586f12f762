"""The few-token layer in each of its forms, asked of the library case by case:
coded in the product kernels or once, the down product whole or in shares; many
columns of one expert, experts named twice, padding.  Against the definition in
64 bits, with test_gpu_ops' bound."""
import ctypes

import numpy as np
import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_moe_dispatch_amd as mep  # noqa: E402
from tests.test_gpu_ops import check_few, few_inputs, few_ref, run_few  # noqa: E402

_form = mep._lib.moe_ops_few_token_form
_form.argtypes, _form.restype = [ctypes.c_int32] * 5, ctypes.c_char_p

CASES = [
    # tokens up to four, then on both sides of the columns' and the weights' limits
    ("direct", 1, 9, 3, 256, 384), ("direct", 4, 2, 2, 384, 256), ("direct", 16, 40, 2, 384, 256),
    ("direct", 10, 8, 2, 256, 128), ("coded", 11, 8, 2, 256, 128), ("coded", 17, 300, 2, 128, 128),
    ("direct split", 4, 8, 2, 128, 65536), ("direct split", 9, 32, 4, 256, 4096), ("coded split", 6, 2, 1, 128, 65536),
    ("coded split", 33, 8, 3, 256, 1024), ("coded split", 64, 9, 2, 256, 256)]


@pytest.mark.parametrize("want,T,E,K,H,F", CASES)
def test_few_forms(want, T, E, K, H, F):
    say(f"[gpu] few form {want} T={T} E={E} K={K} H={H} F={F}")
    assert _form(T, E, K, H, F).decode() == want
    g = np.random.default_rng([23, T, E, K, H, F])
    x, idx, w, *wts = few_inputs(g, T, E, K, H, F)
    check_few(run_few(x, idx, w, *wts), *few_ref(x, idx, w, *wts))
    # most tokens name one expert, some of them twice; the last tokens are padding
    idx[:, 0] = E // 2
    if K > 1:
        idx[::3, -1] = E // 2
    if T > 2:
        idx[-2:] = -1
        x[-2:] = float("nan")
    out = run_few(x, idx, w, *wts)
    live = slice(0, T - 2 if T > 2 else T)
    ref, noise = few_ref(x[live], idx[live], w[live], *wts)
    check_few(out[live], ref, noise)
    assert T <= 2 or bool((out[-2:] == 0).all())


@pytest.mark.parametrize("want,T,E,K,H,F", [("direct", 9, 8, 2, 384, 256), ("direct split", 9, 32, 4, 256, 4096),
                                            ("coded", 11, 8, 2, 256, 128), ("coded split", 33, 8, 3, 256, 1024)])
def test_few_forms_at_once(want, T, E, K, H, F):
    """Each form captured twice, replayed on two streams at once between eager calls."""
    say(f"[gpu] few at once {want}")
    assert _form(T, E, K, H, F).decode() == want
    x, *rest = few_inputs(np.random.default_rng([29, T]), T, E, K, H, F)
    eager = run_few(x, *rest)
    idx, w, *wts = (torch.from_numpy(a).to("cuda") for a in rest)
    nbytes = mep.moe_few_token_workspace(T, K, H, F)
    outs = [torch.empty_like(x) for _ in range(2)]
    spaces = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(2)]
    graphs = []
    torch.cuda.synchronize()
    for out, space in zip(outs, spaces):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mep.moe_few_token_layer(T, E, K, H, F, x, idx, w, *wts, out, space)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for t in outs + spaces:
            t.view(torch.uint8).fill_(0xFF)
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, eager) for out in outs)
        assert torch.equal(run_few(x, *rest), eager)
