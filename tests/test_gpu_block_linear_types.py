"""MokBlockLinear with every pair of types of weights, rows and results, forward and backward, and for inference alone:
results are the products of its own codes, within the bounds of their sums (fp32 results: terms and two scales a block, 2^-23
of the sum of the terms' sizes; bf16: half a step, 2^-8, and 128 times 2^-19 of each block's largest possible term), and the
codes are those of the values that were given."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import block as ob

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_router_top_schedule_amd.block import MokBlockLinear

R, N, K, OFF = 300, 136, 200, [4, 120, 120, 295]


def host(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def close(got, x, xs, w, ws, terms):
    want, size, most = ob.gemm(host(x), host(xs), host(w), host(ws), OFF, np.full(tuple(got.shape), 9.0))
    blocks = ob.up(terms) // 128
    if got.dtype == torch.bfloat16:
        bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * most + (blocks + 128) * 2.0 ** -23 * size
    else:
        bound = (ob.up(terms) + 2 * blocks) * 2.0 ** -23 * size
    y = host(got)
    assert (y[:OFF[0]] == 9).all() and (y[OFF[-1]:] == 9).all()
    assert (np.abs(y - want) <= bound)[OFF[0]:OFF[-1]].all()


@pytest.mark.parametrize("train", [True, False])
@pytest.mark.parametrize("wt", ["float32", "bfloat16"])
@pytest.mark.parametrize("xt", ["float32", "bfloat16"])
@pytest.mark.parametrize("yt", ["float32", "bfloat16"])
def test_types(wt, xt, yt, train):
    wt, xt, yt = (getattr(torch, t) for t in (wt, xt, yt))
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    w, x, dy = (0.05 * rand(3, N, K)).to(wt), rand(R, K).to(xt), rand(R, N).to(xt)
    o = torch.tensor(OFF, dtype=torch.int32, device="cuda")
    lin = MokBlockLinear(w, R, train=train)
    out = torch.full((R, N), 9.0, dtype=yt, device="cuda")
    lin.forward(x, out, offsets=o)
    codes, scales = ob.quantize_weights(host(w))
    assert np.array_equal(host(lin.wq), codes) and np.array_equal(host(lin.ws), scales)
    codes, scales = ob.quantize_rows(host(x))
    assert np.array_equal(host(lin.xq), codes) and np.array_equal(host(lin.xs), scales)
    close(out, lin.xq, lin.xs, lin.wq, lin.ws, K)
    if not train:
        return
    dx, dw = torch.full((R, K), 9.0, dtype=yt, device="cuda"), torch.zeros(3, N, K, device="cuda")
    lin.backward(dy, dx, dw, offsets=o)
    codes, scales = ob.quantize_rows(host(dy))
    assert np.array_equal(host(lin.yq), codes) and np.array_equal(host(lin.ys), scales)
    close(dx, lin.yq, lin.ys, lin.wt, lin.wts, N)
    want, size = ob.wgrad(host(lin.yt), host(lin.yts), host(lin.xt), host(lin.xts), OFF, np.zeros((3, N, K)))
    assert (np.abs(host(dw) - want) <= (256 + 4) * 2.0 ** -23 * size).all()
    # one of the two alone is the same
    dx2, dw2 = torch.full_like(dx, 9.0), torch.zeros_like(dw)
    lin.backward(dy, dx2, None, offsets=o)
    lin.backward(dy, None, dw2, offsets=o)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
