"""Weight gradients of offsets that go past the rows: clamped to the rows that were quantised, in the gradient as in the
quantiser, whatever the column codes' buffers held before. Results against oracle.block, in the bounds of its products:
(rows of the longest group, and one) 2^-23 of the sum of the terms' sizes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import block as ob

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok
from combine_router_top_schedule_amd.block import MokBlockLinear

F = np.float32
NAN = 0x7F   # E4M3's code of NaN

# Groups that would take another 128 columns if the offsets were not clamped to the rows, and ordinary ones.
CASES = [(40, [0, 0, 0, 900]), (2, [0, 0, 500]), (2, [0, 50, 90, 129]), (2, [1, 1, 128, 129, 1000]), (130, [-3, 100, 300, 255]),
         (129, [0, 1, 2 ** 31 - 1]), (200, [0, 60, 60, 190])]


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a, F)).cuda()


def close(dw, yt, yts, xt, xts, off, rows, before=None):
    clean = ob.clean(off, rows)
    host = [t.cpu().numpy().copy() for t in (yt, yts, xt, xts)]
    end = ob.columns(clean)[-1]   # what lies behind the last group takes no part
    for codes, scales in (host[:2], host[2:]):
        codes[:, end:], scales[end // 128:] = 0, 0
    want, size = ob.wgrad(*host, clean, np.zeros(tuple(dw.shape)) if before is None else before.astype(np.float64))
    terms = max(int(np.diff(clean).max()), 1) + 1
    bound = (ob.up(terms) + 2 * ob.up(terms) // 128) * 2.0 ** -23 * size
    assert (np.abs(dw.cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("rows,off", CASES)
def test_linear_with_offsets_past_the_rows(rows, off):
    """MokBlockLinear's dW, twice, its column codes NaN before."""
    rng = np.random.default_rng(rows)
    G, N, K = len(off) - 1, 20, 130
    lin = MokBlockLinear(up(0.05 * rng.standard_normal((G, N, K))), rows)
    for codes, scales in ((lin.xt, lin.xts), (lin.yt, lin.yts)):
        codes.fill_(NAN)
        scales.fill_(float("nan"))
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    lin.forward(up(rng.standard_normal((rows, K))), torch.zeros(rows, N, device="cuda"), offsets=o)
    dw = torch.full((G, N, K), -7.0, device="cuda")
    dy = up(rng.standard_normal((rows, N)))
    lin.backward(dy, None, dw, offsets=o)
    close(dw, lin.yt, lin.yts, lin.xt, lin.xts, off, rows)
    before = dw.cpu().numpy()
    lin.backward(dy, None, dw, offsets=o, accumulate=True)
    close(dw, lin.yt, lin.yts, lin.xt, lin.xts, off, rows, before)


@pytest.mark.parametrize("rows,off", CASES)
def test_wgrad_takes_the_rows(rows, off):
    rng = np.random.default_rng(rows)
    G, N, K = len(off) - 1, 7, 9
    P = mok.block_padded_rows(rows, G)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")

    def columns(width):
        c = torch.full((width, P), NAN, dtype=torch.uint8, device="cuda")
        s = torch.full((P // 128, width), float("nan"), device="cuda")
        mok.mok_block_quantize(up(rng.standard_normal((rows, width))), codes_t=c, scales_t=s, offsets=o)
        return c, s

    y, x, dw = columns(N), columns(K), torch.full((G, N, K), -7.0, device="cuda")
    mok.mok_block_wgrad(*y, *x, dw, offsets=o, rows=rows)
    close(dw, *y, *x, off, rows)
    for bad in (rows + 1000, -1, rows - 1000):   # not the rows of P columns
        with pytest.raises(ValueError):
            mok.mok_block_wgrad(*y, *x, dw, offsets=o, rows=bad)
