"""Muon on matrices whose elements lie beyond 2^31 and 2^32 bytes, and on the longest sides. A small dense matrix is spread
over far rows and columns of a zero one: the result is the small one's, spread the same way, and zero elsewhere. Bounds as
for other matrices: twice what oracle.muon.rounded's roundings cost, and half a step of fp16, 2^-11, and of bf16, 2^-8."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import muon as om

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok

BF = torch.bfloat16


def places(rng, size, count):
    """`count` of 0 .. size - 1, the first and the last ones among them."""
    ends = {0, 1, 127, 128, 255, 256, size - 129, size - 128, size - 2, size - 1} & set(range(size))
    rest = [i for i in rng.permutation(size).tolist() if i not in ends][:max(0, count - len(ends))]
    return torch.tensor(sorted(ends | set(rest)), device="cuda")


def spread(rng, rows, cols, small):
    r, c = places(rng, rows, small[0]), places(rng, cols, small[1])
    d = rng.standard_normal((len(r), len(c))) * np.exp(0.5 * rng.standard_normal((len(r), 1)))
    return r, c, torch.from_numpy(d).float().cuda()


def check(got, r, c, d, steps, extra=0.0):
    """got: the whole result; cleared on the way."""
    u = d.double().cpu().numpy()
    x = om.orthogonalize(u, steps=steps)
    far = 2 * np.linalg.norm(om.rounded(np.pad(u, ((0, 33), (0, 33))), steps=steps)[:u.shape[0], :u.shape[1]] - x)
    mine = got[r[:, None], c].double().cpu().numpy()
    assert np.linalg.norm(mine - x) <= far + (2.0 ** -11 + 2.0 ** -8 + extra) * np.linalg.norm(x)
    got[r[:, None], c] = 0
    assert not got.any()


@pytest.mark.parametrize("rows,cols", [(65536, 40), (40, 65536), (65536, 33000), (33000, 65536), (129, 65535), (65535, 300)])
def test_far_elements(rows, cols):
    rng = np.random.default_rng(rows + cols)
    r, c, d = spread(rng, rows, cols, (50, 70))
    src = torch.zeros(rows, cols, device="cuda")
    src[r[:, None], c] = d
    out = torch.full((rows, cols), -7.0, dtype=BF, device="cuda")
    mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]), steps=3)
    check(out, r, c, d, 3)


def test_far_matrices_of_a_batch():
    """The last of a batch that holds more than 2^32 bytes."""
    rng = np.random.default_rng(1)
    b, rows, cols = 9, 16384, 9000
    r, c, d = spread(rng, rows, cols, (50, 70))
    src = torch.zeros(b, rows, cols, dtype=BF, device="cuda")
    src[-1][r[:, None], c] = d.to(BF)
    out = torch.full((b, rows, cols), -7.0, dtype=BF, device="cuda")
    mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]), steps=3)
    assert not out[:-1].any()
    check(out[-1], r, c, d.to(BF).float(), 3)


def test_a_step_far_away():
    """Parameters, momentum and copy beyond 2^32 bytes: without decay, the update of a zero parameter."""
    rng = np.random.default_rng(2)
    rows, cols = 65536, 20000
    r, c, d = spread(rng, rows, cols, (50, 70))
    p, g, m = (torch.zeros(rows, cols, device="cuda") for _ in range(3))
    g[r[:, None], c] = d
    q = torch.full((rows, cols), -7.0, dtype=BF, device="cuda")
    mok.mok_muon(mok.muon_plan([p], [g], [m], [q]), lr=1.0, momentum=0.5, nesterov=False, adjust="none", steps=3)
    assert torch.equal(m, g) and torch.equal(q, p.to(BF))
    check(p.neg_(), r, c, d, 3)
