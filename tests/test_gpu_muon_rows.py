"""Orthogonalised matrices row by row and column by column, so that no single one can be wrong in a large matrix whose norm
hides it. What the stated roundings cost is oracle.muon.rounded's distance from the definition; a row (or column) may be off
by three times the largest one's cost (the kernel's fp32 sums round single elements the other way, and a row has fewer of
them for this to even out over than a matrix, which is allowed twice its cost), plus half a step of fp16, 2^-11, and of the
bf16 result, 2^-8, of its own size."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import muon as om

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok

BF = torch.bfloat16


def gradient(rng, *shape, kind):
    u = rng.standard_normal(shape)
    if kind == "low":
        r = min(shape) // 4 + 1
        return 1e-3 * (rng.standard_normal((shape[0], r)) @ rng.standard_normal((r, shape[1])) / r ** 0.5 + 0.01 * u)
    return 1e-3 * u * np.exp(0.5 * rng.standard_normal((shape[0], 1))) * np.exp(0.5 * rng.standard_normal((1, shape[1])))


def check(u, got):
    a, b = -(-min(u.shape) // 32), -(-max(u.shape) // 32)
    x = om.orthogonalize(u)
    far = om.rounded(u, small=a <= 4 and -(-b // 8) * a <= 4) - x
    for axis in (0, 1):
        norm = lambda v: np.linalg.norm(v, axis=axis)
        bound = 3 * norm(far).max() + (2.0 ** -11 + 2.0 ** -8) * norm(x)
        bad = ~(norm(got - x) <= bound)
        assert not bad.any(), (axis, np.argwhere(bad)[:5], norm(got - x)[bad][:5], bound[bad][:5])


# one workgroup, turned and not; tiles of 128, whole and cut; a call with 256 tiles of 256 and more
SHAPES = [(33, 40), (64, 64), (96, 250), (128, 256), (250, 128), (129, 129), (97, 257), (333, 129), (60, 1000), (1500, 130), (700, 701),
          (1024, 512)]


@pytest.mark.parametrize("kind", ["features", "low"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_and_columns(shape, kind):
    src = torch.from_numpy(gradient(np.random.default_rng(sum(shape)), *shape, kind=kind)).float().cuda()
    out = torch.zeros(shape, dtype=BF, device="cuda")
    mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]))
    check(src.double().cpu().numpy(), out.double().cpu().numpy())


@pytest.mark.parametrize("shape", [(1100, 1001), (700, 2050)])
def test_rows_and_columns_in_large_tiles(shape):
    rng = np.random.default_rng(sum(shape))
    src = torch.from_numpy(np.stack([gradient(rng, *shape, kind=k) for k in ("features", "low")])).float().cuda()
    src = torch.cat([src] * 9)   # (18 matrices of 20 to 27 tiles)
    out = torch.zeros(src.shape, dtype=BF, device="cuda")
    mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]))
    for k in (0, 1):
        check(src[k].double().cpu().numpy(), out[k].double().cpu().numpy())
        assert all(torch.equal(o, out[k]) for o in out[k::2])
