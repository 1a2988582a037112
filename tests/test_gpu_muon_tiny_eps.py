"""Muon where |u| + eps is so small that its reciprocal is beyond fp32: a zero matrix stays zero and a tiny one gives what
the definition gives, in the roundings that oracle.muon.rounded counts (twice, and half a step of fp16 and of the bf16
result, in the Frobenius norm), at the smallest eps that is accepted too."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import muon as om

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok

F = np.float32
SHAPES = [(1100, 1200), (1200, 1100), (64, 512), (512, 64), (128, 256), (4, 6), (2, 3000)]   # every kind of kernel


@pytest.mark.parametrize("eps", [1e-37, 2.0 ** -149])
@pytest.mark.parametrize("shape", SHAPES)
def test_zero_and_tiny(shape, eps):
    rng = np.random.default_rng(sum(shape))
    # |u| near 2^-127 (elements are then whole multiples of 2^-149, and exact), and ordinary values
    size = 2.0 ** -127 / np.sqrt(shape[0] * shape[1])
    u = np.stack([np.zeros(shape), size * rng.standard_normal(shape), rng.standard_normal(shape)]).astype(F)
    src, out = torch.from_numpy(u).cuda(), torch.full(u.shape, -7.0, dtype=torch.bfloat16, device="cuda")
    mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]), eps=eps)
    got = out.double().cpu().numpy()
    assert (got[0] == 0).all()
    a, b = -(-min(shape) // 32), -(-max(shape) // 32)
    small = a <= 4 and -(-b // 8) * a <= 4
    for k in (1, 2):
        x = om.orthogonalize(u[k], eps=float(F(eps)))
        cost = np.linalg.norm(om.rounded(u[k], small=small, eps=float(F(eps))) - x)
        assert np.linalg.norm(got[k] - x) <= 2 * cost + (2.0 ** -11 + 2.0 ** -8) * np.linalg.norm(x)


@pytest.mark.parametrize("shape", [(1100, 1200), (64, 512)])
def test_a_step_of_zeros(shape):
    """No gradient and no momentum: parameters take the weight decay alone."""
    p = torch.from_numpy(np.random.default_rng(1).standard_normal(shape).astype(F)).cuda()
    g, m, want = torch.zeros_like(p), torch.zeros_like(p), p * F(1 - 0.5 * 0.25)
    mok.mok_muon(mok.muon_plan([p], [g], [m]), lr=0.5, weight_decay=0.25, eps=1e-40)
    assert torch.equal(p, want) and not m.any()
