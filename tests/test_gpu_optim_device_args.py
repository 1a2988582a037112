"""Rate and step number of mok_adamw on the device: values that the host form refuses change nothing."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok
from combine_router_top_schedule_amd.optim import MokAdamW


def tensors(mx, bf):
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = [5000, 33, 1]
    new = lambda dt: [torch.randn(k, generator=gen, device="cuda").to(dt) for k in n]
    z = lambda dt, div=1: [torch.zeros(-(-k // div), dtype=dt, device="cuda") for k in n]
    t = dict(p=new(torch.bfloat16 if bf else torch.float32), g=new(torch.float32))
    if mx:
        t.update(m=z(torch.uint8), v=z(torch.uint8), m_scale=z(torch.uint8, 32), v_scale=z(torch.uint8, 32))
    else:
        t.update(m=z(torch.float32), v=z(torch.float32))
    if not bf:
        t["copy"] = z(torch.bfloat16)
    return t


@pytest.mark.parametrize("bf", [False, True])
@pytest.mark.parametrize("mx", [False, True])
def test_refused_values_change_nothing(mx, bf):
    t = tensors(mx, bf)
    plan = mok.adamw_plan(**t)
    # one step, so that the moments hold something
    mok.mok_adamw(plan, lr=1e-3, step=1)
    before = {k: [x.clone() for x in v] for k, v in t.items()}
    lr = torch.tensor([1e-3], dtype=torch.float64, device="cuda")
    step = torch.tensor([2], dtype=torch.int64, device="cuda")
    for number in (0, -1, -2 ** 63):
        step.fill_(number)
        mok.mok_adamw(plan, lr=1e-3, step=step, weight_decay=0.1)
        mok.mok_adamw(plan, lr=lr, step=step, weight_decay=0.1)
    step.fill_(2)
    for rate in (-1e-3, math.nan, math.inf, -math.inf):
        lr.fill_(rate)
        mok.mok_adamw(plan, lr=lr, step=2, weight_decay=0.1)
        mok.mok_adamw(plan, lr=lr, step=step, weight_decay=0.1)
    for k, v in t.items():
        assert all(torch.equal(a, b) for a, b in zip(v, before[k])), k
    # and the calls that the host takes as well still run: a rate of 0 moves the moments alone
    lr.fill_(0.0)
    mok.mok_adamw(plan, lr=lr, step=step)
    assert all(torch.equal(a, b) for a, b in zip(t["p"], before["p"]))
    assert not torch.equal(t["m"][0], before["m"][0])
    lr.fill_(1e-3)
    step.fill_(2 ** 62)
    mok.mok_adamw(plan, lr=lr, step=step)
    assert all(torch.isfinite(a).all() and not torch.equal(a, b) for a, b in zip(t["p"][:1], before["p"][:1]))


def test_a_refused_call_is_no_step():
    gen = torch.Generator(device="cuda").manual_seed(2)
    new = lambda: torch.randn(100, generator=gen, device="cuda")
    p, g = new(), new()
    q = p.clone()
    opt, ref = MokAdamW([p], [g], max_norm=1.0, state="mxfp8"), MokAdamW([q], [g], max_norm=1.0, state="mxfp8")
    for bad in (-1.0, math.nan, math.inf):
        with pytest.raises(mok.MokError):
            opt.step(lr=bad)
    assert opt.steps == 0
    for _ in range(3):
        opt.step()
        ref.step()
    assert opt.steps == ref.steps == 3 and torch.equal(p, q)
    assert torch.equal(opt.m[0], ref.m[0]) and torch.equal(opt.v[0], ref.v[0])
