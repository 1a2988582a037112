"""The 8-bit moments of mok_adamw against the rounding's definition in whole numbers.

A last bit lost ahead of a stochastic rounding changes a code about once in 10^6 elements, so the
comparison runs over 10^8 of them, in two steps that follow one another; and at the borders themselves,
where the code has to change from one fp32 number to the next."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import optim as oo

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok

M32 = 0xFFFFFFFF


def mix(h):
    h = h ^ (h >> 16)
    h = (h * 0x6A09E667) & M32
    h = h ^ (h >> 15)
    h = (h * 0xBB67AE85) & M32
    return h ^ (h >> 16)


def bits(seed, first, n):
    """Of the elements first .. first + n - 1 (below 2^32) of a call's first tensor."""
    return mix(torch.arange(first, first + n, device="cuda") ^ int(oo.mix(oo.mix(seed))))


def power(code):
    """2^(code - 127) from its bits."""
    return torch.where(code > 0, code << 23, 1 << 22).to(torch.int32).view(torch.float32)


def decode(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().view(-1, 32)
    return (v * power(scales.long())[:, None]).view(-1)


def encode(x, u, positive):
    """Codes and scales of whole runs, from the bits of x alone (no value below 2^-126 but zero)."""
    b = x.view(torch.int32).view(-1, 32).long()
    mag = b & 0x7FFFFFFF
    assert not bool(((mag > 0) & (mag < 0x800000)).any())
    top = mag.amax(1)
    c = ((top >> 23) - 8 + ((top & 0x7FFFFF) > 0x600000)).clamp_min(0)
    man = torch.where(mag > 0, (mag & 0x7FFFFF) | 0x800000, 0)
    low = (mag >> 23) - 150 - (c[:, None] - 127)       # |x| = man 2^low scales
    q = (low + 23).clamp_min(-6) - 3                   # a code's step is 2^q scales
    cut = (q - low).clamp_max(40)                      # >= 20; from 40 on less than 2^-16 of a step is there
    k = (man + (u.view(-1, 32) << (cut - 16))) >> cut
    if positive:
        k = torch.where(man > 0, k.clamp_min(1), k)
    # a step's exponent field, and a mantissa that carries into it at 16 steps; below 8 steps the code is k
    code = torch.where(k < 8, k, ((q + 10) << 3) + k - 8) | ((b < 0).long() << 7)
    return code.to(torch.uint8).view(-1), c.to(torch.uint8)


def test_two_steps_of_many_elements():
    n, part = 1 << 27, 1 << 24
    z = lambda k, dt=torch.float32: torch.zeros(k, dtype=dt, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(6)
    size = torch.randn(n, generator=gen, device="cuda").mul_(2).exp_().mul_(1e-3)
    p = torch.randn(n, generator=gen, device="cuda").mul_(0.02)
    g, m, v, ms, vs = z(n), z(n, torch.uint8), z(n, torch.uint8), z(n // 32, torch.uint8), z(n // 32, torch.uint8)
    plan = mok.adamw_plan(p=[p], g=[g], m=[m], v=[v], m_scale=[ms], v_scale=[vs])
    lr, b1, b2, eps, wd = 3e-3, 0.9, 0.999, 1e-8, 0.1
    for step in range(1, 6):       # three steps make a state, two are compared
        g.normal_(generator=gen).mul_(size)
        old = [t.clone() for t in (p, m, v, ms, vs)]
        mok.mok_adamw(plan, lr=lr, step=step, beta1=b1, beta2=b2, eps=eps, weight_decay=wd, seed=40 + step)
        if step < 4:
            continue
        for a in range(0, n, part):
            w, r = slice(a, a + part), slice(a // 32, (a + part) // 32)
            p0, m0, v0 = old[0][w], decode(old[1][w], old[3][r]), decode(old[2][w], old[4][r])
            gw = g[w]
            mw = m0 * b1 + gw * (1 - b1)
            root = torch.sqrt(v0 * v0 * b2 + gw * gw * (1 - b2))
            down1, down2 = 1 - b1 ** step, 1 - b2 ** step
            pw = p0 * (1 - lr * wd) - mw / (root * (1 / math.sqrt(down2)) + eps) * (lr / down1)
            u = bits(40 + step, a, part)
            for name, x, code, scale, bit in (("m", mw, m, ms, u & 0xFFFF), ("v", root, v, vs, u >> 16)):
                c, s = encode(x, bit, name == "v")
                assert torch.equal(scale[r], s), (step, name, a)
                assert torch.equal(code[w], c), (step, name, a)
            assert torch.equal(p[w], pw), (step, a)


@pytest.mark.parametrize("below", [False, True])
@pytest.mark.parametrize("steps", [(1, 8), (9, 16)], ids=["subnormal", "normal"])
def test_borders(steps, below):
    """With beta1 = 0 a zero moment becomes the gradient. At i - u / 2^16 steps the code is i, one fp32 unit
    below it i - 1."""
    n, seed = 1 << 20, 9
    rng = np.random.default_rng(7)
    u = (oo.bits(seed, 0, n) & 0xFFFF).astype(np.int64)
    i = rng.integers(steps[0], steps[1] + 1, n)
    if steps[0] == 1:
        i[u > 32768] = 1           # (borders below half a step)
    step = 2.0 ** -9 if steps[0] == 1 else 2.0 ** rng.integers(-9, 5, n)
    x = ((i * 65536 - u) / 65536 * step).astype(np.float32)
    if below:
        x = np.nextafter(x, np.float32(0))
    sign = rng.choice([-1.0, 1.0], n).astype(np.float32)
    x *= sign
    x[::32] = 448.0
    want = sign * (i - below) * step
    want[::32] = 448.0
    z = lambda k, dt=torch.uint8: torch.zeros(k, dtype=dt, device="cuda")
    p, m, v, ms, vs = z(n, torch.float32), z(n), z(n), z(n // 32), z(n // 32)
    mok.mok_adamw(mok.adamw_plan(p=[p], g=[torch.from_numpy(x).cuda()], m=[m], v=[v], m_scale=[ms], v_scale=[vs]),
                  lr=1e-3, step=1, beta1=0.0, seed=seed)
    assert (ms == 127).all()
    got = m.view(torch.float8_e4m3fn).float().cpu().numpy()
    assert np.array_equal(got, want.astype(np.float32))
