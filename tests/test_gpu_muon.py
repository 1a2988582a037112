"""Muon on the GPU against oracle.muon.

A result may be off from the definition by what the stated roundings cost, which oracle.muon.rounded finds by doing them
(X, A and B as fp16 operands, exact sums), times 2, as the kernel's fp32 sums have other last bits and so round single
elements the other way, plus half a step of fp16, 2^-11, of the result for matrices so small that this is luck,
plus half a step of the output, 2^-8 for bf16; all in the Frobenius norm of one matrix."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import muon as om

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok
from combine_router_top_schedule_amd.block import MokBlockLinear
from combine_router_top_schedule_amd.optim import MokMuon

BF = torch.bfloat16
F = np.float32


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a, F)).cuda()


def host(t):
    return t.double().cpu().numpy()


def gradient(rng, *shape, kind="features"):
    u = rng.standard_normal(shape)
    if kind == "features":
        u = u * np.exp(0.5 * rng.standard_normal(shape[:-1] + (1,))) * np.exp(0.5 * rng.standard_normal(shape[:-2] + (1, shape[-1])))
    if kind == "low":   # a few directions and noise
        r = min(shape[-2:]) // 4 + 1
        u = rng.standard_normal(shape[:-1] + (r,)) @ rng.standard_normal(shape[:-2] + (r, shape[-1])) / r ** 0.5 + 0.01 * u
    return u * 1e-3


def is_small(r, c):
    a, b = -(-min(r, c) // 32), -(-max(r, c) // 32)
    return a <= 4 and -(-b // 8) * a <= 4


def allowed(u, **kw):
    """(exact result, how far a computed one may be)"""
    x = om.orthogonalize(u, **kw)
    cost = np.linalg.norm(om.rounded(u, small=is_small(*u.shape), **kw) - x)
    return x, 2 * cost + 2.0 ** -11 * np.linalg.norm(x)


SHAPES = [(1, 1), (1, 7), (7, 1), (3, 5), (31, 33), (32, 32), (33, 1023), (1024, 30), (40, 513), (100, 97), (97, 100),
          (96, 256), (96, 257), (128, 256), (256, 128), (257, 128), (128, 257), (129, 64), (129, 129), (130, 1500),
          (700, 301), (1, 5000), (5000, 2)]


@pytest.mark.parametrize("kind", ["features", "low"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalize(shape, dtype, kind):
    src = up(gradient(np.random.default_rng(sum(shape)), *shape, kind=kind)).to(getattr(torch, dtype))
    full = torch.full((src.numel() + 64,), -7.0, dtype=BF, device="cuda")
    out = full[:src.numel()].view(shape)
    mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]))
    x, far = allowed(host(src))
    got = host(out)
    assert (full[src.numel():] == -7).all()
    assert np.linalg.norm(got - x) <= far + 2.0 ** -8 * np.linalg.norm(x), (np.linalg.norm(got - x), far, np.linalg.norm(x))


def test_orthogonalize_many():
    """More tensors than a launch takes, of both kinds, batches and leading dimensions: each as it is alone, bit for bit."""
    rng = np.random.default_rng(1)
    shapes = [(2, 3, 40, 50), (5, 129, 64), (1, 200, 300), (3, 1, 9), (0, 4, 4)] * 11
    src = [up(gradient(rng, *s)) for s in shapes]
    out = [torch.zeros(s, dtype=BF, device="cuda") for s in shapes]
    plan = mok.orthogonalize_plan(src, out)
    mok.mok_orthogonalize(plan)
    for s, o in list(zip(src, out))[::7]:
        for a, b in zip(s.view((-1,) + s.shape[-2:]), o.view((-1,) + s.shape[-2:])):
            alone = torch.zeros_like(b)
            mok.mok_orthogonalize(mok.orthogonalize_plan([a.clone()], [alone]))
            assert torch.equal(alone, b)
            x, far = allowed(host(a))
            assert np.linalg.norm(host(b) - x) <= far + 2.0 ** -8 * np.linalg.norm(x)
    keep = [o.clone() for o in out]
    mok.mok_orthogonalize(plan)
    assert all(torch.equal(a, b) for a, b in zip(keep, out))


@pytest.mark.parametrize("shape", [(2500, 2200), (2, 2048, 700)])
def test_orthogonalize_large_tiles(shape):
    """256 x 256 tiles (a large call) give what the same matrix gives among small ones."""
    rng = np.random.default_rng(2)
    src = up(gradient(rng, *shape))
    big = [up(gradient(rng, 20, 1100, 1000))]
    out, big_out = torch.zeros(shape, dtype=BF, device="cuda"), [torch.zeros(20, 1100, 1000, dtype=BF, device="cuda")]
    mok.mok_orthogonalize(mok.orthogonalize_plan([src] + big, [out] + big_out))
    one, got = src.view((-1,) + src.shape[-2:])[-1], out.view((-1,) + src.shape[-2:])[-1]
    x, far = allowed(host(one))
    assert np.linalg.norm(host(got) - x) <= far + 2.0 ** -8 * np.linalg.norm(x)
    alone = torch.zeros_like(one, dtype=BF)
    mok.mok_orthogonalize(mok.orthogonalize_plan([one.clone()], [alone]))
    assert torch.equal(alone, got)
    x, far = allowed(host(big[0][19]))
    assert np.linalg.norm(host(big_out[0][19]) - x) <= far + 2.0 ** -8 * np.linalg.norm(x)


def test_runs_of_a_bounded_workspace():
    """A batch that is cut where the workspace is full: a matrix of the second run as alone."""
    shape = (60, 2048, 1900)
    src = torch.empty(shape, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    out = torch.zeros(shape, dtype=BF, device="cuda")
    plan = mok.orthogonalize_plan([src], [out])
    assert plan.ws.numel() <= 2 << 30
    mok.mok_orthogonalize(plan)
    for k in (0, 40, 59):
        alone = torch.zeros_like(out[k])
        mok.mok_orthogonalize(mok.orthogonalize_plan([src[k].clone()], [alone]))
        assert torch.equal(alone, out[k]) and float(out[k].float().norm()) > 30


@pytest.mark.parametrize("steps,coefficients", [(1, (1.5, -0.5, 0.0)), (8, (1.5, -0.5, 0.0)), (3, [(4.0, -7.0, 3.5), (3.0, -3.2, 1.2), (1.875, -1.25, 0.375)]),
                                                (16, (1.875, -1.25, 0.375))])
@pytest.mark.parametrize("shape", [(20, 50), (150, 90)])
def test_other_coefficients(shape, steps, coefficients):
    src = up(gradient(np.random.default_rng(3), *shape))
    out = torch.zeros(shape, dtype=BF, device="cuda")
    mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]), steps=steps, coefficients=coefficients, eps=1e-5)
    rows = [coefficients] * steps if not isinstance(coefficients, list) else coefficients
    x, far = allowed(host(src), eps=float(F(1e-5)), steps=steps, coefficients=rows)
    assert np.linalg.norm(host(out) - x) <= far + 2.0 ** -8 * np.linalg.norm(x)


@pytest.mark.parametrize("shape", [(3, 40, 60), (3, 140, 200)])
def test_zero_and_not_finite(shape):
    """Zeros stay zeros, tiny and huge values lose nothing, and a matrix that is not finite spoils itself alone."""
    rng = np.random.default_rng(4)
    u = gradient(rng, *shape)
    cases = [u * 1e-30, u * 1e30, u]
    for bad in (np.nan, np.inf, 0.0):
        v = u.copy()
        if bad == 0.0:
            v[1] = 0
        else:
            v[1, 3, 5] = bad
        cases.append(v)
    for v in cases:
        src, out = up(v), torch.full(shape, 5.0, dtype=BF, device="cuda")
        mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]), eps=1e-37)
        got = host(out)
        if not np.isfinite(v).all():
            assert np.isnan(got[1]).all()
        for k in (0, 1, 2):
            if np.isfinite(v[k]).all():
                x, far = allowed(host(src[k]), eps=float(F(1e-37)))
                assert np.linalg.norm(got[k] - x) <= far + 2.0 ** -8 * np.linalg.norm(x)
        if not v[1].any():
            assert not got[1].any()


class Case:
    """Tensors with guards behind, and their host copies."""

    def __init__(self, shapes, grad="float32", copy=True, seed=0):
        rng = np.random.default_rng(seed)
        self.full = {k: [] for k in "pgmc"}
        for s in shapes:
            n = int(np.prod(s))
            guard = lambda a, dt: torch.cat([a.flatten(), torch.full((32,), -7.0, device="cuda")]).to(dt)
            for k, a, dt in (("p", 0.02 * rng.standard_normal(s), torch.float32), ("g", gradient(rng, *s), getattr(torch, grad)),
                             ("m", gradient(rng, *s), torch.float32), ("c", np.zeros(s), BF)):
                self.full[k].append(guard(up(a), dt))
        view = lambda k: [t[:int(np.prod(s))].view(s) for t, s in zip(self.full[k], shapes)]
        self.p, self.g, self.m, self.c = (view(k) for k in "pgmc")
        if not copy:
            self.c = None
        self.before = [(host(p), host(g), host(m)) for p, g, m in zip(self.p, self.g, self.m)]
        self.plan = mok.muon_plan(self.p, self.g, self.m, self.c)

    def check(self, lr, **kw):
        """p: its two roundings of 2^-24 and the coefficients' two of p and of the update, and the update's allowance; m: a
        product, a sum and two roundings of inputs' products, 4 of 2^-24 of the terms."""
        for i, (p0, g0, m0) in enumerate(self.before):
            mats = lambda a: a.reshape((-1,) + a.shape[-2:])
            for k, (p, g, m, q, n) in enumerate(zip(*map(mats, (p0, g0, m0, host(self.p[i]), host(self.m[i]))))):
                want, mw, u = om.step(p, g, m, lr, **kw)
                scale = kw["max_norm"] / kw["norm"] if kw.get("norm") and kw["norm"] > kw["max_norm"] else 1.0
                assert (np.abs(n - mw) <= 4 * 2.0 ** -24 * (np.abs(m) + np.abs(g) * scale)).all()
                ns = {k: kw[k] for k in ("eps", "steps", "coefficients") if k in kw}
                x, far = allowed(u, **ns)
                r = lr * om.adjustment(kw.get("adjust", "rms"), *p.shape)
                # (u itself is fp32 arithmetic: 6 roundings of 2^-24, which the first step's slope 3.4 to the fifth, 485, may carry)
                far = far + 485 * 6 * 2.0 ** -24 * np.linalg.norm(x)
                assert np.linalg.norm(q - want) <= r * far + 4 * 2.0 ** -24 * (np.linalg.norm(p) + r * np.linalg.norm(x))
            if self.c is not None:
                assert torch.equal(self.c[i], self.p[i].to(BF))
            for k in "pgm" + ("c" if self.c is not None else ""):
                assert (self.full[k][i][-32:] == -7).all()


STEP = [(2, 256, 128), (8, 128), (3, 60, 200), (1, 333, 129), (2, 130, 270), (1, 5)]


@pytest.mark.parametrize("grad,copy,nesterov,adjust", [("float32", True, True, "rms"), ("bfloat16", False, False, "spectral"),
                                                       ("bfloat16", True, True, "none")])
def test_step(grad, copy, nesterov, adjust):
    c = Case(STEP, grad, copy)
    mok.mok_muon(c.plan, lr=2e-3, momentum=0.9, nesterov=nesterov, weight_decay=0.1, adjust=adjust)
    c.check(2e-3, momentum=0.9, nesterov=nesterov, weight_decay=0.1, adjust=adjust)


def test_odd_columns_and_large_tiles():
    c = Case([(20, 1100, 1001), (2, 700, 301), (1, 301, 700)], seed=5)
    c.before = [tuple(a[:1] for a in b) for b in c.before]
    c.p, c.m = [p[:1] for p in c.p], [m[:1] for m in c.m]
    c.c = None
    mok.mok_muon(c.plan, lr=2e-3)
    c.check(2e-3)


def test_clipping_and_left_out_steps():
    for norm, scale in ((2.0, 0.5), (0.25, 1.0)):
        c = Case(STEP, seed=2)
        sq = torch.tensor([norm * norm], dtype=torch.float64, device="cuda")
        mok.mok_muon(c.plan, lr=1e-3, sumsq=sq, max_norm=1.0)
        c.check(1e-3, norm=norm, max_norm=1.0)
    for bad in (float("nan"), float("inf")):
        c = Case(STEP, seed=3)
        keep = [t.clone() for k in "pmc" for t in c.full[k]]
        mok.mok_muon(c.plan, lr=1e-3, sumsq=torch.tensor([bad], dtype=torch.float64, device="cuda"))
        mok.mok_muon(c.plan, lr=torch.tensor([-1.0 if bad != bad else bad], dtype=torch.float64, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(keep, [t for k in "pmc" for t in c.full[k]]))


def test_rate_on_the_device_in_a_graph():
    """A captured step follows gradients and rate that change between replays, as eager steps do."""
    a, b = Case(STEP, seed=4), Case(STEP, seed=4)
    lr = torch.tensor([1e-3], dtype=torch.float64, device="cuda")
    mok.mok_muon(a.plan, lr=lr)
    mok.mok_muon(b.plan, lr=1e-3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mok.mok_muon(a.plan, lr=lr)
    for k in range(3):
        lr.fill_(2e-3 / (k + 1))
        for x, y in zip(a.g, b.g):
            x.mul_(1.5)
            y.mul_(1.5)
        torch.cuda.synchronize()
        graph.replay()
        mok.mok_muon(b.plan, lr=2e-3 / (k + 1))
        torch.cuda.synchronize()
        for x, y in zip(a.p + a.m + a.c, b.p + b.m + b.c):
            assert torch.equal(x, y)


def test_two_plans_at_once():
    a, b, ra, rb = Case(STEP, seed=6), Case(STEP, seed=7), Case(STEP, seed=6), Case(STEP, seed=7)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        mok.mok_muon(a.plan, lr=1e-3, stream=one)
        mok.mok_muon(b.plan, lr=1e-3, stream=two)
    torch.cuda.synchronize()
    for _ in range(3):
        mok.mok_muon(ra.plan, lr=1e-3)
        mok.mok_muon(rb.plan, lr=1e-3)
    for x, y in zip(a.p + b.p + a.m + b.m, ra.p + rb.p + ra.m + rb.m):
        assert torch.equal(x, y)


def test_mok_muon_class():
    c = Case(STEP, grad="bfloat16", seed=8)
    opt = MokMuon(c.p, c.g, c.c, lr=5e-3, max_norm=0.01, weight_decay=0.1)
    c.before = [(p, g, np.zeros_like(m)) for p, g, m in c.before]
    c.m = opt.m
    opt.step(lr=1e-3)
    norm = float(np.sqrt(sum((g ** 2).sum() for _, g, _ in c.before)))
    for k in "m":
        c.full[k] = [torch.full((32,), -7.0, device="cuda")] * len(c.m)
    c.check(1e-3, weight_decay=0.1, norm=norm, max_norm=0.01)


def test_plan_refusals():
    p, g, m = (torch.zeros(2, 3, 4, device="cuda") for _ in range(3))
    c = torch.zeros(2, 3, 4, dtype=BF, device="cuda")
    bad = [lambda: mok.muon_plan([p], [g], [m, m]), lambda: mok.muon_plan([p.double()], [g], [m]), lambda: mok.muon_plan([p], [g.half()], [m]),
           lambda: mok.muon_plan([p], [g[:1]], [m]), lambda: mok.muon_plan([p], [g], [p]), lambda: mok.muon_plan([p, p], [g, g], [m, m.clone()]),
           lambda: mok.muon_plan([p[0, 0]], [g[0, 0]], [m[0, 0]]), lambda: mok.muon_plan([p], [g], [m], [c.float()]),
           lambda: mok.muon_plan([p.transpose(1, 2)], [g.transpose(1, 2)], [m.transpose(1, 2)]), lambda: mok.muon_plan([p], [g.cpu()], [m]),
           lambda: mok.orthogonalize_plan([p], [c.float()]), lambda: mok.orthogonalize_plan([c], [c]), lambda: mok.orthogonalize_plan([p], []),
           lambda: mok.orthogonalize_plan([p], [c[:1]])]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"plan {i} was not refused")
    plan = mok.muon_plan([p], [g], [m], [c])
    for f in (lambda: mok.mok_muon(plan, lr=1.0, max_norm=1.0), lambda: mok.mok_muon(plan, lr=torch.zeros(1, device="cuda")),
              lambda: mok.mok_muon(plan, lr=1.0, sumsq=1.0), lambda: mok.mok_muon(plan, lr=1.0, steps=0)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(mok.MokError):
        mok.mok_muon(plan, lr=-1.0)
    with pytest.raises(mok.MokError):
        mok.orthogonalize_plan([torch.zeros(1, 0, 4, device="cuda")], [torch.zeros(1, 0, 4, dtype=BF, device="cuda")])


def test_training_step_of_an_experts_map():
    """A few steps together: product, gradients, Muon, weights quantised again. What each step's calls give is checked by
    the tests above; here that the next product uses the updated weights, and that nothing goes wrong between them."""
    rng = np.random.default_rng(9)
    R, N, K, off = 160, 40, 70, torch.tensor([0, 100, 160], dtype=torch.int32, device="cuda")
    w = up(0.1 * rng.standard_normal((2, N, K)))
    lin, dw = MokBlockLinear(w, R), torch.zeros_like(w)
    opt = MokMuon([w], [dw], lr=0.02, check_finite=True)
    x, goal = up(rng.standard_normal((R, K))), up(rng.standard_normal((R, N)))
    out, seen = torch.zeros(R, N, device="cuda"), []
    for _ in range(4):
        lin.forward(x, out, offsets=off)
        dy = out - goal
        lin.backward(dy, None, dw, offsets=off)
        before = w.clone()
        opt.step()
        lin.refresh_weights()
        assert not torch.equal(before, w) and torch.isfinite(w).all()
        seen.append(lin.wq.clone())
    assert all(not torch.equal(a, b) for a, b in zip(seen, seen[1:]))


def test_many_small_matrices():
    """100,000 matrices in one call, the last as alone."""
    src = torch.empty(100_000, 9, 5, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    out = torch.zeros(src.shape, dtype=BF, device="cuda")
    mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]))
    for k in (0, 65_537, 99_999):
        alone = torch.zeros(9, 5, dtype=BF, device="cuda")
        mok.mok_orthogonalize(mok.orthogonalize_plan([src[k].clone()], [alone]))
        x, far = allowed(host(src[k]))
        assert torch.equal(alone, out[k]) and np.linalg.norm(host(alone) - x) <= far + 2.0 ** -8 * np.linalg.norm(x)


# (the call takes its coefficients in fp32)
COEFFICIENTS = [tuple(float(F(c)) for c in om.JORDAN)] * 5
THIN = [(1, 1), (1, 1024), (1025, 1), (2, 3), (5, 5), (7, 1024), (8, 1025), (9, 1000), (16, 512), (513, 16), (17, 31), (32, 32),
        (256, 32), (32, 257), (20, 2360), (2360, 19), (31, 5001), (2, 65536), (65536, 32)]


@pytest.mark.parametrize("kind", ["features", "low"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("shape", THIN)
def test_thin_matrices_element_by_element(shape, dtype, kind):
    """Up to 32 rows or columns: the source is exact in fp64 and so are the steps (to 1e-12, errors of A growing by 3.44^2 in
    each of five); what is rounded is the result, to fp32 and then by half a step of bf16, 2^-8, at most (2^-133 below 2^-126)."""
    src = up(gradient(np.random.default_rng(sum(shape)), 2, *shape, kind=kind)).to(getattr(torch, dtype))
    out = torch.zeros(src.shape, dtype=BF, device="cuda")
    mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]))
    for s, o in zip(host(src), host(out)):
        x = om.orthogonalize(s, coefficients=COEFFICIENTS)
        assert (np.abs(o - x) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(x) + 1e-9 * np.abs(x).max()).all()


@pytest.mark.parametrize("shape", [(3, 5), (24, 300), (300, 24), (32, 700), (3000, 7)])
def test_thin_update(shape):
    """Momentum and gradient that make u without a rounding (multiples of 2^-12 below 1, momentum 1/2): the update has those of
    the rate, the result, the decay factor and two products and a sum, each 2^-24 of what it rounds."""
    rng = np.random.default_rng(shape[0])
    g, m = (np.rint(rng.uniform(-1, 1, shape) * 4096) / 4096 for _ in range(2))
    p = rng.standard_normal(shape)
    tp, tg, tm = up(p), up(g), up(m)
    p = host(tp)
    mok.mok_muon(mok.muon_plan([tp], [tg], [tm]), lr=0.01, momentum=0.5, weight_decay=0.1, adjust="spectral")
    want, mw, _ = om.step(p, g, m, 0.01, momentum=0.5, weight_decay=0.1, adjust="spectral", coefficients=COEFFICIENTS)
    assert np.array_equal(host(tm), mw)
    assert (np.abs(host(tp) - want) <= 4 * 2.0 ** -24 * (np.abs(p) + np.abs(want - p * (1 - 0.001))) + 1e-11).all()


def test_thin_zero_and_not_finite():
    for shape in ((4, 6), (5, 3000)):
        src = torch.randn(3, *shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
        src[0] = 0
        src[1, 2, 1] = float("inf")
        out = torch.full(src.shape, -7.0, dtype=BF, device="cuda")
        mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]))
        assert (out[0] == 0).all() and out[1].isnan().all() and out[2].isfinite().all()


def test_thin_and_others_in_one_graph():
    """Small, long thin and large matrices of one call, captured and replayed."""
    shapes = [(2, 6, 40), (1, 30, 3000), (2, 300, 260), (1, 100, 90), (1, 2000, 3)]
    a, b = Case(shapes, seed=8), Case(shapes, seed=8)
    mok.mok_muon(b.plan, lr=1e-3)
    graph = torch.cuda.CUDAGraph()
    mine = Case(shapes, seed=9)
    mok.mok_muon(mine.plan, lr=1e-3)
    with torch.cuda.graph(graph):
        mok.mok_muon(a.plan, lr=1e-3)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(a.p + a.m + a.c, b.p + b.m + b.c):
            assert torch.equal(x, y)
        for x in a.g + b.g:
            x.mul_(0.75)
        mok.mok_muon(b.plan, lr=1e-3)
        torch.cuda.synchronize()


def test_matrices_of_a_few_more_rows_than_thin():
    """33 to 64 rows, in one workgroup or the general kernels."""
    for shape in ((33, 40), (33, 257), (40, 700), (700, 40), (33, 5000), (64, 64)):
        src = up(gradient(np.random.default_rng(3), *shape))
        out = torch.zeros(shape, dtype=BF, device="cuda")
        mok.mok_orthogonalize(mok.orthogonalize_plan([src], [out]))
        x, far = allowed(host(src))
        assert np.linalg.norm(host(out) - x) <= far + 2.0 ** -8 * np.linalg.norm(x)
