"""mok_route_fwd and mok_route_bwd against the fp64 oracle.

Choices have to be those of exact arithmetic, so they are compared for equality. Weights are fp32: a
chosen logit's f = x or log sigmoid(x) carries at most 4 units of 2^-23 of max(1, |f|) (the library's
log1p and exp, a subtraction; none where f = x), its difference to the largest f half a unit more, the exponential turns
that into a relative error and adds 2 units, the sum of K terms K / 2, quotient and scale 2 more; the sum
itself carries the same errors. tol() doubles that. A gradient's terms c q_k |dw_k| and c q_k sum |dw_j q_j|
carry a few of these each; bf16 results are rounded once more, by half a step (2^-8 of the value)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import route as orr

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok

U = 2.0 ** -23


def desc(g):
    return mok.route_desc(g.E, g.K, g.score, g.groups, g.top_groups, g.group_score, g.renorm, g.scale)


def tol(gate, x, idx):
    """Relative error allowed to each row's weights, [N][1]. A softmax subtracts its largest logit first, and
    the inputs are exact: what counts there is the distance to it (beyond 104 the weight is 0 in fp32)."""
    some = idx >= 0
    f = np.where(some, np.take_along_axis(x, np.maximum(idx, 0), 1), 0.0)
    if gate.score == "sigmoid":
        big = np.where(some, np.logaddexp(0, -f), 0).max(1)
    else:
        top = np.where(some, f, -np.inf).max(1) if gate.renorm else x.max(1)
        top = np.where(np.isfinite(top), top, 0.0)
        big = np.minimum(np.where(some, top[:, None] - f, 0).max(1), 104)
    terms = gate.K if gate.renorm else gate.E if gate.score == "softmax" else 1
    return (2 * U * (5 * np.maximum(1.0, big) + terms / 2 + 6))[:, None]


class Run:
    """Inputs on the device with rows `pad` apart, outputs with guard rows behind."""

    def __init__(self, gate, x, bias=None, mask=None, dtype="float32", pad=0):
        self.gate, self.N = gate, len(x)
        wide = torch.full((self.N, gate.E + pad), float("nan"), device="cuda").to(getattr(torch, dtype))
        self.x = wide[:, :gate.E]
        self.x.copy_(torch.from_numpy(np.asarray(x, np.float32)))
        self.x64 = self.x.double().cpu().numpy()
        self.bias = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
        self.b64 = None if bias is None else self.bias.double().cpu().numpy()
        self.mask = None if mask is None else torch.tensor(np.asarray(mask), dtype=torch.uint8, device="cuda")
        self.m = mask
        self.idx = torch.full((self.N + 3, gate.K), -77, dtype=torch.int32, device="cuda")
        self.w = torch.full((self.N + 3, gate.K), -77.0, device="cuda")
        self.load = torch.full((gate.E + 3,), -77, dtype=torch.int32, device="cuda")
        self.dx = torch.full((self.N + 3, gate.E), -77.0, device="cuda").to(getattr(torch, dtype))

    def forward(self, stream=None):
        n = self.N
        mok.mok_route_fwd(desc(self.gate), self.x, self.idx[:n], self.w[:n], bias=self.bias,
                          token_mask=self.mask, load=self.load[:self.gate.E], stream=stream)

    def check_forward(self):
        idx, w, load = orr.forward(self.gate, self.x64, self.b64, self.m)
        got = self.idx.cpu().numpy()
        assert np.array_equal(got[:self.N], idx)
        assert np.array_equal(self.load.cpu().numpy()[:self.gate.E], load)
        gw = self.w.cpu().numpy().astype(np.float64)
        x = np.where(np.asarray(self.m, bool)[:, None], self.x64, 0) if self.m is not None else self.x64
        x = np.nan_to_num(x, nan=0.0)
        err = np.abs(gw[:self.N] - w)
        bad = ~(err <= tol(self.gate, x, idx) * np.abs(w) + 1e-37)
        assert not bad.any(), (np.argwhere(bad)[:5], gw[:self.N][bad][:5], w[bad][:5])
        # what lies behind the last row is as it was
        assert (got[self.N:] == -77).all() and (gw[self.N:] == -77).all()
        assert (self.load.cpu().numpy()[self.gate.E:] == -77).all()
        return idx, w

    def check_backward(self, idx, seed=0):
        g, n = self.gate, self.N
        dw = np.random.default_rng(seed).standard_normal((n, g.K)).astype(np.float32)
        dw[idx < 0] = np.nan    # not to be used
        mok.mok_route_bwd(desc(g), self.x, torch.from_numpy(idx).cuda(), torch.from_numpy(dw).cuda(),
                          self.dx[:n])
        ref = orr.backward(g, self.x64, idx, dw)
        got = self.dx.double().cpu().numpy()
        # sum over the slots of |dw| q scale, the size of what is added up
        with np.errstate(invalid="ignore", over="ignore"):
            size = np.zeros((n, g.E))
            for r in range(n):
                of = [int(i) for i in idx[r] if i >= 0]
                if of:
                    q = orr.weights_row(g, self.x64[r], of)
                    t = np.abs(dw[r, :len(of)])
                    size[r, of] += q * t + q * (q * t).sum() / g.scale
                    if g.score == "softmax" and not g.renorm:
                        size[r] += orr.scores(g, self.x64[r]) * (q * t).sum()
        x = np.where((idx >= 0).any(1)[:, None], np.nan_to_num(self.x64, nan=0.0), 0)
        bound = 4 * tol(g, x, idx) * size + 1e-37
        if self.dx.dtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * np.abs(ref)
        bad = ~(np.abs(got[:n] - ref) <= bound)
        assert not bad.any(), (np.argwhere(bad)[:5], got[:n][bad][:5], ref[bad][:5])
        assert (got[n:] == -77).all() or (got[n:] == float(torch.tensor(-77.0).bfloat16())).all()


G = orr.Gate
GATES = {
    "layer": G(8, 2),
    "one": G(1, 1, "sigmoid"),
    "dsv3": G(256, 8, "sigmoid", 8, 4, "top2", True, 2.5),
    "kimi": G(384, 8, "sigmoid", 1, 1, "max", True, 2.5),
    "max_groups": G(160, 6, "softmax", 8, 3, "max", False, 16.0),
    "softmax_top2": G(64, 4, "softmax", 4, 2, "top2", True),
    "odd": G(60, 4, "softmax", 1, 1, "max", False),
    "odd_groups": G(63, 5, "sigmoid", 9, 4, "top2", False, 1.5),
    "single_expert_groups": G(24, 3, "sigmoid", 24, 5, "top2"),
    "many_groups": G(128, 16, "sigmoid", 64, 8, "max"),
    "widest": G(1024, 16, "sigmoid", 16, 5, "top2", True, 2.5),
    "widest_softmax": G(1023, 16, "softmax", 1, 1, "max", False),
    "all_chosen": G(16, 16, "sigmoid", 1, 1, "max", False),
    "two": G(2, 1, "softmax", 1, 1, "max", False),
}


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("name", list(GATES))
def test_route(name, bias, dtype):
    gate = GATES[name]
    rng = np.random.default_rng(len(name))
    n = 157
    x = rng.standard_normal((n, gate.E)) * 1.5
    mask = rng.random(n) > 0.1
    x[~mask] = np.nan
    hole = rng.random((n, gate.E)) < 0.1
    x[hole & mask[:, None]] = -np.inf
    x[3], mask[3] = -np.inf, True                  # nothing to choose
    x[4], mask[4] = -np.inf, True
    x[4, gate.E // 2] = 0.5                        # one
    x[5], mask[5] = -3.4e38, True                  # barred in all but name: a row of equal logits
    x[6], mask[6] = 0.25, True
    if gate.score == "sigmoid":                    # scores too small and too near 1 for fp32
        x[7], mask[7] = -200 - rng.random(gate.E), True
        x[8], mask[8] = 20 + rng.random(gate.E), True
    r = Run(gate, x, 0.02 * rng.integers(-9, 10, gate.E) if bias else None, mask, dtype, pad=len(name) % 4)
    r.forward()
    idx, _ = r.check_forward()
    r.check_backward(idx)


@pytest.mark.parametrize("n", [0, 1, 2, 7, 8, 9, 31, 33, 1000])
@pytest.mark.parametrize("name", ["layer", "dsv3", "odd", "many_groups"])
def test_route_token_counts(name, n):
    gate = GATES[name]
    rng = np.random.default_rng(n)
    r = Run(gate, rng.standard_normal((n, gate.E)), 0.1 * rng.standard_normal(gate.E))
    r.forward()
    idx, _ = r.check_forward()
    r.check_backward(idx)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("name", ["layer", "dsv3", "kimi", "softmax_top2", "odd", "widest"])
def test_route_ties_go_to_the_lower_id(name, bias):
    gate = GATES[name]
    rng = np.random.default_rng(5)
    x = rng.integers(-1, 2, (64, gate.E)) * 0.5
    x[:4] = 0.0
    x[3, ::2] = -0.0
    r = Run(gate, x, 0.25 * rng.integers(0, 2, gate.E) if bias else None)
    r.forward()
    r.check_forward()


@pytest.mark.parametrize("name", ["dsv3", "kimi", "widest", "odd_groups", "softmax_top2", "max_groups"])
def test_route_choices_closer_than_fp32(name):
    """Keys that fp32 cannot tell apart: logits near 16 whose sigmoids round to the same few floats, and
    logits that differ in their last bit under a bias."""
    gate = GATES[name]
    rng = np.random.default_rng(6)
    x = np.where(rng.random((96, gate.E)) < 0.5, 1.0, 0.25) + rng.integers(0, 5, (96, gate.E)) * 2.0 ** -22
    x[:32] = 14 + 2 * rng.random((32, gate.E))
    b = rng.integers(0, 3, gate.E) * 0.125
    r = Run(gate, x, b)
    r.forward()
    r.check_forward()


@pytest.mark.parametrize("bias", [False, True])
def test_route_many_rows_of_equal_logits(bias):
    """Many tokens that fp32 cannot decide (all their logits alike), and others between them."""
    gate, n = G(64, 8, "sigmoid", 8, 4, "top2", True, 2.5), 200001
    x = torch.zeros(n, 64, device="cuda")
    some = torch.arange(0, n, 17, device="cuda")
    x[some] = torch.randn(len(some), 64, device="cuda")
    b = torch.zeros(64, device="cuda") if bias else None
    idx = torch.full((n, 8), -5, dtype=torch.int32, device="cuda")
    w, load = torch.empty(n, 8, device="cuda"), torch.empty(64, dtype=torch.int32, device="cuda")
    mok.mok_route_fwd(desc(gate), x, idx, w, bias=b, load=load)
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[some] = False
    assert (idx[rest] == torch.arange(8, device="cuda")).all() and (w[rest] == 2.5 / 8).all()
    pick = some[:300]
    ref, _, _ = orr.forward(gate, x[pick].double().cpu().numpy(), None if b is None else np.zeros(64))
    assert np.array_equal(idx[pick].cpu().numpy(), ref)
    assert torch.equal(load.long(), torch.bincount(idx.flatten().long(), minlength=64))


def test_route_bias_bars_and_forces_experts():
    gate = GATES["kimi"]
    rng = np.random.default_rng(7)
    b = np.zeros(gate.E)
    b[::3] = -np.inf
    b[5] = np.inf
    b[7] = np.nan
    r = Run(gate, rng.standard_normal((40, gate.E)), b)
    r.forward()
    idx, _ = r.check_forward()
    assert (idx[:, 0] == 5).all() and not (idx % 3 == 0).any() and not (idx == 7).any()


def test_route_infinite_and_nan_logits():
    gate = G(16, 4, "sigmoid", 1, 1, "max", True)
    x = np.random.default_rng(8).standard_normal((3, 16))
    x[0, 3] = np.inf
    x[1, 3] = np.nan
    r = Run(gate, x)
    r.forward()
    idx, _ = r.check_forward()
    assert idx[0, 0] == 3 and 3 not in idx[1]
    # the softmax of such a row is not a number, and says so
    soft = G(16, 4, "softmax", 1, 1, "max", False)
    r = Run(soft, x)
    r.forward()
    assert r.idx[0, 0] == 3 and torch.isnan(r.w[1]).all() and torch.isfinite(r.w[2]).all()


def test_route_backward_takes_any_choice():
    """Slots that name no expert, or one named before, get no gradient and touch nothing."""
    for gate in (GATES["dsv3"], GATES["odd"], GATES["all_chosen"]):
        rng = np.random.default_rng(9)
        r = Run(gate, rng.standard_normal((21, gate.E)))
        idx = np.stack([rng.permutation(gate.E)[:gate.K] for _ in range(21)]).astype(np.int32)
        idx[:, 1] = idx[:, 0]
        idx[2:4, 0] = -1
        idx[5] = [gate.E, 2 ** 31 - 1, -2 ** 31, -5][:gate.K] + [gate.E + 1] * (gate.K - 4)
        clean = idx.copy()
        for row in clean:
            for k in range(gate.K):
                if not 0 <= row[k] < gate.E or row[k] in row[:k]:
                    row[k] = -1
        dw = rng.standard_normal((21, gate.K)).astype(np.float32)
        out = []
        for i in (idx, clean):
            mok.mok_route_bwd(desc(gate), r.x, torch.from_numpy(i).cuda(), torch.from_numpy(dw).cuda(),
                              r.dx[:21])
            out.append(r.dx.clone())
        assert torch.equal(out[0], out[1])
        ref = orr.backward(gate, r.x64, clean, dw)
        assert np.abs(out[0][:21].double().cpu().numpy() - ref).max() <= 1e-5 * np.abs(ref).max()


def test_route_gradient_against_differences():
    gate = GATES["dsv3"]
    rng = np.random.default_rng(10)
    x = rng.standard_normal((4, gate.E))
    r = Run(gate, x)
    r.forward()
    idx, _ = r.check_forward()
    dw = rng.standard_normal((4, gate.K)).astype(np.float32)
    mok.mok_route_bwd(desc(gate), r.x, r.idx[:4], torch.from_numpy(dw).cuda(), r.dx[:4])
    got, h = r.dx.double().cpu().numpy(), 2.0 ** -6
    for n in range(4):
        for k in range(gate.K):
            e = int(idx[n, k])
            loss = []
            for d in (h, -h):
                # the weights of the kernel itself, at logits moved by h (the choice stays: every other
                # expert is barred)
                y = np.full((1, gate.E), -np.inf)
                of = idx[n].astype(int)
                y[0, of] = r.x64[n, of]
                y[0, e] += d
                q = Run(gate, y)
                q.forward()
                at = {int(i): float(v) for i, v in zip(q.idx[0].cpu(), q.w[0].cpu())}
                loss.append(sum(float(dw[n, j]) * at[int(idx[n, j])] for j in range(gate.K)))
            d = (loss[0] - loss[1]) / (2 * h)
            # h^2 / 6 times a third derivative (below 6 scale max|dw|: products of q and sigmoid are below 1),
            # and the weights' rounding over h
            bound = h * h * gate.scale * np.abs(dw[n]).max() + gate.K * np.abs(dw[n]).max() * 2e-6 / h
            assert abs(d - got[n, e]) <= bound


def test_route_on_a_stream_and_in_a_graph():
    gate = GATES["dsv3"]
    rng = np.random.default_rng(11)
    r = Run(gate, rng.standard_normal((300, gate.E)), 0.1 * rng.standard_normal(gate.E))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r.forward(stream=s)
    s.synchronize()
    idx, _ = r.check_forward()
    graph = torch.cuda.CUDAGraph()
    dw = torch.randn(300, gate.K, device="cuda")
    with torch.cuda.graph(graph):
        r.forward()
        mok.mok_route_bwd(desc(gate), r.x, r.idx[:300], dw, r.dx[:300])
    for seed in range(4):
        x = np.random.default_rng(seed).standard_normal((300, gate.E))
        r.x.copy_(torch.from_numpy(x.astype(np.float32)))
        r.x64 = r.x.double().cpu().numpy()
        r.idx[:300], r.dx[:300] = -5, -5
        r.load[:gate.E] = 12345
        graph.replay()
        torch.cuda.synchronize()
        r.check_forward()
        got = [t.clone() for t in (r.idx, r.w, r.load, r.dx)]
        r.forward()
        mok.mok_route_bwd(desc(gate), r.x, r.idx[:300], dw, r.dx[:300])
        assert all(torch.equal(a, b) for a, b in zip(got, (r.idx, r.w, r.load, r.dx)))


@pytest.mark.parametrize("name", ["dsv3", "odd", "odd_groups"])
def test_route_rows_beyond_32_bits(name):
    """Rows so far apart that an element's number passes 2^32 (8.6 GB of bf16)."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    gate, far = GATES[name], 2 ** 31
    r = Run(gate, np.random.default_rng(12).standard_normal((3, gate.E)), None, None, "bfloat16")
    x = torch.empty(2 * far + gate.E, dtype=torch.bfloat16, device="cuda").as_strided((3, gate.E), (far, 1))
    x.copy_(r.x)
    r.x = x
    r.forward()
    idx, _ = r.check_forward()
    r.check_backward(idx)


def test_route_binding_refusals():
    gate = GATES["dsv3"]
    x = torch.zeros(4, 256, device="cuda")
    i = torch.zeros(4, 8, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 8, device="cuda")
    d = desc(gate)
    ok = dict(logits=x, topk_idx=i, topk_w=w)
    for bad in (dict(logits=x[:, :255]), dict(logits=x.half()), dict(logits=x.T.contiguous().T),
                dict(logits=x[:1].expand(4, 256)), dict(topk_idx=i.long()), dict(topk_idx=i[:3]),
                dict(topk_w=w.double()), dict(topk_w=w[:, :7]), dict(bias=x[0].double()),
                dict(bias=x[0, :255]), dict(token_mask=i[:, 0]), dict(token_mask=x[:3, 0].bool()),
                dict(load=w[0]), dict(topk_idx=i.cpu())):
        with pytest.raises(ValueError):
            mok.mok_route_fwd(d, **{**ok, **bad})
    for bad in (dict(dw=w.double()), dict(dlogits=x.bfloat16()), dict(dlogits=x[:, ::2])):
        with pytest.raises(ValueError):
            mok.mok_route_bwd(d, **{**dict(logits=x, topk_idx=i, dw=w, dlogits=x), **bad})
    with pytest.raises(mok.MokError):
        mok.mok_route_fwd(mok.route_desc(256, 8, groups=7), x, i, w)
