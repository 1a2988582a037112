"""mok_route_fwd on rows whose softmax is not a number, in every form of the gate that scores take part in."""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import route as orr

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok


def forward(gate, x, bias=None, dtype=torch.float32):
    """(idx, w, load, logits in fp64 as the kernel sees them)"""
    d = mok.route_desc(gate.E, gate.K, gate.score, gate.groups, gate.top_groups, gate.group_score,
                       gate.renorm, gate.scale)
    x = torch.from_numpy(np.asarray(x, np.float32)).cuda().to(dtype)
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    idx = torch.full((len(x), gate.K), -77, dtype=torch.int32, device="cuda")
    w, load = torch.full((len(x), gate.K), -77.0, device="cuda"), torch.empty(gate.E, dtype=torch.int32, device="cuda")
    mok.mok_route_fwd(d, x, idx, w, bias=b, load=load)
    return idx.cpu().numpy(), w.double().cpu().numpy(), load.cpu().numpy(), x.double().cpu().numpy()


# whole runs of 4 experts (several tokens a wave), and 4 groups of 6 or 9 groups of 7 (one token a wave)
SHAPES = [(64, 4, 4, 2), (256, 8, 8, 4), (512, 6, 16, 3), (1024, 12, 32, 4), (24, 5, 4, 2), (63, 4, 9, 3)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("group_score,bias", [("top2", False), ("top2", True), ("max", True), ("max", False)])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_softmax_rows_without_scores(shape, group_score, bias, dtype):
    E, K, G, Kg = shape
    rng = np.random.default_rng(E)
    x = rng.standard_normal((40, E))
    x[3, 5], x[4, E - 1], x[5, 0] = np.nan, np.inf, -np.inf
    x[6, [1, E // 2]] = np.inf
    x[7, [1, E // 2]] = np.inf, np.nan
    x[8] = np.nan
    x[9] = -np.inf
    x[10] = -np.inf
    x[10, 7] = np.nan
    none = {8, 9, 10}
    if bias or group_score == "top2":
        none |= {3, 4, 6, 7}
    b = 0.125 * rng.integers(-2, 3, E) if bias else None
    for renorm in (True, False):
        gate = orr.Gate(E, K, "softmax", G, Kg, group_score, renorm)
        idx, w, load, x64 = forward(gate, x, b, dtype)
        with np.errstate(invalid="ignore"):
            ref = np.full((40, K), -1)
            for n in range(40):
                of = orr.choose_row(gate, x64[n], b)
                ref[n, :len(of)] = of
        assert np.array_equal(idx, ref)
        assert {n for n in range(40) if (idx[n] < 0).all()} == none
        assert np.array_equal(load, np.bincount(idx[idx >= 0], minlength=E))
        assert (w[idx < 0] == 0).all()
        for n in range(40):
            some = idx[n] >= 0
            if not some.any():
                continue
            bad = x64[n, idx[n][some]] if renorm else x64[n]
            assert np.isnan(w[n, some]).all() == bool((np.isnan(bad) | (bad == np.inf)).any()), n
            if not np.isnan(w[n, some]).any():
                of = [int(e) for e in idx[n][some]]
                # fp32: a few units of 2^-23 of logits below 5 and up to 1024 terms (their tree: 40)
                assert np.abs(w[n, some] / orr.weights_row(gate, x64[n], of) - 1).max() <= 2.0 ** -23 * 100
                assert (idx[n][some] // (E // G)).max() < G and len(set(idx[n][some] // (E // G))) <= Kg


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_sigmoid_rows_go_by_their_other_logits(shape, bias):
    """A sigmoid score of one expert does not depend on the others: NaN bars its own, +inf has the score 1."""
    E, K, G, Kg = shape
    rng = np.random.default_rng(E + 1)
    x = rng.standard_normal((8, E))
    x[0, 5], x[1, E - 1], x[2, [1, E // 2]] = np.nan, np.inf, np.inf
    x[3, ::3] = np.nan
    b = 0.125 * rng.integers(-2, 3, E) if bias else None
    for group_score, renorm in itertools.product(("max", "top2"), (True, False)):
        gate = orr.Gate(E, K, "sigmoid", G, Kg, group_score, renorm, 2.5)
        idx, w, load, x64 = forward(gate, x, b)
        ref, rw, rl = orr.forward(gate, x64, b)
        assert np.array_equal(idx, ref) and np.array_equal(load, rl)
        assert np.abs(w - rw).max() <= 2.0 ** -23 * 100
