"""mok_route_fwd and mok_route_bwd in every layout of tokens, experts and choices that the calls pick
(lanes a token, experts a lane, length of the sorted lists), in every way of forming scores, against the
fp64 oracle. Tolerances are those of the gate's other tests, derived there."""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import route as orr

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

from tests.test_gpu_route import Run

# experts, choices, groups, groups that stay: the sizes at which layouts change, odd ones, groups of whole runs of 4
# experts and of others, as many groups as lanes, and more
SHAPES = [
    (64, 8, 8, 4), (65, 8, 1, 1), (100, 5, 1, 1), (128, 8, 8, 4), (129, 8, 1, 1), (180, 3, 5, 2), (256, 8, 8, 4),
    (256, 8, 16, 4), (257, 8, 1, 1), (384, 8, 8, 3), (384, 8, 12, 4), (385, 2, 1, 1), (400, 8, 10, 4), (512, 8, 16, 5),
    (513, 7, 1, 1), (640, 5, 20, 6), (1024, 8, 32, 4), (90, 11, 1, 1), (256, 16, 16, 6), (260, 9, 13, 5),
    (501, 16, 1, 1), (512, 16, 16, 7), (520, 10, 1, 1), (1024, 16, 32, 8), (1021, 16, 1, 1), (1023, 8, 33, 9)]
MODES = list(itertools.product(("sigmoid", "softmax"), ("max", "top2"), (False, True)))


@pytest.mark.parametrize("score,group_score,bias", MODES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_route_layouts(shape, score, group_score, bias):
    E, K, G, Kg = shape
    if G == 1 and group_score == "top2":
        group_score = "max"      # (with one group the plain weights, and bf16, where the others have fp32)
        renorm, dtype = False, "bfloat16"
    else:
        renorm, dtype = (E + K + bias) % 2 == 0, "bfloat16" if E % 3 == 0 else "float32"
    gate = orr.Gate(E, K, score, G, Kg, group_score, renorm, 2.5)
    rng = np.random.default_rng(E + 10 * K + G)
    n = 67
    x = rng.standard_normal((n, E)) * 1.5
    x[10:20] = 0.5 * rng.integers(-1, 2, (10, E))                                        # ties
    x[20:30] = np.where(rng.random((10, E)) < 0.5, 1.0, 0.25) + rng.integers(0, 5, (10, E)) * 2.0 ** -22
    x[30:40] = 14 + 2 * rng.random((10, E))                                              # scores near 1
    x[rng.random((n, E)) < 0.05] = -np.inf
    mask = rng.random(n) > 0.1
    x[~mask] = np.nan
    x[3], x[4], x[5], mask[3:7] = -np.inf, -np.inf, 0.25, True
    x[4, E - 1] = 0.5
    x[6] = -60 - rng.random(E)
    # (equal steps of a bias make sums of two keys equal that fp64 rounds apart)
    b = None if not bias else 0.02 * rng.integers(-9, 10, E) if group_score == "max" else 0.1 * rng.standard_normal(E)
    r = Run(gate, x, b, mask, dtype, pad=(0, 3, 4)[E % 3])
    r.forward()
    idx, _ = r.check_forward()
    r.check_backward(idx)
