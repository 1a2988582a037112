"""Pins of the oracles of block-scaled FP8 and Muon."""
import numpy as np
import pytest

from oracle import block as ob
from oracle import muon as om
from oracle.mx import e4m3_decode

F = np.float32


def test_blocks_by_hand():
    x = np.zeros((2, 130), F)
    x[0, :3] = 448, -1, 0.4375
    x[0, 128:] = 2, -1
    c, s = ob.quantize_rows(x)
    assert c.shape == (2, 256) and s.shape == (2, 2)
    assert s[0, 0] == 1 and s[1, 0] == F(2) / F(448) and s[0, 1] == F(2.0 ** -100) / F(448)
    assert e4m3_decode(c[0, :3]).tolist() == [448, -1, 0.4375]
    assert e4m3_decode(c[0, 128:130]).tolist() == [448, -224] and not c[0, 130:].any() and not c[1].any()


def test_not_finite():
    x = np.ones((1, 128), F)
    x[0, 5] = np.nan
    c, s = ob.quantize_rows(x)
    assert c[0, 5] == 0x7F and s[0, 0] == F(1) / F(448) and (e4m3_decode(np.delete(c[0], 5)) == 448).all()
    x[0, 5] = np.inf
    c, s = ob.quantize_rows(x)
    assert c[0, 5] == 0x7F and np.isinf(s[0, 0]) and not np.delete(c[0], 5).any()
    assert np.isnan(ob.values_rows(c, s)).all()


@pytest.mark.parametrize("shape", [(1, 1), (3, 128), (130, 257)])
def test_error_and_transposes(shape):
    rng = np.random.default_rng(0)
    x = rng.standard_normal(shape).astype(F)
    c, s = ob.quantize_rows(x)
    v = ob.values_rows(c, s)
    assert not v[:, shape[1]:].any()
    # half a step of E4M3 (2^-4 of a normal value, 2^-10 of the scale below 2^-6 of it), and fp32's
    assert (np.abs(v[:, :shape[1]] - x) <= np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(s.T, 128, 1)[:, :shape[1]] * 2.0 ** -10) * (1 + 2.0 ** -20)).all()
    w = rng.standard_normal((2,) + shape).astype(F)
    (a, sa), (b, sb) = ob.quantize_weights(w), ob.quantize_weights(w.transpose(0, 2, 1))
    assert (ob.values_weights(a, sa)[:, :, :shape[1]] == ob.values_weights(b, sb)[:, :, :shape[0]].transpose(0, 2, 1)).all()


def test_offsets_and_columns():
    assert ob.clean([-3, 5, 2, 99], 10).tolist() == [0, 5, 5, 10]
    assert ob.columns([0, 5, 5, 134]) == [0, 128, 128, 384]
    assert ob.padded_rows(0, 1) == 0 and ob.padded_rows(1, 1) == 128 and ob.padded_rows(128, 1) == 128
    for off in ([0, 1, 2, 3], [0, 128, 256, 400], [0, 0, 0, 129]):
        assert ob.columns(off)[-1] <= ob.padded_rows(off[-1], 3)


def test_gradients_against_differences():
    """dx by the transposed weights and dw by columns are the derivatives of sum(dy out)."""
    rng = np.random.default_rng(1)
    R, N, K, off = 9, 5, 4, [1, 4, 4, 9]
    x, w, dy = rng.standard_normal((R, K)), rng.standard_normal((3, N, K)), rng.standard_normal((R, N))

    def loss(x, w):
        return sum((dy[a:b] * (x[a:b] @ w[g].T)).sum() for g, (a, b) in enumerate(zip(off, off[1:])))

    # the oracle's products of values that E4M3 holds: scales of one
    grid = lambda v: e4m3_decode(ob._encode(v.astype(F)))
    x, w, dy = grid(x), grid(w), grid(dy)
    pad = lambda v, k: np.pad(v, [(0, 0)] * (v.ndim - 1) + [(0, 128 - k)])
    ones = np.ones
    dx = np.zeros((R, K))
    ob.gemm(ob._encode(pad(dy, N).astype(F)), ones((1, R)), ob._encode(pad(w.transpose(0, 2, 1), N).astype(F)), ones((3, 1, 1)), off, dx)
    dw = np.zeros((3, N, K))
    P = ob.padded_rows(R, 3)
    cols = []
    for v in (dy, x):
        c = np.zeros((v.shape[1], P), np.uint8)
        for g, at in zip(range(3), ob.columns(off)):
            c[:, at:at + off[g + 1] - off[g]] = ob._encode(v[off[g]:off[g + 1]].T.astype(F))
        cols.append(c)
    ob.wgrad(cols[0], ones((P // 128, N)), cols[1], ones((P // 128, K)), off, dw)
    for got, at in ((dx, x), (dw, w)):
        for i in np.ndindex(at.shape):
            keep = at[i]
            at[i] = keep + 0.5
            hi = loss(x, w)
            at[i] = keep - 0.5
            lo = loss(x, w)
            at[i] = keep
            assert abs(hi - lo - got[i]) < 1e-12


def test_orthogonalize():
    rng = np.random.default_rng(2)
    q = np.linalg.qr(rng.standard_normal((6, 6)))[0][:4]
    s = np.array([0.9, 0.5, 0.3, 0.05])
    u = (np.linalg.qr(rng.standard_normal((4, 4)))[0] * s) @ q
    x = om.orthogonalize(u, eps=1e-30)
    t = s / np.linalg.norm(s)
    for _ in range(5):
        t = 3.4445 * t - 4.7750 * t ** 3 + 2.0315 * t ** 5
    assert np.allclose(np.linalg.svd(x, compute_uv=False), np.sort(t)[::-1], atol=1e-12)
    assert np.allclose(om.orthogonalize(u.T), om.orthogonalize(u).T)
    assert not om.orthogonalize(np.zeros((3, 2))).any()
    assert np.allclose(om.orthogonalize([[2.0]], steps=1, coefficients=[(1.5, -0.5, 0.0)]), 1.0)


@pytest.mark.parametrize("small", [False, True])
def test_rounded_is_near(small):
    """Random matrices: some 2^-9 of the result."""
    rng = np.random.default_rng(3)
    for shape in ((7, 40), (64, 33), (1, 9)):
        u = rng.standard_normal(shape)
        x = om.orthogonalize(u)
        assert np.linalg.norm(om.rounded(u, small=small) - x) < 2.0 ** -7 * np.linalg.norm(x)


def test_step():
    p, g, m = np.array([[1.0, 2.0]]), np.array([[0.3, 0.4]]), np.array([[0.0, 0.0]])
    q, m1, u = om.step(p, g, m, lr=0.1, momentum=0.5, weight_decay=0.2, adjust="none", steps=1, coefficients=[(1, 0, 0)])
    assert np.allclose(m1, g) and np.allclose(u, 1.5 * g)
    assert np.allclose(q, p * 0.98 - 0.1 * np.array([[0.6, 0.8]]))
    q2, m2, _ = om.step(p, g, m, lr=0.1, norm=0.5, max_norm=0.25)
    assert np.allclose(m2, g / 2)
