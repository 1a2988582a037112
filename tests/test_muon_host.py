"""Refusals of the Muon calls, all on the host before anything is launched: these tests need no GPU (the
pointers are never followed)."""
import ctypes
import math

import pytest

import combine_router_top_schedule_amd as mok

NULL, SHAPE, DTYPE, ALIGN = 1, 2, 3, 4
P = 4096   # a well-aligned address that no call below gets to use


def tensor(p=P, copy=P, g=P, m=P, batch=2, rows=3, cols=4):
    return (mok.MokMuonTensor * 1)(mok.MokMuonTensor(p, copy, g, m, batch, rows, cols))


def config(**kw):
    ns = mok._newton_schulz(kw.pop("eps", 1e-7), 5, mok.NEWTON_SCHULZ)
    ns.steps = kw.pop("steps", 5)
    if "coefficient" in kw:
        ns.coefficients[4] = kw.pop("coefficient")
    return ctypes.byref(mok.MokMuonConfig(**{**dict(lr=1e-3, momentum=0.9, max_norm=math.inf, nesterov=1, ns=ns), **kw}))


@pytest.mark.parametrize("bad,code", [
    (dict(lr=-1.0), SHAPE), (dict(lr=math.nan), SHAPE), (dict(lr=math.inf), SHAPE), (dict(momentum=1.0), SHAPE),
    (dict(momentum=-0.1), SHAPE), (dict(momentum=math.nan), SHAPE), (dict(weight_decay=-1.0), SHAPE),
    (dict(weight_decay=math.nan), SHAPE), (dict(nesterov=2), SHAPE), (dict(adjust=3), SHAPE), (dict(adjust=-1), SHAPE),
    (dict(grad_elem=2), DTYPE), (dict(eps=0.0), SHAPE), (dict(eps=math.nan), SHAPE), (dict(eps=1e-60), SHAPE),
    (dict(steps=0), SHAPE), (dict(steps=17), SHAPE), (dict(coefficient=math.inf), SHAPE),
    (dict(sumsq_dev=P, max_norm=0.0), SHAPE), (dict(sumsq_dev=P, max_norm=math.nan), SHAPE),
    (dict(sumsq_dev=P + 4), ALIGN), (dict(lr_dev=P + 4), ALIGN)])
def test_config(bad, code):
    assert mok.lib().mok_muon(1, tensor(), config(**bad), P, None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(batch=-1), SHAPE), (dict(batch=(1 << 20) + 1), SHAPE), (dict(rows=0), SHAPE), (dict(cols=0), SHAPE),
    (dict(rows=(1 << 16) + 1), SHAPE), (dict(cols=(1 << 16) + 1), SHAPE),
    (dict(batch=3, rows=1 << 16, cols=1 << 16), SHAPE), (dict(p=None), NULL), (dict(g=None), NULL), (dict(m=None), NULL),
    (dict(p=P + 8), ALIGN), (dict(copy=P + 8), ALIGN), (dict(g=P + 8), ALIGN), (dict(m=P + 8), ALIGN)])
def test_tensors(bad, code):
    L, n = mok.lib(), ctypes.c_size_t()
    assert L.mok_muon(1, tensor(**bad), config(), P, None) == code
    if code == SHAPE:
        assert L.mok_muon_ws_size(1, tensor(**bad), ctypes.byref(n)) == SHAPE


def test_pointers():
    L, n = mok.lib(), ctypes.c_size_t()
    assert L.mok_muon(1, tensor(), None, P, None) == NULL
    assert L.mok_muon(-1, tensor(), config(), P, None) == SHAPE
    assert L.mok_muon(1, None, config(), P, None) == NULL
    assert L.mok_muon(1, tensor(), config(), None, None) == NULL
    assert L.mok_muon(1, tensor(), config(), P + 128, None) == ALIGN
    assert L.mok_muon_ws_size(1, tensor(), None) == NULL and L.mok_muon_ws_size(-1, tensor(), ctypes.byref(n)) == SHAPE
    assert L.mok_muon_ws_size(1, None, ctypes.byref(n)) == NULL
    assert L.mok_muon_ws_size(1, tensor(rows=500, cols=700), ctypes.byref(n)) == 0 and n.value > 2 * 500 * 700 * 7


def test_workspace_is_bounded():
    """Many matrices go through in runs of at most 2 GiB; one alone may need more."""
    L, n = mok.lib(), ctypes.c_size_t()
    assert L.mok_muon_ws_size(1, tensor(batch=1000, rows=2048, cols=2048), ctypes.byref(n)) == 0
    assert (1 << 30) < n.value <= (2 << 30)
    assert L.mok_muon_ws_size(1, tensor(batch=2, rows=1 << 15, cols=1 << 15), ctypes.byref(n)) == 0
    assert 7 << 30 < n.value < 16 << 30


def test_orthogonalize():
    L, n, ns = mok.lib(), ctypes.c_size_t(), mok._newton_schulz(1e-7, 5, mok.NEWTON_SCHULZ)
    t = lambda src=P, out=P, batch=1, rows=3, cols=4: (mok.MokOrthogonalizeTensor * 1)(
        mok.MokOrthogonalizeTensor(src, out, batch, rows, cols))
    call = lambda k=1, x=t(), elem=0, c=ctypes.byref(ns), ws=P: L.mok_orthogonalize(k, x, elem, c, ws, None)
    assert call(c=None) == NULL and call(k=-1) == SHAPE and call(x=None) == NULL and call(ws=None) == NULL
    assert call(elem=5) == DTYPE and call(ws=P + 16) == ALIGN
    assert call(x=t(src=None)) == NULL and call(x=t(out=None)) == NULL
    assert call(x=t(src=P + 4)) == ALIGN and call(x=t(out=P + 4)) == ALIGN and call(x=t(rows=0)) == SHAPE
    bad = mok._newton_schulz(1e-7, 5, mok.NEWTON_SCHULZ)
    bad.steps = 0
    assert call(c=ctypes.byref(bad)) == SHAPE
    assert L.mok_orthogonalize_ws_size(1, t(), ctypes.byref(n)) == 0 and n.value >= 256
    assert L.mok_orthogonalize_ws_size(1, t(cols=0), ctypes.byref(n)) == SHAPE
    assert L.mok_orthogonalize_ws_size(1, t(), None) == NULL


def test_coefficients():
    assert list(mok._newton_schulz(1e-7, 2, [(1, 2, 3), (4, 5, 6)]).coefficients[:6]) == [1, 2, 3, 4, 5, 6]
    assert list(mok._newton_schulz(1e-7, 2, (1, 2, 3)).coefficients[:6]) == [1, 2, 3, 1, 2, 3]
    for steps, c in ((2, [(1, 2, 3)]), (1, [(1, 2)]), (0, (1, 2, 3)), (17, (1, 2, 3))):
        with pytest.raises(ValueError):
            mok._newton_schulz(1e-7, steps, c)


def test_plans_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    z = torch.zeros(2, 3)
    for f in (lambda: mok.muon_plan([z], [z], [z]), lambda: mok.orthogonalize_plan([z], [z]), lambda: mok.muon_plan([], [], []),
              lambda: mok.orthogonalize_plan([], [])):
        with pytest.raises(ValueError):
            f()
