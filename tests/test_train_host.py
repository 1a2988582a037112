"""Refusals of the routing and optimizer calls, all on the host before anything is launched: these
tests need no GPU (the pointers are never followed)."""
import ctypes
import math

import pytest

import combine_router_top_schedule_amd as mok

NULL, SHAPE, DTYPE, ALIGN = 1, 2, 3, 4
P = 4096   # a well-aligned address that no call below gets to use


def route(N=4, ld=None, E=16, K=2, score=1, G=4, Kg=2, gscore=1, renorm=1, elem=0, scale=1.0):
    return mok.MokRouteDesc(N, E if ld is None else ld, E, K, score, G, Kg, gscore, renorm, elem, scale)


@pytest.mark.parametrize("bad,code", [
    (dict(E=0, G=1), SHAPE), (dict(E=1028), SHAPE), (dict(K=0), SHAPE), (dict(K=17, E=64), SHAPE),
    (dict(K=9), SHAPE), (dict(G=3), SHAPE), (dict(G=0), SHAPE), (dict(G=128, E=256), SHAPE),
    (dict(Kg=0), SHAPE), (dict(Kg=5), SHAPE), (dict(score=2), SHAPE), (dict(gscore=-1), SHAPE),
    (dict(renorm=2), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE),
    (dict(scale=math.inf), SHAPE), (dict(scale=math.nan), SHAPE), (dict(ld=15), SHAPE),
    (dict(N=-1), SHAPE), (dict(N=1 << 31), SHAPE), (dict(elem=2), DTYPE)])
def test_route_descriptors(bad, code):
    d = ctypes.byref(route(**bad))
    assert mok.lib().mok_route_fwd(d, P, None, None, P, P, None, None) == code
    assert mok.lib().mok_route_bwd(d, P, P, P, P, None) == code


def test_route_pointers():
    L, d = mok.lib(), ctypes.byref(route())
    assert L.mok_route_fwd(None, P, None, None, P, P, None, None) == NULL
    for k in (0, 3, 4):
        args = [P, None, None, P, P, None]
        args[k] = None
        assert L.mok_route_fwd(d, *args, None) == NULL
        args[k] = P + 2
        assert L.mok_route_fwd(d, *args, None) == ALIGN
    assert L.mok_route_fwd(d, P, P + 1, None, P, P, None, None) == ALIGN
    assert L.mok_route_fwd(d, P, None, None, P, P, P + 2, None) == ALIGN
    for k in range(4):
        args = [P, P, P, P]
        args[k] = None
        assert L.mok_route_bwd(d, *args, None) == NULL
    assert L.mok_route_bwd(d, P, P, P, P + 8, None) == ALIGN
    assert L.mok_route_bwd(ctypes.byref(route(N=0)), None, None, None, None, None) == 0


def test_sumsq():
    L = mok.lib()
    n = ctypes.c_size_t()
    assert L.mok_sumsq_ws_size(1, ctypes.byref(n)) == 0 and n.value > 0
    assert L.mok_sumsq_ws_size(1, None) == NULL and L.mok_sumsq_ws_size(-1, ctypes.byref(n)) == SHAPE
    t = lambda g=P, k=5: (mok.MokSumsqTensor * 1)(mok.MokSumsqTensor(g, k))
    assert L.mok_grad_sumsq(-1, t(), 0, P, P, None) == SHAPE
    assert L.mok_grad_sumsq(1, t(), 2, P, P, None) == DTYPE
    assert L.mok_grad_sumsq(1, None, 0, P, P, None) == NULL
    assert L.mok_grad_sumsq(1, t(), 0, None, P, None) == NULL
    assert L.mok_grad_sumsq(1, t(), 0, P, None, None) == NULL
    assert L.mok_grad_sumsq(1, t(), 0, P + 4, P, None) == ALIGN
    assert L.mok_grad_sumsq(1, t(None), 0, P, P, None) == NULL
    assert L.mok_grad_sumsq(1, t(P + 8), 0, P, P, None) == ALIGN
    assert L.mok_grad_sumsq(1, t(P, -1), 0, P, P, None) == SHAPE
    assert L.mok_grad_sumsq(1, t(P, (1 << 33) + 1), 0, P, P, None) == SHAPE


def config(**kw):
    c = mok.MokAdamwConfig(1e-3, 0.9, 0.999, 1e-8, 0.1, 1.0, 1, 0, 0, 0, 0, None, None, None)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def tensor(**kw):
    t = mok.MokAdamwTensor(P, None, P, P, P, None, None, 5)
    for k, v in kw.items():
        setattr(t, k, v)
    return (mok.MokAdamwTensor * 1)(t)


@pytest.mark.parametrize("bad,code", [
    (dict(lr=-1.0), SHAPE), (dict(lr=math.nan), SHAPE), (dict(lr=math.inf), SHAPE),
    (dict(beta1=1.0), SHAPE), (dict(beta1=-0.1), SHAPE), (dict(beta2=1.0), SHAPE),
    (dict(beta2=math.nan), SHAPE), (dict(eps=0.0), SHAPE), (dict(eps=1e-60), SHAPE),
    (dict(eps=1e60), SHAPE), (dict(weight_decay=-1.0), SHAPE), (dict(step=0), SHAPE),
    (dict(grad_elem=3), DTYPE), (dict(param_elem=-1), DTYPE), (dict(state=2), DTYPE),
    (dict(sumsq_dev=P, max_norm=0.0), SHAPE), (dict(sumsq_dev=P, max_norm=math.nan), SHAPE),
    (dict(sumsq_dev=P + 4), ALIGN), (dict(lr_dev=P + 4), ALIGN), (dict(step_dev=P + 4), ALIGN)])
def test_adamw_configs(bad, code):
    assert mok.lib().mok_adamw(1, tensor(), ctypes.byref(config(**bad)), None) == code


@pytest.mark.parametrize("bad,kw,code", [
    (dict(n=-1), {}, SHAPE), (dict(n=(1 << 33) + 1), {}, SHAPE), (dict(p=None), {}, NULL),
    (dict(g=None), {}, NULL), (dict(m=None), {}, NULL), (dict(v=None), {}, NULL),
    (dict(p=P + 4), {}, ALIGN), (dict(g=P + 8), {}, ALIGN), (dict(copy=P + 2), {}, ALIGN),
    (dict(copy=P), dict(param_elem=1), DTYPE), ({}, dict(state=1), NULL),
    (dict(m_scale=P), dict(state=1), NULL)])
def test_adamw_tensors(bad, kw, code):
    assert mok.lib().mok_adamw(1, tensor(**bad), ctypes.byref(config(**kw)), None) == code


def test_adamw_counts():
    L, c = mok.lib(), ctypes.byref(config())
    assert L.mok_adamw(1, tensor(), None, None) == NULL
    assert L.mok_adamw(1, None, c, None) == NULL
    assert L.mok_adamw(-1, tensor(), c, None) == SHAPE
    # nothing to do is no error: no tensors, or only empty ones (whose pointers are not looked at)
    assert L.mok_adamw(0, None, c, None) == 0
    assert L.mok_adamw(1, tensor(n=0, p=None, g=None, m=None, v=None), c, None) == 0


def test_bindings_refuse_host_tensors_and_empty_lists():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 16)
    i, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    d = mok.route_desc(16, 2)
    with pytest.raises(ValueError):
        mok.mok_route_fwd(d, x, i, w)
    with pytest.raises(ValueError):
        mok.mok_route_bwd(d, x, i, w, x)
    with pytest.raises(ValueError):
        mok.adamw_plan([x], [x], [x], [x])
    with pytest.raises(ValueError):
        mok.sumsq_plan([])
    with pytest.raises(ValueError):
        mok.adamw_plan([], [], [], [])
    with pytest.raises(KeyError):
        mok.route_desc(16, 2, score="relu")
