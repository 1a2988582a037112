"""Refusals of the block-scaled FP8 calls, all on the host before anything is launched: these tests need no
GPU (the pointers are never followed)."""
import ctypes

import pytest

import combine_router_top_schedule_amd as mok

NULL, SHAPE, DTYPE, ALIGN = 1, 2, 3, 4
P = 4096   # a well-aligned address that no call below gets to use


def desc(rows=4, stride=None, groups=2, n=16, k=24, elem=0, of="k"):
    return mok.MokBlockDesc(rows, (k if of == "k" else n) if stride is None else stride, groups, n, k, elem)


BAD = [(dict(rows=-1), SHAPE), (dict(rows=(1 << 27) + 1), SHAPE), (dict(groups=0), SHAPE), (dict(groups=1025), SHAPE),
       (dict(k=0), SHAPE), (dict(k=(1 << 20) + 1), SHAPE)]


@pytest.mark.parametrize("bad,code", BAD + [(dict(stride=23), SHAPE), (dict(elem=2), DTYPE),
                                            (dict(rows=(1 << 22) + 1), SHAPE)])
def test_quantize_descriptors(bad, code):
    assert mok.lib().mok_block_quantize(ctypes.byref(desc(**bad)), P, P, P, P, P, P, None) == code


def test_quantize_pointers():
    L, d = mok.lib(), ctypes.byref(desc())
    assert L.mok_block_quantize(None, P, P, P, P, P, P, None) == NULL
    for x, off, c, s, ct, st in ((None, P, P, P, P, P), (P, None, P, P, P, P), (P, P, None, P, P, P), (P, P, P, None, P, P),
                                 (P, P, P, P, None, P), (P, P, P, P, P, None), (P, P, None, None, None, None)):
        assert L.mok_block_quantize(d, x, off, c, s, ct, st, None) == NULL
    for i, by in ((0, 2), (1, 2), (2, 8), (3, 2), (4, 8), (5, 2)):
        args = [P] * 6
        args[i] += by
        assert L.mok_block_quantize(d, *args, None) == ALIGN
    assert L.mok_block_quantize(ctypes.byref(desc(rows=0)), None, P, None, None, None, None, None) == 0


@pytest.mark.parametrize("bad,code", [(dict(groups=0), SHAPE), (dict(groups=1025), SHAPE), (dict(n=0), SHAPE),
                                      (dict(n=(1 << 20) + 1), SHAPE), (dict(k=0), SHAPE), (dict(elem=7), DTYPE),
                                      (dict(groups=1024, n=1 << 20, k=1 << 20), SHAPE)])
def test_weights_descriptors(bad, code):
    assert mok.lib().mok_block_quantize_weights(ctypes.byref(desc(**bad)), P, P, P, P, P, None) == code


def test_weights_pointers():
    L, d = mok.lib(), ctypes.byref(desc())
    assert L.mok_block_quantize_weights(None, P, P, P, P, P, None) == NULL
    for i in range(5):
        args = [P] * 5
        args[i] = None
        assert L.mok_block_quantize_weights(d, *args, None) == NULL
    for i, by in ((0, 2), (1, 8), (2, 2), (3, 8), (4, 2)):
        args = [P] * 5
        args[i] += by
        assert L.mok_block_quantize_weights(d, *args, None) == ALIGN


@pytest.mark.parametrize("bad,code", BAD + [(dict(n=0), SHAPE), (dict(n=(1 << 20) + 1), SHAPE), (dict(stride=15), SHAPE),
                                            (dict(elem=-1), DTYPE), (dict(rows=1 << 27, n=1 << 20), SHAPE)])
def test_gemm_descriptors(bad, code):
    assert mok.lib().mok_block_gemm(ctypes.byref(desc(of="n", **bad)), P, P, P, P, P, P, None) == code


def test_gemm_pointers():
    L, d = mok.lib(), ctypes.byref(desc(of="n"))
    assert L.mok_block_gemm(None, P, P, P, P, P, P, None) == NULL
    for i in range(6):
        args = [P] * 6
        args[i] = None
        assert L.mok_block_gemm(d, *args, None) == NULL
    for i, by in ((0, 8), (1, 2), (2, 8), (3, 2), (4, 2), (5, 2)):
        args = [P] * 6
        args[i] += by
        assert L.mok_block_gemm(d, *args, None) == ALIGN
    assert L.mok_block_gemm(ctypes.byref(desc(rows=0, of="n")), None, None, None, None, P, None, None) == 0


@pytest.mark.parametrize("bad,code", BAD + [(dict(n=0), SHAPE), (dict(rows=(1 << 22) + 1), SHAPE)])
def test_wgrad_descriptors(bad, code):
    assert mok.lib().mok_block_wgrad(ctypes.byref(desc(**bad)), P, P, P, P, P, P, 0, None) == code


def test_wgrad_pointers():
    L, d = mok.lib(), ctypes.byref(desc())
    assert L.mok_block_wgrad(None, P, P, P, P, P, P, 0, None) == NULL
    assert L.mok_block_wgrad(d, P, P, P, P, P, P, 2, None) == SHAPE
    for i in range(6):
        args = [P] * 6
        args[i] = None
        assert L.mok_block_wgrad(d, *args, 0, None) == NULL
    for i, by in ((0, 8), (1, 2), (2, 8), (3, 2), (4, 2), (5, 2)):
        args = [P] * 6
        args[i] += by
        assert L.mok_block_wgrad(d, *args, 0, None) == ALIGN


def test_padded_rows():
    assert [mok.block_padded_rows(*a) for a in ((0, 1), (1, 1), (128, 1), (129, 1), (3, 3), (1000, 4))] == [
        0, 128, 128, 256, 384, 1408]
    for bad in ((-1, 1), (1, 0), (1, 1025), ((1 << 27) + 1, 1)):
        with pytest.raises(ValueError):
            mok.block_padded_rows(*bad)


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        mok.mok_block_quantize(torch.zeros(2, 128))
    with pytest.raises(ValueError):
        mok.mok_block_quantize_weights(torch.zeros(1, 2, 128), None, None)
