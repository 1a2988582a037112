"""The choice of mok_block_gemm's kernel, which is a matter of sizes alone and needs no GPU."""
import ctypes

import pytest

import combine_router_top_schedule_amd as mok


def kernel(rows, groups, n, k, elem=mok.MOK_ELEM_BF16, stride=0):
    return mok.lib().mok_block_gemm_kernel(ctypes.byref(mok.MokBlockDesc(rows, stride, groups, n, k, elem)))


def test_choice():
    few, mid, wide = mok.MOK_BLOCK_FEW_ROWS, mok.MOK_BLOCK_TILES_128, mok.MOK_BLOCK_TILES_256
    assert kernel(1, 1, 4096, 7168) == few and kernel(44, 6, 7168, 2048) == few
    assert kernel(16384, 4, 4096, 7168) == wide
    assert kernel(16384, 4, 4096, 7168, mok.MOK_ELEM_F32) == mid   # (fp32 results have no larger tiles)
    assert kernel(3000, 6, 7168, 2048) == mid
    assert kernel(5003, 7, 1001, 1416, mok.MOK_ELEM_F32) == mid
    assert kernel(0, 3, 16, 128) in (few, mid, wide)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=(1 << 27) + 1), dict(groups=0), dict(groups=1025), dict(n=0), dict(n=(1 << 20) + 1),
                                 dict(k=0), dict(k=(1 << 20) + 1), dict(elem=2), dict(elem=-1)])
def test_out_of_range(bad):
    assert kernel(**{**dict(rows=4, groups=2, n=16, k=128), **bad}) == -1
    assert mok.lib().mok_block_gemm_kernel(None) == -1
