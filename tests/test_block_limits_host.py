"""The most blocks of 128 x 128 that a block-scaled FP8 call takes, as include/mok.h states them: one more is refused, without
a GPU (the pointers are never followed), and mok_block_gemm_kernel knows the limit of products on both sides."""
import ctypes

import pytest

import combine_router_top_schedule_amd as mok

SHAPE, P = 2, 4096


def desc(rows, groups, n, k):
    return ctypes.byref(mok.MokBlockDesc(rows, max(n, k), groups, n, k, 0))


def blocks(n):
    return -(-n // 128)


# (rows, groups, n): of (rows / 128 + groups) blocks(n) the first at 2^22 and above
@pytest.mark.parametrize("rows,groups,n", [(1 << 22, 1, 1 << 17), ((1 << 22) - 128, 1, 128 * 128), (0, 1024, (1 << 19) - 127),
                                           (1 << 27, 4, 512), ((1 << 27) - 512, 4, 4 * 128)])
def test_products(rows, groups, n):
    least = -(-(1 << 22) // (rows // 128 + groups))   # blocks of n that are refused
    if least > 8192:
        pytest.skip("no width goes so far")
    L = mok.lib()
    over, under = max(n, 128 * (least - 1) + 1), 128 * (least - 1)
    assert (rows // 128 + groups) * blocks(over) >= 1 << 22 > (rows // 128 + groups) * blocks(under)
    assert L.mok_block_gemm_kernel(desc(rows, groups, over, 128)) == -1
    if rows:
        assert L.mok_block_gemm(desc(rows, groups, over, 128), P, P, P, P, P, P, None) == SHAPE
    assert under == 0 or L.mok_block_gemm_kernel(desc(rows, groups, under, 128)) >= 0


def test_column_codes():
    L = mok.lib()
    for rows, groups in ((1 << 22, 1), (1 << 20, 3), (1000, 1024)):
        k = 128 * (((1 << 22) - 1) // (rows // 128 + groups + 2)) + 1
        if k <= 1 << 20:
            assert L.mok_block_quantize(desc(rows, groups, 1, k), P, P, None, None, P, P, None) == SHAPE


def test_weights_and_their_gradient():
    L = mok.lib()
    for groups, n, k in ((4, 1 << 17, 1 << 17), (1024, 8192, 8192), (1, 1 << 18, (1 << 18) - 127)):
        assert groups * blocks(n) * blocks(k) >= 1 << 22
        assert L.mok_block_wgrad(desc(128, groups, n, k), P, P, P, P, P, P, 0, None) == SHAPE
    for groups, n, k in ((8, 1 << 17, 1 << 17), (1024, 8192, 16384), (2, 1 << 18, (1 << 18) - 127)):
        assert groups * blocks(n) * blocks(k) >= 1 << 23
        assert L.mok_block_quantize_weights(desc(0, groups, n, k), P, P, P, None, None, None) == SHAPE
