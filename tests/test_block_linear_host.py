"""What MokBlockLinear and the binding of the weight gradient refuse or pass on, without a GPU: the calls of the library
are replaced by ones that note their arguments."""
import pytest

torch = pytest.importorskip("torch")

import combine_router_top_schedule_amd as mok
from combine_router_top_schedule_amd import block

R, N, K = 30, 70, 200
OFF = torch.zeros(4, dtype=torch.int32)


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("mok_block_quantize", "mok_block_quantize_weights", "mok_block_gemm", "mok_block_wgrad"):
        monkeypatch.setattr(block, name, lambda *a, _name=name, **kw: seen.append((_name, a, kw)))
    return seen


@pytest.mark.parametrize("train", [False, True])
def test_forward_refuses_other_shapes(calls, train):
    lin = block.MokBlockLinear(torch.zeros(3, N, K), R, train=train)
    del calls[:]
    # (250 and 129 columns round up to the same 256 as 200)
    for shape in ((R, 250), (R, 129), (R, K + 1), (R, 128), (R - 1, K), (R + 1, K), (K,), (1, R, K)):
        with pytest.raises(ValueError):
            lin.forward(torch.zeros(shape), torch.zeros(R, N), offsets=OFF)
    for shape in ((R, N + 1), (R + 1, N), (R, 128), (N,)):
        with pytest.raises(ValueError):
            lin.forward(torch.zeros(R, K), torch.zeros(shape), offsets=OFF)
    for off in (None, OFF[:3], torch.zeros(5, dtype=torch.int32), OFF.view(2, 2)):
        with pytest.raises(ValueError):
            lin.forward(torch.zeros(R, K), torch.zeros(R, N), offsets=off)
    assert not calls   # nothing of a refused call is enqueued
    lin.forward(torch.zeros(R, K), torch.zeros(R, N), offsets=OFF)
    assert [c[0] for c in calls] == ["mok_block_quantize", "mok_block_gemm"]


def test_backward_refuses_other_shapes(calls):
    lin = block.MokBlockLinear(torch.zeros(3, N, K), R)
    del calls[:]
    dy, dx, dw = torch.zeros(R, N), torch.zeros(R, K), torch.zeros(3, N, K)
    for shape in ((R, 71), (R, 128), (R, 1), (R - 1, N), (R + 1, N), (N,)):
        for a, b in ((dx, None), (None, dw), (dx, dw)):
            with pytest.raises(ValueError):
                lin.backward(torch.zeros(shape), a, b, offsets=OFF)
    for a, b in ((torch.zeros(R, K + 1), None), (torch.zeros(R + 1, K), dw), (dx, torch.zeros(3, N, K + 1)),
                 (None, torch.zeros(2, N, K)), (None, torch.zeros(N, K))):
        with pytest.raises(ValueError):
            lin.backward(dy, a, b, offsets=OFF)
    for off in (None, OFF[:3]):
        with pytest.raises(ValueError):
            lin.backward(dy, dx, dw, offsets=off)
    assert not calls
    lin.backward(dy, dx, dw, offsets=OFF)
    assert [c[0] for c in calls] == ["mok_block_quantize", "mok_block_gemm", "mok_block_wgrad"]


def test_one_group_needs_no_offsets(calls):
    lin = block.MokBlockLinear(torch.zeros(1, N, K), R)
    lin.forward(torch.zeros(R, K), torch.zeros(R, N))
    lin.backward(torch.zeros(R, N), torch.zeros(R, K), torch.zeros(1, N, K), offsets=OFF[:2])


def test_weights_have_three_dimensions(calls):
    for shape in ((N, K), (1, 2, N, K)):
        with pytest.raises(ValueError):
            block.MokBlockLinear(torch.zeros(shape), R)
