"""Errors of the library that the block-scaled FP8 binding passes on: outputs left out, buffers that begin at no multiple of
16 bytes, sizes beyond the limits. The library refuses them before it launches anything, so they are made with host tensors
here, and with device tensors where there is a GPU."""
import pytest

torch = pytest.importorskip("torch")

import combine_router_top_schedule_amd as mok

NULL, SHAPE, ALIGN = 1, 2, 4
R, N, K, G = 4, 6, 200, 2


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def dev(request, monkeypatch):
    if request.param == "cuda" and not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    if request.param == "cpu":
        def launch(fn, dev, stream, *args):
            code = getattr(mok.lib(), fn)(*args, None)
            if code:
                raise mok.MokError(fn, code)
        monkeypatch.setattr(mok, "_device_of", lambda t: t.get_device())
        monkeypatch.setattr(mok, "_launch", launch)
    return request.param


def codes(dev, *shape, off=0):
    """uint8 zeros, `off` bytes behind a multiple of 16."""
    n = torch.Size(shape).numel()
    return torch.zeros(n + 16, dtype=torch.uint8, device=dev)[off:off + n].view(shape)


def refused(code, f):
    with pytest.raises(mok.MokError) as e:
        f()
    assert e.value.code == code


@pytest.mark.parametrize("off", [1, 4, 8, 15])
def test_codes_off_16_bytes(dev, off):
    f32 = lambda *s: torch.zeros(*s, device=dev)
    o = torch.zeros(G + 1, dtype=torch.int32, device=dev)
    P = mok.block_padded_rows(R, G)
    x, w, out, dw = f32(R, K), f32(G, N, K), f32(R, N), f32(G, N, K)
    s, st, ws, wst = f32(2, R), f32(P // 128, K), f32(G, 1, 2), f32(G, 2, 1)
    refused(ALIGN, lambda: mok.mok_block_quantize(x, codes(dev, R, 256, off=off), s, offsets=o))
    refused(ALIGN, lambda: mok.mok_block_quantize(x, codes_t=codes(dev, K, P, off=off), scales_t=st, offsets=o))
    refused(ALIGN, lambda: mok.mok_block_quantize(x, codes(dev, R, 256), s, codes(dev, K, P, off=off), st, offsets=o))
    refused(ALIGN, lambda: mok.mok_block_quantize_weights(w, codes(dev, G, N, 256, off=off), ws))
    refused(ALIGN, lambda: mok.mok_block_quantize_weights(w, codes(dev, G, N, 256), ws, codes(dev, G, K, 128, off=off), wst))
    refused(ALIGN, lambda: mok.mok_block_gemm(codes(dev, R, 256, off=off), s, codes(dev, G, N, 256), ws, out, offsets=o))
    refused(ALIGN, lambda: mok.mok_block_gemm(codes(dev, R, 256), s, codes(dev, G, N, 256, off=off), ws, out, offsets=o))
    yt, yts, xt = codes(dev, N, P), f32(P // 128, N), codes(dev, K, P)
    refused(ALIGN, lambda: mok.mok_block_wgrad(codes(dev, N, P, off=off), yts, xt, st, dw, offsets=o, rows=R))
    refused(ALIGN, lambda: mok.mok_block_wgrad(yt, yts, codes(dev, K, P, off=off), st, dw, offsets=o, rows=R))


def test_nothing_to_write(dev):
    refused(NULL, lambda: mok.mok_block_quantize(torch.zeros(R, K, device=dev)))
    refused(NULL, lambda: mok.mok_block_quantize(torch.zeros(R, K, device=dev), offsets=torch.zeros(3, dtype=torch.int32, device=dev)))


def test_sizes_beyond_the_limits(dev):
    f32 = lambda *s: torch.zeros(*s, device=dev)
    refused(SHAPE, lambda: mok.mok_block_quantize(f32(R, 0), codes(dev, R, 0), f32(0, R)))
    refused(SHAPE, lambda: mok.mok_block_quantize_weights(f32(1, 0, 128), codes(dev, 1, 0, 128), f32(1, 0, 1)))
    refused(SHAPE, lambda: mok.mok_block_gemm(codes(dev, R, 128), f32(1, R), codes(dev, 1, 0, 128), f32(1, 0, 1), f32(R, 0)))
    wide = (1 << 20) + 1
    refused(SHAPE, lambda: mok.mok_block_quantize(f32(1, wide), codes(dev, 1, wide + 127), f32((wide + 127) // 128, 1)))
    o = torch.zeros(1026, dtype=torch.int32, device=dev)
    refused(SHAPE, lambda: mok.mok_block_quantize(f32(R, K), codes(dev, R, 256), f32(2, R), offsets=o))
