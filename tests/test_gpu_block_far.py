"""Block-scaled FP8 at the ends of its ranges: widths of 2^20, rows so far apart that their offsets pass 32 bits, 1,024
groups. Operands of products are codes of -1, 0 and 1 with scales that are powers of two, so that sums are exact and
results are compared for equality, on the GPU as they are large."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok

BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def up(n):
    return -(-n // 128) * 128


def small(g, *shape):
    """-1, 0 and 1."""
    return torch.randint(-1, 2, shape, device="cuda", generator=g).float()


def codes(v):
    """E4M3 codes of -1, 0 and 1, padded to whole blocks along the last axis."""
    return torch.nn.functional.pad(v, (0, up(v.shape[-1]) - v.shape[-1])).to(E4M3).view(torch.uint8).contiguous()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def kernel(rows, groups, n, k, dtype):
    elem = mok.MOK_ELEM_BF16 if dtype is BF else mok.MOK_ELEM_F32
    return mok.lib().mok_block_gemm_kernel(ctypes.byref(mok.MokBlockDesc(rows, n, groups, n, up(k), elem)))


@pytest.mark.parametrize("rows,n,k,dtype", [(3, 20, 1 << 20, torch.float32), (3, 1 << 20, 100, BF), (700, 300, 200_000, torch.float32),
                                            (2100, 2100, 70_000, BF), (40, 1 << 20, 130, torch.float32), (300, 1 << 19, 130, BF)])
def test_gemm_of_wide_operands(rows, n, k, dtype):
    """Sums of up to 2^20 terms of -1, 0 and 1 stay below 2^24: exact in fp32, rounded once to bf16."""
    g = gen(1)
    x, w = small(g, rows, k), small(g, 1, n, k)
    xs, ws = torch.ones(up(k) // 128, rows, device="cuda"), torch.full((1, up(n) // 128, up(k) // 128), 0.5, device="cuda")
    out = torch.full((rows, n), -7.0, dtype=dtype, device="cuda")
    mok.mok_block_gemm(codes(x), xs, codes(w), ws, out)
    assert torch.equal(out, ((x @ w[0].t()) * 0.5).to(dtype))


def test_every_kernel_is_among_the_wide_ones():
    kinds = {kernel(r, 1, n, k, t) for r, n, k, t in ((3, 20, 1 << 20, torch.float32), (700, 300, 200_000, torch.float32), (2100, 2100, 70_000, BF),
                                                      (300, 1 << 19, 130, BF), (7000, 2100, 1000, BF))}
    assert kinds == {mok.MOK_BLOCK_FEW_ROWS, mok.MOK_BLOCK_TILES_128, mok.MOK_BLOCK_TILES_256}


@pytest.mark.parametrize("rows,n,k", [(130, 130, 1 << 20), (130, 1 << 20, 130)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_wgrad_of_wide_operands(rows, n, k, accumulate):
    g = gen(2)
    dy, x = small(g, rows, n), small(g, rows, k)
    one = lambda width: torch.ones(up(rows) // 128, width, device="cuda")
    dw = small(g, 1, n, k)
    want = dy.t().contiguous() @ x + (dw[0] if accumulate else 0)
    mok.mok_block_wgrad(codes(dy.t()), one(n), codes(x.t()), one(k), dw, accumulate=accumulate, rows=rows)
    assert torch.equal(dw[0], want)


@pytest.mark.parametrize("rows,n,k,dtype", [(20, 40, 200, BF), (3000, 1001, 2000, BF), (3000, 1001, 2000, torch.float32), (7500, 2001, 1000, BF)])
def test_results_far_apart(rows, n, k, dtype):
    """Rows 2^20 elements apart (of 20 rows: 2^27), their last byte beyond 2^32."""
    g, ld = gen(3), 1 << (27 if rows == 20 else 20)
    x, w = small(g, rows, k), small(g, 2, n, k)
    off = torch.tensor([1, rows // 3, rows - 1], dtype=torch.int32, device="cuda")
    xs, ws = torch.ones(up(k) // 128, rows, device="cuda"), torch.ones(2, up(n) // 128, up(k) // 128, device="cuda")
    out = torch.full((rows, ld), -7.0, dtype=dtype, device="cuda")[:, 3:3 + n]
    assert (rows - 1) * ld * out.element_size() > 1 << 32
    mok.mok_block_gemm(codes(x), xs, codes(w), ws, out, offsets=off)
    want = torch.full((rows, n), -7.0, device="cuda")
    want[1:rows // 3] = x[1:rows // 3] @ w[0].t()
    want[rows // 3:rows - 1] = x[rows // 3:rows - 1] @ w[1].t()
    assert torch.equal(out, want.to(dtype))


@pytest.mark.parametrize("cols", [False, True])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_quantising_rows_far_apart(dtype, cols):
    rows, k, ld = 3000, 200, 1 << 20
    x = torch.zeros(rows, ld, dtype=dtype, device="cuda")[:, 8:8 + k]
    x.copy_(small(gen(4), rows, k))
    off = torch.tensor([0, 1111, 2900], dtype=torch.int32, device="cuda")
    P = mok.block_padded_rows(rows, 2)

    def run(t):
        out = [torch.full(s, 3, dtype=dt, device="cuda") for s, dt in (
            ((rows, 256), torch.uint8), ((2, rows), torch.float32), ((k, P), torch.uint8), ((P // 128, k), torch.float32))]
        mok.mok_block_quantize(t, out[0], out[1], *(out[2:] if cols else (None, None)), offsets=off)
        return out

    assert all(torch.equal(a, b) for a, b in zip(run(x), run(x.contiguous())))


def test_quantising_wide_rows():
    """2^20 columns, both directions and as weights: the codes of single rows and columns of them."""
    g, k = gen(5), 1 << 20
    x = torch.randn(130, k, device="cuda", generator=g)
    P = mok.block_padded_rows(130, 1)
    c, s = torch.empty(130, k, dtype=torch.uint8, device="cuda"), torch.empty(k // 128, 130, device="cuda")
    ct, st = torch.empty(k, P, dtype=torch.uint8, device="cuda"), torch.empty(P // 128, k, device="cuda")
    mok.mok_block_quantize(x, c, s, ct, st)
    alone, scales = torch.empty_like(c), torch.empty_like(s)
    mok.mok_block_quantize(x, alone, scales)
    assert torch.equal(alone, c) and torch.equal(scales, s)
    amax = x.view(130, -1, 128).abs().amax(2)
    top = torch.full_like(amax, 448)   # (a tensor: torch divides by a number by multiplying by its reciprocal)
    assert torch.equal(s.t(), amax / top)
    f = top / amax
    assert torch.equal(c.view(130, -1, 128), (x.view(130, -1, 128) * f[..., None]).to(E4M3).view(torch.uint8))
    for a in (0, k - 1000):   # columns, as the rows of a narrower matrix
        t, cs, ss = x[:, a:a + 1000].t().contiguous(), torch.empty(1000, P, dtype=torch.uint8, device="cuda"), torch.empty(P // 128, 1000, device="cuda")
        mok.mok_block_quantize(t, cs, ss)
        assert torch.equal(cs, ct[a:a + 1000]) and torch.equal(ss, st[:, a:a + 1000])
    w = x.view(1, 130, k)
    wc, wsc = torch.empty(1, 130, k, dtype=torch.uint8, device="cuda"), torch.empty(1, 2, k // 128, device="cuda")
    wt, wts = torch.empty(1, k, 256, dtype=torch.uint8, device="cuda"), torch.empty(1, k // 128, 2, device="cuda")
    mok.mok_block_quantize_weights(w, wc, wsc, wt, wts)
    assert torch.equal(wsc[0, 0], amax[:128].amax(0) / top[0]) and torch.equal(wsc[0, 1], amax[128:].amax(0) / top[0])
    assert torch.equal(wts, wsc.transpose(1, 2).contiguous())
    assert torch.equal(wt[0, :, :130], wc[0].t()) and not wt[0, :, 130:].any()


@pytest.mark.parametrize("rows,n,k,dtype", [(3000, 130, 256, BF), (100_000, 512, 640, BF), (100_000, 500, 640, torch.float32)])
def test_a_thousand_groups(rows, n, k, dtype):
    """1,024 groups of uneven lengths, many of them empty: each row by its own group's weights, and the weight gradient."""
    g, G = gen(6), 1024
    cuts = torch.randint(0, rows + 1, (G + 1,), device="cuda", generator=g).sort().values
    cuts[100:400] = cuts[100]
    x, w = small(g, rows, k), small(g, G, n, k)
    off = cuts.to(torch.int32)
    xs, ws = torch.ones(up(k) // 128, rows, device="cuda"), torch.ones(G, up(n) // 128, up(k) // 128, device="cuda")
    out = torch.full((rows, n), -7.0, dtype=dtype, device="cuda")
    mok.mok_block_gemm(codes(x), xs, codes(w), ws, out, offsets=off)
    P = mok.block_padded_rows(rows, G)
    col = lambda width: (torch.empty(width, P, dtype=torch.uint8, device="cuda"), torch.empty(P // 128, width, device="cuda"))
    dy = small(g, rows, n)
    y, c, dw = col(n), col(k), torch.full((G, n, k), -7.0, device="cuda")
    mok.mok_block_quantize(dy, codes_t=y[0], scales_t=y[1], offsets=off)
    mok.mok_block_quantize(x, codes_t=c[0], scales_t=c[1], offsets=off)
    mok.mok_block_wgrad(*y, *c, dw, offsets=off, rows=rows)
    want = torch.full((rows, n), -7.0, device="cuda")
    for e, (a, b) in enumerate(zip(cuts.tolist(), cuts[1:].tolist())):
        if b == a:
            assert not dw[e].any()
            continue
        want[a:b] = x[a:b] @ w[e].t()
        # codes are 0 and 448 (of -1, 0 and 1), scales 1 / 448: each product is 1 but for the scales' roundings
        exact = dy[a:b].t().contiguous() @ x[a:b]
        size = dy[a:b].abs().t().contiguous() @ x[a:b].abs()
        assert ((dw[e] - exact).abs() <= (b - a + 4) * 2.0 ** -23 * size).all()
    assert torch.equal(out, want.to(dtype))
