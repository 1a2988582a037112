"""Block-scaled FP8 on the GPU against oracle.block.

Codes and scales are formed by fp32 operations that the header states, so they are compared bit for bit. Products:
fp32 results sum exact products of codes (8 bits times 8 bits) in fp32, at most up(K) additions and two
products by scales a block, so they are within (up(K) + 2 up(K) / 128) 2^-23 of the sum of the terms' sizes (2^-23: the matrix
cores may cut where IEEE rounds). bf16 results may lose, in each block of 128, 128 times 2^-19 of the largest possible
term (the FP8 instructions cut products some 20 bits below the largest), and half a step, 2^-8, of the result."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import block as ob

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok
from combine_router_top_schedule_amd.block import MokBlockLinear

F = np.float32
BF = torch.bfloat16


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.float().cpu().numpy() if t.dtype == BF else t.cpu().numpy()


def features(rng, rows, k):
    """Features of different sizes, a few of them large."""
    return (rng.standard_normal((rows, k)) * np.exp(0.5 * rng.standard_normal(k)) * np.where(rng.random(k) < 0.02, 20, 1)).astype(F)


def dev_offsets(off):
    return None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")


def quantize(x, off, rows=True, cols=True, groups=None):
    """(codes, scales, codes_t, scales_t), buffers filled with 0xA5 and -3 before."""
    R, K = x.shape
    G = 1 if off is None else len(off) - 1
    P = mok.block_padded_rows(R, G)
    c = torch.full((R, ob.up(K)), 0xA5, dtype=torch.uint8, device="cuda") if rows else None
    s = torch.full((ob.up(K) // 128, R), -3.0, device="cuda") if rows else None
    ct = torch.full((K, P), 0xA5, dtype=torch.uint8, device="cuda") if cols else None
    st = torch.full((P // 128, K), -3.0, device="cuda") if cols else None
    mok.mok_block_quantize(x, c, s, codes_t=ct, scales_t=st, offsets=dev_offsets(off))
    return c, s, ct, st


def same_codes(a, b):
    """Equal, E4M3's two codes of NaN (0x7F, 0xFF) as one: which of them stands for a NaN is not stated."""
    one = lambda c: np.where((c & 0x7F) == 0x7F, 0x7F, c)
    return np.array_equal(one(a), one(b))


def check_quantize(x, off, rows=True, cols=True):
    v = host(x)
    R, K = v.shape
    clean = ob.clean([0, R] if off is None else off, R)
    c, s, ct, st = quantize(x, off, rows, cols)
    if rows:
        rc, rs = ob.quantize_rows(v)
        assert same_codes(host(c), rc) and np.array_equal(host(s), rs, equal_nan=True)
    if cols:
        P = ob.padded_rows(R, len(clean) - 1)
        rc, rs = np.full((K, P), 0xA5, np.uint8), np.full((P // 128, K), -3, F)
        ob.quantize_columns(v, clean, rc, rs)
        assert same_codes(host(ct), rc) and np.array_equal(host(st), rs, equal_nan=True)


SHAPES = [(1, 1, None), (1, 128, None), (3, 129, [0, 3]), (16, 1024, [0, 5, 16]), (17, 1025, [0, 0, 17, 17]),
          (127, 130, None), (128, 64, [0, 128]), (129, 7, [2, 100, 127]), (300, 257, [0, 1, 130, 130, 299]),
          (600, 40, [100, 228, 228, 356, 484]), (1000, 33, list(range(0, 1001, 10)) + [1000] * 30)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,k,off", SHAPES)
def test_quantize(rows, k, off, dtype):
    x = up(features(np.random.default_rng(rows + k), rows, k)).to(getattr(torch, dtype))
    check_quantize(x, off)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_one_direction_and_strides(dtype):
    x = up(features(np.random.default_rng(5), 150, 264)).to(getattr(torch, dtype))
    off = [3, 50, 149]
    check_quantize(x, off, cols=False)
    check_quantize(x, off, rows=False)
    check_quantize(x[:, 3:203], off)        # rows that begin at no multiple of 16 bytes
    check_quantize(x[:, 8:208], off)
    check_quantize(x[::2], [0, 10, 75])
    check_quantize(x[:, :1], off)
    check_quantize(x[4:5, 1:260], None)


def test_quantize_special_values():
    x = np.zeros((260, 300), F)
    rng = np.random.default_rng(6)
    x[1] = np.nan
    x[2, 7] = np.nan
    x[3, 9] = np.inf
    x[4, 200] = -np.inf
    x[5] = 2.0 ** -120 * rng.standard_normal(300)
    x[6] = 2.0 ** -140 * rng.standard_normal(300)
    x[7] = 3e38 * rng.uniform(-1, 1, 300)
    x[8] = -0.0
    x[9, ::2] = 2.0 ** -99
    x[10] = np.linspace(-448, 448, 300)
    x[11:] = rng.standard_normal((249, 300)) * np.exp2(rng.integers(-30, 30, (249, 300)))
    x[200, 100] = np.nan
    x[250, 299] = np.inf
    check_quantize(up(x), [0, 9, 140, 260])
    check_quantize(up(x).to(BF), [0, 9, 140, 260])
    check_quantize(up(x), None, cols=False)


@pytest.mark.parametrize("off", [[-5, 4, 2, 900], [7, 3, 3, 3], [40, 40, 40], [2 ** 31 - 1] * 3, [-2 ** 31, -1, 0]])
def test_offsets_out_of_range(off):
    """Clamped to the rows, and an offset below an earlier one counts as that one: nothing outside is touched."""
    rng = np.random.default_rng(7)
    x = up(features(rng, 40, 130))
    check_quantize(x, off)
    check_gemm(40, 20, 130, off, "float32", seed=7)
    check_wgrad(40, 20, 130, off, seed=7)


def test_no_rows():
    e = torch.empty(0, 130, device="cuda")
    check_quantize(e, [0, 0, 0])
    w, ws = weights(np.random.default_rng(0), 2, 5, 130)
    mok.mok_block_gemm(torch.empty(0, 256, dtype=torch.uint8, device="cuda"), torch.empty(2, 0, device="cuda"), w, ws,
                       torch.empty(0, 5, device="cuda"), offsets=dev_offsets([0, 0, 0]))
    for G in (1, 3):
        P = mok.block_padded_rows(0, G)
        dw = torch.full((G, 5, 6), 7.0, device="cuda")
        t = lambda n: (torch.empty(n, P, dtype=torch.uint8, device="cuda"), torch.empty(P // 128, n, device="cuda"))
        mok.mok_block_wgrad(*t(5), *t(6), dw, offsets=dev_offsets([0] * (G + 1)), accumulate=True)
        assert (dw == 7).all()
        mok.mok_block_wgrad(*t(5), *t(6), dw, offsets=dev_offsets([0] * (G + 1)))
        assert (dw == 0).all()


def weights(rng, g, n, k):
    w = up((0.02 * rng.standard_normal((g, n, k))).astype(F))
    c = torch.empty(g, n, ob.up(k), dtype=torch.uint8, device="cuda")
    s = torch.empty(g, ob.up(n) // 128, ob.up(k) // 128, device="cuda")
    mok.mok_block_quantize_weights(w, c, s)
    return c, s


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("g,n,k", [(1, 1, 1), (2, 128, 128), (3, 130, 257), (1, 7, 640), (5, 300, 5), (2, 256, 1000)])
def test_quantize_weights(g, n, k, dtype):
    rng = np.random.default_rng(n + k)
    w = up((0.02 * rng.standard_normal((g, n, k))).astype(F)).to(getattr(torch, dtype))
    if n > 100:
        w[0, 3, 3] = float("nan")
    if k > 500:
        w[-1, -1, -1] = float("inf")
    c = torch.full((g, n, ob.up(k)), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.empty(g, ob.up(n) // 128, ob.up(k) // 128, device="cuda")
    ct = torch.full((g, k, ob.up(n)), 0xA5, dtype=torch.uint8, device="cuda")
    st = torch.empty(g, ob.up(k) // 128, ob.up(n) // 128, device="cuda")
    mok.mok_block_quantize_weights(w, c, s, codes_t=ct, scales_t=st)
    rc, rs = ob.quantize_weights(host(w))
    assert same_codes(host(c), rc) and np.array_equal(host(s), rs)
    rc, rs = ob.quantize_weights(host(w).transpose(0, 2, 1))
    assert same_codes(host(ct), rc) and np.array_equal(host(st), rs)
    alone = torch.full_like(c, 0xA5)
    mok.mok_block_quantize_weights(w, alone, s)
    assert torch.equal(alone, c)


def close(got, want, size, most, k, bf):
    blocks = ob.up(k) // 128
    if bf:
        bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * most + (blocks + 128) * 2.0 ** -23 * size
    else:
        bound = (ob.up(k) + 2 * blocks) * 2.0 ** -23 * size
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], bound[bad][:5])


def check_gemm(rows, n, k, off, dtype, seed=0, pad=0):
    """Against the oracle; rows in no group and what lies between strided rows keep what they held."""
    rng = np.random.default_rng(seed)
    g = 1 if off is None else len(off) - 1
    x = up(features(rng, rows, k))
    c, s, _, _ = quantize(x, off, cols=False)
    w, ws = weights(rng, g, n, k)
    wide = torch.full((rows, n + pad), -7.0, dtype=getattr(torch, dtype), device="cuda")
    out = wide[:, :n]
    mok.mok_block_gemm(c, s, w, ws, out, offsets=dev_offsets(off))
    clean = ob.clean([0, rows] if off is None else off, rows)
    want = np.full((rows, n), -7.0)
    want, size, most = ob.gemm(host(c), host(s), host(w), host(ws), clean, want)
    live = np.zeros(rows, bool)
    for a, b in zip(clean, clean[1:]):
        live[a:b] = True
    got = host(wide)
    assert (got[~live] == -7).all() and (got[:, n:] == -7).all()
    close(got[live, :n], want[live], size[live], most[live], k, dtype == "bfloat16")
    return c, s, w, ws, out


GEMMS = [(1, 1, 1, None), (1, 64, 256, None), (5, 33, 130, [0, 2, 5]), (16, 128, 128, None), (17, 130, 384, [0, 17, 17]),
         (33, 65, 1300, [1, 30, 33]), (64, 40, 256, None), (65, 256, 512, [0, 1, 65]), (130, 300, 200, [0, 129, 130]),
         (200, 1000, 130, None), (700, 520, 384, [0, 0, 300, 301, 690])]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,n,k,off", GEMMS)
def test_gemm(rows, n, k, off, dtype):
    check_gemm(rows, n, k, off, dtype, seed=rows + n)


@pytest.mark.parametrize("rows,n,k,off,dtype", [
    (3000, 2100, 9000, [0, 1000, 2990], "float32"),        # 128 x 128 tiles, more than 64 blocks of the sum
    (2500, 1900, 8400, [10, 1300, 1300, 2500], "bfloat16"),
    (9000, 4100, 384, [0, 3000, 8990], "bfloat16"),        # 256 x 256 tiles
    (8192, 2048, 8832, None, "bfloat16"),                  # the same, more than 64 blocks
    (2000, 1024, 128, [i * 2 for i in range(1001)], "bfloat16")])   # 1,000 groups of 2 rows
def test_gemm_large(rows, n, k, off, dtype):
    check_gemm(rows, n, k, off, dtype, seed=3)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows", [3, 140, 2600])
def test_gemm_strided_out(rows, dtype):
    for pad in (1, 4, 8):
        check_gemm(rows, 257 if pad == 1 else 264, 200, [0, 2, rows - 1], dtype, seed=pad, pad=pad)


def test_gemm_not_finite_stays_in_its_row():
    """A NaN or an infinity in a row of x makes that row NaN and no other; one in w a column of its group."""
    rng = np.random.default_rng(11)
    for rows in (5, 300):
        x = features(rng, rows, 200)
        x[1, 5], x[3, 150] = np.nan, np.inf
        off = [0, rows - 2, rows]
        c, s, _, _ = quantize(up(x), off, cols=False)
        w, ws = weights(rng, 2, 40, 200)
        out = torch.zeros(rows, 40, device="cuda")
        mok.mok_block_gemm(c, s, w, ws, out, offsets=dev_offsets(off))
        bad = np.isnan(host(out))
        assert bad[[1, 3]].all() and not np.delete(bad, [1, 3], 0).any()
        w[1, 7, 3] = 0x7F
        mok.mok_block_gemm(c, s, w, ws, out, offsets=dev_offsets(off))
        bad = np.isnan(host(out))
        others = [r for r in range(rows - 2, rows) if r not in (1, 3)]
        assert bad[rows - 2:, 7].all() and not np.delete(bad[others], 7, 1).any()


def test_gemm_is_independent_of_the_batch():
    """A row's result does not depend on the other rows of its tile, and calls repeat bit for bit."""
    c, s, w, ws, out = check_gemm(700, 300, 900, [0, 400, 700], "bfloat16", seed=12)
    again = torch.empty_like(out)
    for _ in range(3):
        mok.mok_block_gemm(c, s, w, ws, again, offsets=dev_offsets([0, 400, 700]))
        assert torch.equal(again, out)
    mok.mok_block_gemm(c[100:], s[:, 100:].contiguous(), w, ws, again[100:], offsets=dev_offsets([0, 300, 600]))
    assert torch.equal(again[100:], out[100:])


def check_wgrad(rows, n, k, off, accumulate=False, seed=0):
    rng = np.random.default_rng(seed)
    g = 1 if off is None else len(off) - 1
    clean = ob.clean([0, rows] if off is None else off, rows)
    _, _, yt, yts = quantize(up((1e-3 * rng.standard_normal((rows, n))).astype(F)), off, rows=False)
    _, _, xt, xts = quantize(up(features(rng, rows, k)), off, rows=False)
    dw0 = rng.standard_normal((g, n, k)).astype(F)
    dw = up(dw0)
    mok.mok_block_wgrad(yt, yts, xt, xts, dw, offsets=dev_offsets(off), accumulate=accumulate)
    want = dw0.astype(np.float64) if accumulate else np.zeros((g, n, k))
    want, size = ob.wgrad(host(yt), host(yts), host(xt), host(xts), clean, want)
    close(host(dw), want, size, None, max(int(np.diff(clean).max()), 1) + 1, False)
    return yt, yts, xt, xts, dw


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows,n,k,off", [
    (1, 1, 1, None), (130, 5, 7, None), (128, 128, 128, [0, 128]), (257, 130, 129, [0, 1, 1, 257]), (300, 33, 300, [7, 130, 290]),
    (2000, 260, 140, [0, 1000, 1500, 2000]), (700, 40, 50, list(range(0, 701, 7)))])
def test_wgrad(rows, n, k, off, accumulate):
    check_wgrad(rows, n, k, off, accumulate, seed=rows)


def test_wgrad_large():
    yt, yts, xt, xts, dw = check_wgrad(9000, 1300, 900, [0, 8500, 8990], seed=5)
    again = torch.empty_like(dw)
    for _ in range(3):
        mok.mok_block_wgrad(yt, yts, xt, xts, again, offsets=dev_offsets([0, 8500, 8990]))
        assert torch.equal(again, dw)


def test_linear_forward_backward_against_the_formula():
    """MokBlockLinear's results are the oracle's products of its own codes; dx and dw are its gradients."""
    rng = np.random.default_rng(20)
    R, N, K, off = 300, 136, 200, [0, 120, 120, 295]
    w = up((0.05 * rng.standard_normal((3, N, K))).astype(F))
    lin = MokBlockLinear(w, R)
    x, dy = up(features(rng, R, K)), up(rng.standard_normal((R, N)).astype(F))
    out, dx = torch.full((R, N), 9.0, device="cuda"), torch.full((R, K), 9.0, device="cuda")
    dw = torch.empty_like(w)
    o = dev_offsets(off)
    lin.forward(x, out, offsets=o)
    lin.backward(dy, dx, dw, offsets=o)
    xv, wv = ob.values_rows(host(lin.xq), host(lin.xs)), ob.values_weights(host(lin.wq), host(lin.ws))
    yv = ob.values_rows(host(lin.yq), host(lin.ys))
    # (the bound of close() for sums of up to 384 terms, of the sizes' largest row and column sums)
    for g, (a, b) in enumerate(zip(off, off[1:])):
        for got, p, q in ((out, xv[a:b], wv[g].T), (dx, yv[a:b, :N], wv[g][:, :K])):
            n = min(p.shape[1], q.shape[0])
            want, size = p[:, :n] @ q[:n], np.abs(p[:, :n]) @ np.abs(q[:n])
            assert (np.abs(host(got)[a:b] - want) <= 400 * 2.0 ** -23 * size).all()
    assert (host(out)[295:] == 9).all() and (host(dx)[295:] == 9).all() and (host(dw)[1] == 0).all()
    yt, xt = ob.values_rows(host(lin.yt), host(lin.yts)), ob.values_rows(host(lin.xt), host(lin.xts))
    at = ob.columns(off)
    for g in (0, 2):
        want = yt[:, at[g]:at[g + 1]] @ xt[:, at[g]:at[g + 1]].T
        size = np.abs(yt[:, at[g]:at[g + 1]]) @ np.abs(xt[:, at[g]:at[g + 1]]).T
        assert (np.abs(host(dw)[g] - want) <= 400 * 2.0 ** -23 * size).all()
    # and the quantised gradient is near the plain one: each operand is off by half a step of E4M3, 2^-4 of a value, in
    # random directions, so a sum by well under 2^-4 of its terms' root of squares
    plain = np.stack([host(dy)[a:b].T.astype(np.float64) @ host(x)[a:b] for a, b in zip(off, off[1:])])
    root = np.sqrt(np.stack([(host(dy)[a:b].T.astype(np.float64) ** 2) @ (host(x)[a:b].astype(np.float64) ** 2)
                             for a, b in zip(off, off[1:])]))
    assert np.linalg.norm(host(dw) - plain) <= 2.0 ** -4 * np.linalg.norm(root)


def test_linear_in_a_graph():
    """Forward and backward captured, replayed on new inputs with eager work between."""
    rng = np.random.default_rng(21)
    R, N, K = 200, 130, 150
    lin = MokBlockLinear(up((0.05 * rng.standard_normal((2, N, K))).astype(F)).to(BF), R)
    x, dy = up(features(rng, R, K)).to(BF), up(rng.standard_normal((R, N)).astype(F)).to(BF)
    o = dev_offsets([0, 90, 200])
    out, dx = torch.empty(R, N, dtype=BF, device="cuda"), torch.empty(R, K, dtype=BF, device="cuda")
    dw = torch.zeros(2, N, K, device="cuda")

    def go(out, dx, dw):
        lin.forward(x, out, offsets=o)
        lin.backward(dy, dx, dw, offsets=o, accumulate=True)

    go(out, dx, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(out, dx, dw)
    for step in range(3):
        x.copy_(up(features(rng, R, K)))
        dy.copy_(up(rng.standard_normal((R, N)).astype(F)))
        o.copy_(dev_offsets([0, 60 + step, 200 - step]))
        e = torch.full_like(out, 3), torch.full_like(dx, 3), dw.clone()
        out.fill_(3), dx.fill_(3)
        go(*e)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(e, (out, dx, dw)):
            assert torch.equal(a, b)


def test_on_another_stream():
    rng = np.random.default_rng(22)
    c, s, w, ws, out = check_gemm(300, 200, 500, None, "bfloat16", seed=22)
    side, other = torch.cuda.Stream(), torch.empty_like(out)
    side.wait_stream(torch.cuda.current_stream())
    mok.mok_block_gemm(c, s, w, ws, other, stream=side)
    with torch.cuda.stream(side):
        third = torch.empty_like(out)
        mok.mok_block_gemm(c, s, w, ws, third)
    side.synchronize()
    assert torch.equal(other, out) and torch.equal(third, out)


def test_after_a_schedule_table():
    """The offsets of a layer's schedule table and its dispatched rows go straight into a product."""
    import datagen
    from combine_router_top_schedule_amd.layer import MokLayer
    cfg = datagen.CONFIGS["tiny"]
    layer = MokLayer(mok.desc_from_config(cfg), staged=True, fused=False)
    layer.schedule(torch.from_numpy(datagen.logits(cfg)).cuda())
    x = torch.from_numpy(datagen.x_all(cfg).view(np.int16)).cuda()
    layer.dispatch(layer.segs(x))
    rows = cfg.N * cfg.K
    xd = layer.xd[:rows * cfg.H * 2].view(BF).view(rows, cfg.H)
    off = layer.saved[96 * 4:(96 + cfg.E_loc + 1) * 4].view(torch.int32)
    w = up((0.05 * np.random.default_rng(1).standard_normal((cfg.E_loc, 72, cfg.H))).astype(F))
    lin = MokBlockLinear(w, rows, train=False)
    out = torch.empty(rows, 72, device="cuda")
    lin.forward(xd, out, offsets=off)
    want, size, most = ob.gemm(host(lin.xq), host(lin.xs), host(lin.wq), host(lin.ws), host(off), np.zeros((rows, 72)))
    close(host(out), want, size, most, cfg.H, False)
    with pytest.raises(RuntimeError):
        lin.backward(out, dw=w)


def test_binding_refusals():
    x = torch.zeros(4, 200, device="cuda")
    c, s = torch.zeros(4, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, 4, device="cuda")
    w, ws = torch.zeros(2, 6, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, 1, 2, device="cuda")
    o, out = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, 6, device="cuda")
    P = mok.block_padded_rows(4, 2)
    yt, yts, xt, xts = (torch.zeros(6, P, dtype=torch.uint8, device="cuda"), torch.zeros(P // 128, 6, device="cuda"),
                        torch.zeros(7, P, dtype=torch.uint8, device="cuda"), torch.zeros(P // 128, 7, device="cuda"))
    dw = torch.zeros(2, 6, 7, device="cuda")
    bad = [
        lambda: mok.mok_block_quantize(x.half(), c, s), lambda: mok.mok_block_quantize(x, c),
        lambda: mok.mok_block_quantize(x, c[:, :128], s), lambda: mok.mok_block_quantize(x, c, s.t()),
        lambda: mok.mok_block_quantize(x.t(), c, s), lambda: mok.mok_block_quantize(x, c, s, offsets=o.long()),
        lambda: mok.mok_block_quantize(x[0], c, s), lambda: mok.mok_block_quantize(x, c.float(), s),
        lambda: mok.mok_block_quantize(x, c, s, offsets=o[:1]), lambda: mok.mok_block_quantize(x, c, s.cpu()),
        lambda: mok.mok_block_gemm(c, s, w, ws, out), lambda: mok.mok_block_gemm(c, s, w[:1], ws, out, offsets=o),
        lambda: mok.mok_block_gemm(c[:, :200], s, w, ws, out, offsets=o), lambda: mok.mok_block_gemm(c, s, w, ws, out.half(), offsets=o),
        lambda: mok.mok_block_gemm(c, s, w, ws, out.cpu(), offsets=o), lambda: mok.mok_block_gemm(c, s, w, ws, out[:3], offsets=o),
        lambda: mok.mok_block_wgrad(yt, yts, xt, xts, dw), lambda: mok.mok_block_wgrad(yt[:, :100], yts, xt, xts, dw, offsets=o),
        lambda: mok.mok_block_wgrad(yt, yts, xt, xts, dw.bfloat16(), offsets=o), lambda: mok.mok_block_wgrad(yt, yts, xt, xts, dw[0], offsets=o),
        lambda: mok.mok_block_wgrad(yt, yts, xt, xts[:, :6], dw, offsets=o),
        lambda: mok.mok_block_quantize_weights(out, c, s), lambda: mok.mok_block_quantize_weights(dw.transpose(1, 2), w, ws)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    for f in (lambda: mok.mok_block_quantize(x), lambda: mok.mok_block_quantize(x, c.view(-1)[8:].new_zeros(4, 256), s)):
        try:
            f()
        except mok.MokError as e:
            assert e.code in (1, 4)


def test_many_rows_and_few_columns():
    """More row tiles than a grid's second dimension holds."""
    R, N, K = 5_000_000, 16, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(0, 0x7F, (R, K), dtype=torch.uint8, device="cuda", generator=g)
    xs = torch.rand(1, R, device="cuda", generator=g)
    w, ws = weights(np.random.default_rng(1), 1, N, K)
    out = torch.zeros(R, N, dtype=BF, device="cuda")
    mok.mok_block_gemm(x, xs, w, ws, out)
    for a in (0, 2_499_990, R - 10):
        want, size, most = ob.gemm(host(x[a:a + 10]), host(xs[:, a:a + 10]), host(w), host(ws), [0, 10], np.zeros((10, N)))
        close(host(out[a:a + 10]), want, size, most, K, True)
    c, s = torch.zeros(R, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1, R, device="cuda")
    mok.mok_block_quantize(out, c, s)
    for a in (0, R - 10):
        rc, rs = ob.quantize_rows(host(out[a:a + 10]))
        assert same_codes(host(c[a:a + 10]), rc) and np.array_equal(host(s[:, a:a + 10]), rs)
