"""mok_block_gemm's tile kernels, 128 x 128 and 256 x 256, where tiles end inside groups, rows and columns: against
oracle.block in the bounds of its products (see close()), rows in no group and what lies beside strided rows untouched. Every
test asks first that its sizes go to the kernel it is about."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import block as ob

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok

F, BF = np.float32, torch.bfloat16
KIND = {"128": mok.MOK_BLOCK_TILES_128, "256": mok.MOK_BLOCK_TILES_256}


def kernel(rows, groups, n, k, dtype):
    elem = mok.MOK_ELEM_BF16 if dtype is BF else mok.MOK_ELEM_F32
    return mok.lib().mok_block_gemm_kernel(ctypes.byref(mok.MokBlockDesc(rows, n, groups, n, ob.up(k), elem)))


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a, F)).cuda()


def host(t):
    return t.float().cpu().numpy() if t.dtype == BF else t.cpu().numpy()


class Case:
    """Quantised operands of one product."""

    def __init__(self, rows, n, k, off, seed=0, spoil=None):
        rng = np.random.default_rng(seed)
        self.rows, self.n, self.k, self.off = rows, n, k, off
        self.groups = 1 if off is None else len(off) - 1
        x = (rng.standard_normal((rows, k)) * np.exp(0.5 * rng.standard_normal(k)) * np.where(rng.random(k) < 0.02, 20, 1)).astype(F)
        w = (0.02 * rng.standard_normal((self.groups, n, k))).astype(F)
        if spoil:
            spoil(x, w)
        kp, kb, nb = ob.up(k), ob.up(k) // 128, ob.up(n) // 128
        u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")
        f32 = lambda *s: torch.empty(s, device="cuda")
        self.x, self.xs, self.w, self.ws = u8(rows, kp), f32(kb, rows), u8(self.groups, n, kp), f32(self.groups, nb, kb)
        self.o = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
        mok.mok_block_quantize(up(x), self.x, self.xs, offsets=self.o)
        mok.mok_block_quantize_weights(up(w), self.w, self.ws)

    def run(self, out):
        mok.mok_block_gemm(self.x, self.xs, self.w, self.ws, out, offsets=self.o)
        return out

    def live(self):
        clean = ob.clean([0, self.rows] if self.off is None else self.off, self.rows)
        mask = np.zeros(self.rows, bool)
        for a, b in zip(clean, clean[1:]):
            mask[a:b] = True
        return clean, mask


def close(c, got):
    """fp32: sums of exact products, (terms and two scales a block) 2^-23 of the sum of the terms' sizes. bf16: half a step,
    2^-8, of the result, in each block 128 times 2^-19 of its largest possible term (what the FP8 instructions cut),
    and the blocks' fp32 sums."""
    clean, live = c.live()
    want, size, most = ob.gemm(host(c.x), host(c.xs), host(c.w), host(c.ws), clean, np.full((c.rows, c.n), -7.0))
    blocks = ob.up(c.k) // 128
    if got.dtype == BF:
        bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * most + (blocks + 128) * 2.0 ** -23 * size
    else:
        bound = (ob.up(c.k) + 2 * blocks) * 2.0 ** -23 * size
    y = host(got)
    assert (y[~live] == -7).all()
    bad = live[:, None] & ~(np.abs(y - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], y[bad][:5], want[bad][:5], bound[bad][:5])


# (kind, result, rows, n, k, offsets): three groups and more, one empty, rows before the first and behind the last, ends
# inside tiles of 128 and of 256 rows and columns, one row in a group
SIZES = [("256", BF, 7500, 2001, 1000, [37, 2000, 2000, 4300, 4301, 7411]),
         ("256", BF, 7400, 2043, 900, [0, 255, 511, 768, 7399]),
         ("256", BF, 7700, 1985, 1100, None),
         ("128", BF, 3000, 1001, 2000, [5, 700, 700, 829, 830, 2900]),
         ("128", BF, 3001, 1115, 2000, None),
         ("128", torch.float32, 3000, 1001, 2000, [5, 700, 700, 829, 830, 2900]),
         ("128", torch.float32, 3001, 1115, 2000, None)]


@pytest.mark.parametrize("kind,dtype,rows,n,k,off", SIZES)
def test_strides_and_ends(kind, dtype, rows, n, k, off):
    c = Case(rows, n, k, off, seed=rows)
    assert kernel(rows, c.groups, n, k, dtype) == KIND[kind]
    each = 16 // (2 if dtype is BF else 4)   # elements in 16 bytes
    wide = -(-n // each) * each
    first = None
    # rows as long as they are; rows of whole 16 bytes, whose last piece is partial; longer ones; such rows that begin between
    for ld, skip in ((n, 0), (wide, 0), (wide + 3 * each, each), (wide + each, 1)):
        full = torch.full((rows * ld + 64,), -7.0, dtype=dtype, device="cuda")
        out = full[:rows * ld].view(rows, ld)[:, skip:skip + n]
        if skip + n > ld:
            continue
        c.run(out)
        if first is None:
            close(c, out)
            first = out.clone()
        assert torch.equal(out, first)   # (results do not depend on how they are stored)
        gaps = full.clone()
        gaps[:rows * ld].view(rows, ld)[:, skip:skip + n] = -7
        assert (gaps == -7).all()


@pytest.mark.parametrize("kind,dtype,rows,n,k,off", [SIZES[0], SIZES[3], SIZES[5]])
def test_not_finite_stays_in_its_row(kind, dtype, rows, n, k, off):
    """A NaN or an infinity in a row of x makes that row NaN and no other, one in w a column of its group (an infinity, whose
    block of 128 columns has one scale, all of these)."""
    assert kernel(rows, len(off) - 1, n, k, dtype) == KIND[kind]
    a, b, e = off[1], off[3], off[-1]

    def spoil(x, w):
        x[a - 1, 5], x[b, 150], x[e - 1, k - 1], x[e] = np.nan, np.inf, -np.inf, np.nan
        w[3, n - 1, 3], w[4, 130, 7], w[4, 300, k - 1] = np.nan, np.nan, np.inf

    c = Case(rows, n, k, off, seed=2, spoil=spoil)
    bad = np.isnan(host(c.run(torch.full((rows, n), -7.0, dtype=dtype, device="cuda"))))
    want = np.zeros((rows, n), bool)
    want[off[3]:off[4], n - 1] = True
    want[off[4]:e, 130] = True
    want[off[4]:e, 256:384] = True
    want[[a - 1, b, e - 1]] = True   # (row e is in no group)
    assert (bad == want).all()


@pytest.mark.parametrize("kind,dtype,rows,n,k,off", [SIZES[0], SIZES[3], SIZES[5]])
def test_repeats_and_is_independent_of_other_rows(kind, dtype, rows, n, k, off):
    """Calls repeat bit for bit, and a row's result is the same where other rows stand beside it in its tile."""
    c = Case(rows, n, k, off, seed=3)
    assert kernel(rows, c.groups, n, k, dtype) == KIND[kind]
    out = c.run(torch.full((rows, n), -7.0, dtype=dtype, device="cuda"))
    for _ in range(3):
        assert torch.equal(c.run(torch.full_like(out, -7.0)), out)
    cut = 303   # without the first rows: every group's tiles begin elsewhere in memory, the first group's in other rows
    d = Case.__new__(Case)
    d.__dict__.update(c.__dict__)
    d.x, d.xs = c.x[cut:].contiguous(), c.xs[:, cut:].contiguous()
    d.o = (c.o - cut).clamp(min=0)
    assert kernel(rows - cut, c.groups, n, k, dtype) == KIND[kind]
    again = d.run(torch.full((rows - cut, n), -7.0, dtype=dtype, device="cuda"))
    assert torch.equal(again, out[cut:])
