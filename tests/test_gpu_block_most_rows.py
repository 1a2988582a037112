"""The most rows whose column codes are written and read, 2^22, in one group and in several: accepted by the quantiser and
by the weight gradient, and right. One-column operands of ones in exact scales, so every sum is exact."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok


@pytest.mark.parametrize("rows,groups", [(1 << 22, 1), (1 << 22, 2), (1 << 22, 4), ((1 << 22) - 50, 64)])
@pytest.mark.parametrize("say", [False, True])
def test_most_rows(rows, groups, say):
    # 448 times a scale of 1 is the value 448: a code and a scale without a rounding
    x = torch.full((rows, 1), 448.0, device="cuda")
    P = mok.block_padded_rows(rows, groups)
    c, s = torch.empty(1, P, dtype=torch.uint8, device="cuda"), torch.empty(P // 128, 1, device="cuda")
    cuts = [rows * g // groups // 7 * 7 for g in range(groups)] + [rows]
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    mok.mok_block_quantize(x, codes_t=c, scales_t=s, offsets=off)
    dw = torch.full((groups, 1, 1), -7.0, device="cuda")
    mok.mok_block_wgrad(c, s, c, s, dw, offsets=off, **(dict(rows=rows) if say else {}))
    # 448^2 = 49 * 2^12 a row: sums of up to 2^22 of them have more than 24 bits, a block's 128 adds 2^19 * 49; at most
    # 2^15 additions, each off by 2^-24 of the result
    for got, a, b in zip(dw.view(-1).tolist(), cuts, cuts[1:]):
        want = 448.0 ** 2 * (b - a)
        assert abs(got - want) <= (b - a + 127) // 128 * 2.0 ** -24 * want
