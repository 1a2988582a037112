"""The number of rows that the binding of the weight gradient hands to the library, without a GPU: host tensors, and in
place of the call one that notes its arguments."""
import pytest

torch = pytest.importorskip("torch")

import combine_router_top_schedule_amd as mok

MOST = 1 << 22


@pytest.fixture
def rows_of(monkeypatch):
    monkeypatch.setattr(mok, "_device_of", lambda t: t.get_device())   # (-1 for host tensors, here the same for all)
    seen = []
    monkeypatch.setattr(mok, "_launch", lambda fn, dev, stream, desc, *a: seen.append(desc._obj.rows))

    def call(held, groups, **kw):
        P = mok.block_padded_rows(held, groups)
        c, s = torch.empty(1, P, dtype=torch.uint8), torch.empty(P // 128, 1)
        mok.mok_block_wgrad(c, s, c, s, torch.empty(groups, 1, 1), offsets=torch.zeros(groups + 1, dtype=torch.int32), **kw)
        return seen.pop()

    return call


@pytest.mark.parametrize("groups", [1, 2, 4, 64, 1024])
@pytest.mark.parametrize("rows", [0, 1, 40, 127, 128, 129, MOST - 500, MOST - 127, MOST - 50, MOST - 1, MOST])
def test_rows(rows_of, rows, groups):
    assert rows_of(rows, groups, rows=rows) == rows
    bound = rows_of(rows, groups)
    assert rows <= bound <= MOST   # (the library takes no more)
    assert mok.block_padded_rows(bound, groups) == mok.block_padded_rows(rows, groups)


def test_rows_of_other_codes(rows_of):
    for say in (-1, 0, 2, 131, MOST + 1, 1 << 30):   # 384 columns in 3 groups: 3 to 130 rows
        with pytest.raises(ValueError):
            rows_of(40, 3, rows=say)
    assert [rows_of(40, 3, rows=n) for n in (3, 130)] == [3, 130]
