"""Groups of experts whose scores fp32 cannot order, under biases of 8 and more, against fp64.

Two experts of a group have a bias b and scores just beside the middle between two fp32 numbers near b + 1/2,
so a key loses up to half a unit of its size, a sum of two keys another half unit, and groups whose exact
scores lie a few 2^-24 apart differ by whole units in fp32. Tokens whose border between the last group that
stays and the first that goes is below 1e-11 are left out: fp64 sums of numbers below 2^9 are off by up to
2^-44 = 6e-14 each."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok

U = 2.0 ** -24


@pytest.mark.parametrize("E", [64, 256, 512])
@pytest.mark.parametrize("power", [3, 4, 5, 6, 8])
@pytest.mark.parametrize("group_score", ["top2", "max"])
def test_groups_nearer_than_fp32(group_score, power, E):
    G, Kg, n = 8, 4, 60_000
    b = 2.0 ** power - 0.5
    two = 2 if group_score == "top2" else 1
    gen = torch.Generator(device="cuda").manual_seed(power)
    bias = torch.zeros(G, E // G, device="cuda")
    bias[:, :two] = b
    # scores in half units of b + 1/2 above 1/2 (odd ones: the middles), and up to 3 u beside
    half = (2 * torch.randint(0, 4, (n, G, two), generator=gen, device="cuda") + 1).double() * 2 ** power * U
    s = 0.5 + half + (6 * torch.rand(n, G, two, generator=gen, device="cuda").double() - 3) * U
    x = torch.full((n, G, E // G), -30.0, device="cuda")
    x[..., :two] = torch.log(s / (1 - s)).float()
    x = x.view(n, E)
    key = 1 / (1 + torch.exp(-x.double())) + bias.double().view(E)
    score = torch.sort(key.view(n, G, -1), -1, descending=True)[0][..., :two].sum(-1)
    order, at = torch.sort(score, dim=1, descending=True, stable=True)
    clear = order[:, Kg - 1] - order[:, Kg] > 1e-11
    assert clear.sum() > 0.99 * n
    K = Kg * two
    want = torch.sort((at[:, :Kg, None] * (E // G) + torch.arange(two, device="cuda")).reshape(n, K), 1)[0]
    idx = torch.empty(n, K, dtype=torch.int32, device="cuda")
    w = torch.empty(n, K, device="cuda")
    mok.mok_route_fwd(mok.route_desc(E, K, "sigmoid", G, Kg, group_score), x, idx, w, bias=bias.view(E))
    got = torch.sort(idx.long(), 1)[0]
    wrong = (got != want).any(1) & clear
    assert not wrong.any(), (int(wrong.sum()), got[wrong][:3].tolist(), want[wrong][:3].tolist())
