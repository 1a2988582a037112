"""The layer with a given choice of experts, and whole training steps: router projection, gate, layer
forward and backward, gate and projection backward, gradient norm, AdamW, weights packed again; against
the fp64 oracles. A layer with a given choice rounds where the layer always does, so its tolerance is the
layer's (1e-2 of the largest value)."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import datagen
from oracle import moe_oracle as mo
from oracle import optim as oo
from oracle import route as orr

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import combine_router_top_schedule_amd as mok
from combine_router_top_schedule_amd.optim import MokAdamW
from tests._gpu import BF16_TOL, MX_TOL, BwdCase, dev_u16, frob_rel_err, host_u16, max_rel_err

TINY = datagen.CONFIGS["tiny"]
CFGS = {
    "tiny": TINY,
    "share": TINY.replace(S=3, T=100, E=16, K=4, e0=5, E_loc=6, H=256, x_std=1.0),
    "wide": TINY.replace(S=4, T=512, H=512, E=64, K=8, I=256, E_loc=64, x_std=1.0, ring_bytes=32 << 20),
    "mx": TINY.replace(S=2, T=128, E=16, K=4, E_loc=16, M=32, dtype="mxfp8", ring_bytes=32 << 20, x_std=1.0),
}


def oracle_of(case, idx, p):
    """Forward (and what its backward needs) of the given choice."""
    cfg = case.cfg
    W, K = case.oracle_weights(), cfg.K
    sched = mo.schedule(idx, cfg.e0, cfg.E_loc, cfg.M, 32 if cfg.dtype == "mxfp8" else 1)
    x = np.zeros((sched.rows, cfg.H))
    real = sched.perm >= 0
    x[real] = mo.decode_bf16(case.x_h)[sched.perm[real] // K]
    xd = mo.dispatch(x, W.dtype)
    if W.dtype != "bf16":
        xd[~real] = 0.0
    g, u, h, y = mo.expert_ffn(xd, sched, W)
    return mo.Forward(idx, p, sched, xd, g, u, h, y, mo.combine(y, idx, p, sched, cfg.e0, cfg.E_loc), x), W


def choice(cfg, kind, seed=0):
    """Experts and weights: any ("free": unsorted experts, weights of both signs, tokens with few or no
    experts), with the same choice as the kernels are to see it after tidying."""
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(cfg.E)[:cfg.K] for _ in range(cfg.N)]).astype(np.int32)
    p = rng.standard_normal((cfg.N, cfg.K)).astype(np.float32)
    if kind == "free":
        idx[rng.random(idx.shape) < 0.3] = -1
        idx[3] = -1
    clean, q = idx.copy(), p.copy()
    if kind == "untidy":
        idx[::5, 1] = idx[::5, 0]
        idx[2, 0], idx[4, 0], idx[6, 0] = cfg.E, -9, 2 ** 31 - 1
        p[7] = np.nan_to_num(p[7])
        clean = idx.copy()
        for n in range(cfg.N):
            for k in range(cfg.K):
                if not 0 <= clean[n, k] < cfg.E or clean[n, k] in idx[n, :k]:
                    clean[n, k] = -1
    q[clean < 0] = 0
    return idx, p, clean, q


@pytest.mark.parametrize("kind", ["plain", "free", "untidy"])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("name", list(CFGS))
def test_layer_with_a_given_choice(name, fused, kind):
    cfg = CFGS[name]
    idx, p, clean, q = choice(cfg, kind)
    case = BwdCase(cfg, staged=not fused, fused=fused)
    L = case.layer
    L.idx.copy_(torch.from_numpy(idx).flatten())
    L.p.copy_(torch.from_numpy(p).flatten())
    case.out.fill_(0x1234)
    if fused:
        L.forward_routed(case.x_seg, case.out_seg)
    else:
        L.schedule_routed()
        L.dispatch(case.x_seg)
        L.expert_ffn()
        L.combine(case.out_seg)
    case.dp.fill_(-7)
    mok.mok_layer_bwd(case.d, case.dout_seg, case.x_seg, L.w, L.idx, L.p, L.saved, L.ring, L.slots,
                      case.dx_seg, case.dp, None, case.dwg, case.dwu, case.dwd, case.bws)
    torch.cuda.synchronize()
    assert mok.mok_device_status(L.ws) == 0 and mok.mok_device_status(case.bws) == 0
    gi, gp = case.idx_p()
    assert np.array_equal(gi, clean) and np.array_equal(gp, q)
    fw, W = oracle_of(case, clean, q.astype(np.float64))
    bw = mo.backward(fw, mo.bf16_rows(case.dout_h), W, cfg.K, cfg.e0, cfg.E_loc, cfg.E + 1)
    touched = fw.sched.touched
    err, tol = (max_rel_err, BF16_TOL) if cfg.dtype == "bf16" else (frob_rel_err, MX_TOL)
    assert err(case.out_rows(touched), fw.out) <= tol
    rest = np.setdiff1d(np.arange(cfg.N), touched)
    assert (host_u16(case.out)[rest] == 0x1234).all()
    assert err(mo.decode_bf16(host_u16(case.dx))[touched], bw.dx) <= tol
    dp = case.dp.cpu().numpy().reshape(cfg.N, cfg.K)
    local = (clean >= cfg.e0) & (clean < cfg.e0 + cfg.E_loc)
    assert err(dp[local], bw.dp[local]) <= tol and (dp[~local] == -7).all()
    for got, ref in ((case.dwg, bw.dwg), (case.dwu, bw.dwu), (case.dwd, bw.dwd)):
        assert err(got.cpu().numpy().astype(np.float64), ref) <= tol


@pytest.mark.parametrize("fused", [False, True])
def test_sole_pairs_of_weight_nan_and_minus_zero(fused):
    """Tokens with one expert, whose weight the rows' epilogue cannot take as it is."""
    cfg = CFGS["wide"]
    idx, p, _, _ = choice(cfg, "plain")
    idx[3, 1:] = idx[5, 1:] = -1
    outs = []
    for w3, w5 in ((1.0, 1.0), (np.nan, -0.0)):
        p[3, 0], p[5, 0] = w3, w5
        case = BwdCase(cfg, staged=not fused, fused=fused)
        L = case.layer
        L.idx.copy_(torch.from_numpy(idx).flatten())
        L.p.copy_(torch.from_numpy(p).flatten())
        if fused:
            L.forward_routed(case.x_seg, case.out_seg)
        else:
            L.schedule_routed()
            L.dispatch(case.x_seg)
            L.expert_ffn()
            L.combine(case.out_seg)
        torch.cuda.synchronize()
        assert mok.mok_device_status(L.ws) == 0
        outs.append(mo.decode_bf16(host_u16(case.out)))
    assert np.isfinite(outs[0]).all() and outs[0][3].any() and outs[0][5].any()
    assert np.isnan(outs[1][3]).all() and not outs[1][5].any()
    rest = np.setdiff1d(np.arange(cfg.N), [3, 5])
    assert np.array_equal(outs[0][rest], outs[1][rest])


def test_given_choice_equals_the_layers_own():
    """With the layer's own choice and weights given, every output is the same bit for bit."""
    cfg = CFGS["wide"]
    a, b = BwdCase(cfg, staged=False, fused=True), BwdCase(cfg, staged=False, fused=True)
    a.run(fused=True)
    b.layer.idx.copy_(a.layer.idx)
    b.layer.p.copy_(a.layer.p)
    b.layer.forward_routed(b.x_seg, b.out_seg)
    L = b.layer
    mok.mok_layer_bwd(b.d, b.dout_seg, b.x_seg, L.w, L.idx, L.p, L.saved, L.ring, L.slots, b.dx_seg, b.dp,
                      None, b.dwg, b.dwu, b.dwd, b.bws)
    torch.cuda.synchronize()
    for k in ("out", "dx", "dp", "dwg", "dwu", "dwd"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k
    assert torch.equal(a.layer.idx, b.layer.idx) and torch.equal(a.layer.p, b.layer.p)
    # and through route, whose softmax over the chosen is that gate
    dl = torch.full((cfg.N, cfg.E), -7.0, device="cuda")
    b.layer.route(mok.route_desc(cfg.E, cfg.K), b.logits)
    assert torch.equal(a.layer.idx, b.layer.idx)
    b.layer.route_backward(mok.route_desc(cfg.E, cfg.K), b.logits, b.dp, dl)
    assert max_rel_err(dl.double().cpu().numpy(), a.dlogits.double().cpu().numpy()) <= 1e-5


def test_given_choice_and_dlogits_is_reported():
    case = BwdCase(TINY, staged=False, fused=True)
    L = case.layer
    idx, p, _, _ = choice(TINY, "plain")
    L.idx.copy_(torch.from_numpy(idx).flatten())
    L.p.copy_(torch.from_numpy(p).flatten())
    L.forward_routed(case.x_seg, case.out_seg)
    case.dlogits.fill_(-7)
    mok.mok_layer_bwd(case.d, case.dout_seg, case.x_seg, L.w, L.idx, L.p, L.saved, L.ring, L.slots,
                      case.dx_seg, case.dp, case.dlogits, case.dwg, case.dwu, case.dwd, case.bws)
    torch.cuda.synchronize()
    assert mok.mok_device_status(case.bws) == 9 and (case.dlogits == -7).all()
    # the next forward and backward of the layer's own gate are as ever
    case.run(fused=True)
    fw, bw = case.oracle_backward()
    assert max_rel_err(case.dlogits.cpu().numpy().astype(np.float64), bw.dlogits) <= BF16_TOL


def test_gate_and_layer_in_a_graph():
    """Gate, layer forward and backward, gate backward, captured and replayed on changing logits, with the
    calls made one by one in between."""
    cfg = CFGS["wide"]
    gate = mok.route_desc(cfg.E, cfg.K, "sigmoid", 4, 2, "top2", True, 2.5)
    case = BwdCase(cfg, staged=False, fused=True)
    L, dl = case.layer, torch.empty(cfg.N, cfg.E, device="cuda")
    load = torch.empty(cfg.E, dtype=torch.int32, device="cuda")

    def one():
        L.route(gate, case.logits, None, None, load)
        L.forward_routed(case.x_seg, case.out_seg)
        mok.mok_layer_bwd(case.d, case.dout_seg, case.x_seg, L.w, L.idx, L.p, L.saved, L.ring, L.slots,
                          case.dx_seg, case.dp, None, case.dwg, case.dwu, case.dwd, case.bws)
        L.route_backward(gate, case.logits, case.dp, dl)

    one()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    outs = lambda: [t.clone() for t in (L.idx, L.p, load, case.out, case.dx, case.dp, dl, case.dwg, case.dwd)]
    for k in range(4):
        case.logits.copy_(torch.randn(cfg.N, cfg.E, generator=torch.Generator().manual_seed(k)))
        graph.replay()
        torch.cuda.synchronize()
        got = outs()
        one()
        torch.cuda.synchronize()
        assert mok.mok_device_status(L.ws) == 0 and mok.mok_device_status(case.bws) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, outs()))


def test_given_choice_host_refusals():
    lib, d = mok.lib(), mok.desc_from_config(TINY)
    w = mok.MokWeights()
    P = 4096
    for k in range(4):
        args = [P] * 4
        args[k] = None
        assert lib.mok_schedule_routed(ctypes.byref(d), *args, None) == 1
    assert lib.mok_schedule_routed(ctypes.byref(d), P, P, P + 8, P, None) == 4
    assert lib.mok_layer_fwd_routed(ctypes.byref(d), P, ctypes.byref(w), P, P, P, P, P, P, P, None) == 1
    assert lib.mok_layer_fwd_routed(ctypes.byref(d), P, None, P, P, P, P, P, P, P, None) == 1


@pytest.mark.parametrize("state", ["float32", "mxfp8"])
@pytest.mark.parametrize("name", ["tiny", "wide", "mx"])
def test_training_steps(name, state):
    """Two steps of everything. Each stage is compared with the oracle on the inputs that it had."""
    cfg = CFGS[name]
    groups = 4 if cfg.E >= 16 else 2
    gate = orr.Gate(cfg.E, cfg.K, "sigmoid", groups, groups // 2, "top2", True, 2.5)
    desc = mok.route_desc(cfg.E, cfg.K, "sigmoid", groups, groups // 2, "top2", True, 2.5)
    case = BwdCase(cfg, staged=False, fused=True)
    L, N = case.layer, cfg.N
    f32 = lambda t: t.view(torch.bfloat16).float()
    wr = dev_u16(datagen.router_weight(cfg))
    copies = [case.wg, case.wu, case.wd, wr]
    masters = [f32(t) for t in copies]
    dwr = torch.empty(cfg.E, cfg.H, device="cuda")
    grads = [case.dwg, case.dwu, case.dwd, dwr]
    opt = MokAdamW(masters, grads, [t.view(torch.bfloat16) for t in copies], lr=1e-2, weight_decay=0.1,
                   max_norm=1.0, state=state)
    bias = (0.01 * torch.randn(cfg.E, generator=torch.Generator().manual_seed(1))).cuda()
    mask = (torch.arange(N, device="cuda") % 7 != 3).to(torch.uint8)
    logits, dlogits = torch.empty(N, cfg.E, device="cuda"), torch.empty(N, cfg.E, device="cuda")
    load = torch.empty(cfg.E, dtype=torch.int32, device="cuda")
    rws = torch.empty(mok.router_ws_size(case.d), dtype=torch.uint8, device="cuda")
    for step in (1, 2):
        before = [t.clone() for t in masters]
        moments = [(m.clone(), v.clone()) for m, v in zip(opt.m, opt.v)]
        mok.mok_router_fwd(case.d, case.x_seg, wr, logits)
        L.route(desc, logits, bias, mask, load)
        L.forward_routed(case.x_seg, case.out_seg)
        case.dx.zero_()
        mok.mok_layer_bwd(case.d, case.dout_seg, case.x_seg, L.w, L.idx, L.p, L.saved, L.ring, L.slots,
                          case.dx_seg, case.dp, None, case.dwg, case.dwu, case.dwd, case.bws)
        L.route_backward(desc, logits, case.dp, dlogits)
        dx_layer = case.dx.clone()
        mok.mok_router_bwd(case.d, case.x_seg, wr, dlogits, dwr, case.dx_seg, rws)
        wr_h, w_h = host_u16(wr).copy(), {k: host_u16(getattr(case, k)).copy() for k in ("wg", "wu", "wd")}
        opt.step()
        L.refresh_weights()
        torch.cuda.synchronize()
        assert mok.mok_device_status(L.ws) == 0 and mok.mok_device_status(case.bws) == 0
        # the gate, on the logits that it had
        x64 = logits.double().cpu().numpy()
        idx, w, ld = orr.forward(gate, x64, bias.double().cpu().numpy(), mask.cpu().numpy())
        gi, gp = case.idx_p()
        assert np.array_equal(gi, idx) and np.array_equal(load.cpu().numpy(), ld)
        assert max_rel_err(gp.astype(np.float64), w) <= 1e-5
        # the layer, on that choice and the weights before the step
        case.w_h = w_h
        fw, W = oracle_of(case, idx, gp.astype(np.float64))
        bw = mo.backward(fw, mo.bf16_rows(case.dout_h), W, cfg.K, cfg.e0, cfg.E_loc, cfg.E + 1)
        err, tol = (max_rel_err, BF16_TOL) if cfg.dtype == "bf16" else (frob_rel_err, MX_TOL)
        assert err(case.out_rows(fw.sched.touched), fw.out) <= tol
        assert err(mo.decode_bf16(host_u16(dx_layer))[fw.sched.touched], bw.dx) <= tol
        # the gate's and the projection's gradients, from the layer's dp
        dp = np.where(idx >= 0, case.dp.double().cpu().numpy().reshape(N, cfg.K), 0)
        dl = orr.backward(gate, x64, idx, dp)
        assert max_rel_err(dlogits.double().cpu().numpy(), dl) <= 1e-5
        dwr_o, _ = mo.router_backward(mo.decode_bf16(case.x_h), mo.decode_bf16(wr_h), dl)
        assert max_rel_err(dwr.double().cpu().numpy(), dwr_o) <= BF16_TOL
        # the step, on the gradients that it had
        g64 = [t.double().cpu().numpy().ravel() for t in grads]
        sumsq = sum(float((g * g).sum()) for g in g64)
        assert abs(opt.sumsq.item() - sumsq) <= 1e-10 * sumsq
        if state == "float32":
            for p0, p1, (m, v), g, c in zip(before, masters, moments, grads, copies):
                n = lambda t: t.cpu().numpy().ravel()
                ref = oo.step32(n(p0), n(g), n(m), n(v), 1e-2, 0.9, 0.999, 1e-8, 0.1, step, opt.sumsq.item(), 1.0)
                assert np.array_equal(n(p1), ref[0])
                assert torch.equal(c.view(torch.bfloat16), p1.bfloat16())
        assert any(not torch.equal(a, b) for a, b in zip(before, masters))
