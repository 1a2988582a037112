"""Cases that measure the gate of the routed layer and the optimizer step: the choice of experts and
its gradient, the squared norm of all gradients, and AdamW over many tensors.

`run` computes an operator in elementary torch operations, or, with `own` true, by the framework's
calls. Shapes are those of this repository's workloads (its tiny test layer, the DeepSeek-V3- and
Kimi-K2-shaped shares) and generic odd ones.
"""
import math

import torch

own = False

INF = float("inf")
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------------------------- the cases

def _route(name, op, tokens, experts, top_k, score, groups=1, top_groups=1, group_score="max",
           bias=False, renorm=True, scale=1.0, dtype="float32", pad=0, masked=0.0, holes=0.0):
    case = dict(op=op, tokens=tokens, experts=experts, top_k=top_k, score=score, groups=groups,
                top_groups=top_groups, group_score=group_score, bias=bias, renorm=renorm,
                scale=scale, dtype=dtype, pad=pad, masked=masked, holes=holes)
    return dict(case, name=name) if name else case


def _step(name, op, layout, **kw):
    case = dict(op=op, grad="float32", param="float32", copy=True, state="float32", clip=False,
                step=100, tensors=0, total=0, experts=0, hidden=0, inter=0, routed=0)
    case.update(layout)
    case.update(kw)
    return dict(case, name=name) if name else case


TINY = dict(experts=8, hidden=128, inter=256, routed=8)          # the tiny test layer
DSV3 = dict(experts=4, hidden=7168, inter=2048, routed=256)      # one GPU's share, DeepSeek-V3 shapes
KIMI = dict(experts=6, hidden=7168, inter=2048, routed=384)      # one GPU's share, Kimi-K2 shapes


def listed():
    return [
        # the tiny test layer's gate: the smallest call, where latency counts
        _route("route_tiny", "route_fwd", 64, 8, 2, "softmax"),
        # all 64 x 2048 source tokens of the DeepSeek-V3-shaped workload, its gate
        _route("route_dsv3", "route_fwd", 131072, 256, 8, "sigmoid", 8, 4, "top2", True, True, 2.5),
        # the Kimi-K2-shaped workload, logits of a bf16 projection
        _route("route_kimi_bf16", "route_fwd", 131072, 384, 8, "sigmoid", 1, 1, "max", True, True, 2.5,
               "bfloat16"),
        # an ordinary batch with a padded tail, experts masked per token, odd sizes, strided rows,
        # plain softmax weights
        _route("route_softmax_odd", "route_fwd", 5003, 60, 4, "softmax", 1, 1, "max", False, False, 1.0,
               "float32", 5, 0.1, 0.05),
        # gradients of two of them at training size
        _route("route_bwd_dsv3", "route_bwd", 131072, 256, 8, "sigmoid", 8, 4, "top2", True, True, 2.5),
        _route("route_bwd_softmax", "route_bwd", 20011, 384, 6, "softmax", 1, 1, "max", False, False, 1.0,
               "bfloat16", 0, 0.1, 0.05),
        # the optimizer step of the tiny test layer: latency
        _step("adamw_tiny", "adamw", TINY),
        # the optimizer step of one GPU's share, clipped by the norm of all gradients
        _step("adamw_dsv3", "adamw", DSV3, clip=True),
        # the larger share with its states in 8 bits
        _step("adamw_mx8_kimi", "adamw", KIMI, state="mx8"),
        # many small tensors of odd sizes, bf16 gradients and parameters without an fp32 master
        _step("adamw_mx8_ragged", "adamw", {}, tensors=37, total=3_000_000, grad="bfloat16",
              param="bfloat16", copy=False, state="mx8", clip=True),
        # the norm that clips
        _step("sumsq_ragged", "sumsq", {}, tensors=37, total=3_000_000, grad="bfloat16"),
        _step("sumsq_dsv3", "sumsq", DSV3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route_fwd", "route_fwd", "route_bwd", "adamw", "adamw", "sumsq"])
    if op.startswith("route"):
        groups = rng.choice([1, 1, 1, 2, 4, 8, 16])
        size = _log(rng, 4, max(5, min(384, 1024 // groups)))
        experts = groups * size
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, top_groups * size))
        tokens = _log(rng, 1, min(131072, 30_000_000 // experts))
        score = rng.choice(["sigmoid", "softmax"])
        return _route(None, op, tokens, experts, top_k, score, groups, top_groups,
                      rng.choice(["max", "top2"]), rng.random() < 0.5, rng.random() < 0.6,
                      rng.choice([1.0, 2.5]), rng.choice(["float32", "bfloat16"]),
                      rng.choice([0, 0, 3, 8]), rng.choice([0.0, 0.1]), rng.choice([0.0, 0.05]))
    if rng.random() < 0.4:
        hidden = 128 * _log(rng, 1, 56)
        inter = 128 * _log(rng, 1, 16)
        layout = dict(experts=rng.randint(1, 4), hidden=hidden, inter=inter, routed=rng.choice([8, 60, 256]))
    else:
        tensors = _log(rng, 1, 150)
        layout = dict(tensors=tensors, total=max(tensors * 8, _log(rng, 2000, 30_000_000)))
    grad = rng.choice(["float32", "bfloat16"])
    if op == "sumsq":
        return _step(None, op, layout, grad=grad)
    param = rng.choice(["float32", "float32", "bfloat16"])
    return _step(None, op, layout, grad=grad, param=param, copy=param == "float32" and rng.random() < 0.7,
                 state=rng.choice(["float32", "mx8"]), clip=rng.random() < 0.5, step=rng.choice([1, 7, 100, 20000]))


def work(case):
    if case["op"].startswith("route"):
        n, e, k = case["tokens"], case["experts"], case["top_k"]
        b = 4 if case["dtype"] == "float32" else 2
        live = n - int(n * case["masked"])
        if case["op"] == "route_fwd":
            return {"bytes": live * e * b + n * k * 8 + 4 * e * (1 + case["bias"]) + (n if case["masked"] else 0),
                    "flops": 8 * live * e}
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": n * e * b + live * (e if dense else k) * b + n * k * 4 + live * k * 4,
                "flops": live * (6 * e if dense else 12 * k)}
    n = sum(_sizes(case))
    g = 4 if case["grad"] == "float32" else 2
    if case["op"] == "sumsq":
        return {"bytes": n * g + 8, "flops": 2 * n}
    p = 4 if case["param"] == "float32" else 2
    s = 8 if case["state"] == "float32" else 2 + 2 / 32
    return {"bytes": n * (g + 2 * p + 2 * s + 2 * case["copy"]), "flops": 14 * n}


# ----------------------------------------------------------------------------------- the inputs

def _sizes(case):
    """Elements of each tensor: the layer's weights and its router, or sizes spread over two decades."""
    if not case["tensors"]:
        m = case["experts"] * case["hidden"] * case["inter"]
        return [m, m, m, case["routed"] * case["hidden"]]
    n = case["tensors"]
    part = [math.exp(4.6 * ((7 * i + 3) % n) / n) for i in range(n)]
    return [max(1, int(case["total"] * p / sum(part)) | 1) for p in part]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"].startswith("route"):
        return _prepare_route(case, g)
    sizes = _sizes(case)
    # every tensor begins at a multiple of 256 elements of one flat buffer; what lies between is zero
    padded = [-(-n // 256) * 256 for n in sizes]
    starts = [sum(padded[:i]) for i in range(len(sizes))]
    total = sum(padded)
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, n in zip(starts, sizes):
        live[a:a + n] = True
    rand = lambda std: torch.randn(total, generator=g, device="cuda").mul_(std).mul_(live)
    st = dict(case=case, sizes=sizes, padded=padded, starts=starts)
    # gradients of very different sizes, as those of early and late training steps and rare experts
    st["g"] = (rand(1e-3) * torch.exp(2 * torch.randn(total, generator=g, device="cuda"))).to(getattr(torch, case["grad"]))
    views = lambda t: [t[a:a + n] for a, n in zip(starts, sizes)]
    if case["op"] == "sumsq":
        if own:
            import combine_router_top_schedule_amd as mok
            st["out"] = torch.zeros(1, dtype=torch.float64, device="cuda")
            st["plan"] = mok.sumsq_plan(views(st["g"]))
        return st
    st["p"] = rand(0.02).to(getattr(torch, case["param"]))
    st["copy"] = st["p"].bfloat16() if case["copy"] else None
    m, r = rand(5e-4), rand(2e-3).abs_()
    if case["state"] == "mx8":
        zero = torch.zeros(total, dtype=torch.int64, device="cuda")
        (st["m"], st["ms"]), (st["v"], st["vs"]) = _encode(m, zero, False), _encode(r, zero, True)
    else:
        st["m"], st["v"] = m, r.square_()
    st["sumsq"] = st["g"].double().square().sum().reshape(1) if case["clip"] else None
    st["hyper"] = dict(lr=2e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=case["step"],
                       seed=1 + case["step"], max_norm=1.0)
    if own:
        import combine_router_top_schedule_amd as mok
        scale = lambda k: [st[k][a // 32:a // 32 + -(-n // 32)] for a, n in zip(starts, sizes)]
        kw = dict(m_scale=scale("ms"), v_scale=scale("vs")) if case["state"] == "mx8" else {}
        st["plan"] = mok.adamw_plan(p=views(st["p"]), g=views(st["g"]), m=views(st["m"]), v=views(st["v"]),
                                    copy=views(st["copy"]) if case["copy"] else None, **kw)
    return st


def _prepare_route(case, g):
    n, e, k = case["tokens"], case["experts"], case["top_k"]
    dt = getattr(torch, case["dtype"])
    wide = torch.randn(n, e + case["pad"], generator=g, device="cuda")
    if case["holes"]:   # experts that a token may not take
        wide.masked_fill_(torch.rand(wide.shape, generator=g, device="cuda") < case["holes"], -INF)
    mask = None
    if case["masked"]:  # padded tokens: what their rows hold means nothing
        mask = torch.rand(n, generator=g, device="cuda") >= case["masked"]
        wide[~mask] = float("nan")
    st = dict(case=case, x=wide.to(dt)[:, :e], mask=None if mask is None else mask.to(torch.uint8))
    # a bias that signed steps of 0.001 have built up
    st["bias"] = torch.randn(e, generator=g, device="cuda").mul_(20).round_().mul_(1e-3) if case["bias"] else None
    if case["op"] == "route_fwd":
        st["idx"] = torch.empty(n, k, dtype=torch.int32, device="cuda")
        st["w"] = torch.empty(n, k, device="cuda")
        st["load"] = torch.empty(e, dtype=torch.int32, device="cuda")
    else:
        st["idx"] = _choose(case, st["x"], st["bias"], st["mask"])
        st["dw"] = torch.randn(n, k, generator=g, device="cuda")
        st["dx"] = torch.empty(n, e, dtype=dt, device="cuda")
    if own:
        import combine_router_top_schedule_amd as mok
        st["desc"] = mok.route_desc(E=e, K=k, score=case["score"], groups=case["groups"],
                                    top_groups=case["top_groups"], group_score=case["group_score"],
                                    renorm=case["renorm"], scale=case["scale"])
    return st


# -------------------------------------------------------------------------------- the operators

def run(st):
    return {"route_fwd": _route_fwd, "route_bwd": _route_bwd, "adamw": _adamw, "sumsq": _sumsq}[st["case"]["op"]](st)


def _choose(case, x, bias, mask):
    """The chosen experts, best first, -1 where none is left. Keys are compared in 64 bits: two of
    a few million scores are often closer than 32 bits tell apart."""
    n, e, k, groups = case["tokens"], case["experts"], case["top_k"], case["groups"]
    x = x.double()
    if mask is not None:
        x = torch.where(mask[:, None] != 0, x, -INF)
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
    else:
        z = torch.exp(x - x.amax(1, keepdim=True))
        s = z / z.sum(1, keepdim=True)
    biased = s if bias is None else s + bias
    key = x if bias is None else biased     # a score rises with its logit
    able = (x > -INF) & (key > -INF)
    key = torch.where(able, key, -INF)
    if groups > 1:
        if case["group_score"] == "top2":
            two = torch.sort(torch.where(able, biased, -INF).view(n, groups, -1), -1, descending=True)[0][..., :2]
            best = torch.where(two[..., 0] > -INF, torch.where(two > -INF, two, 0.0).sum(-1), -INF)
        else:
            best = key.view(n, groups, -1).amax(-1)
        kept = torch.sort(best, dim=-1, descending=True, stable=True)[1][:, :case["top_groups"]]
        open_ = torch.zeros(n, groups, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        key = torch.where(open_.repeat_interleave(e // groups, 1), key, -INF)
    val, idx = torch.sort(key, dim=-1, descending=True, stable=True)
    return torch.where(val[:, :k] > -INF, idx[:, :k], -1).to(torch.int32)


def _chosen(x, idx):
    """Logits at the chosen experts, and where there are any."""
    some = idx >= 0
    return torch.where(some, x.gather(1, idx.clamp_min(0).long()), -INF), some


def _route_fwd(st):
    case = st["case"]
    if own:
        import combine_router_top_schedule_amd as mok
        mok.mok_route_fwd(st["desc"], st["x"], st["idx"], st["w"], bias=st["bias"], token_mask=st["mask"],
                          load=st["load"])
        return {"idx": st["idx"], "w": st["w"], "load": st["load"]}
    idx = _choose(case, st["x"], st["bias"], st["mask"])
    x = st["x"].float()
    xk, some = _chosen(x, idx)
    if case["renorm"]:
        s = _ratio(case, xk)
    elif case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-xk))
    else:
        top = x.amax(1, keepdim=True)
        s = torch.exp(xk - top) / torch.exp(x - top).sum(1, keepdim=True)
    w = torch.where(some, s * case["scale"], 0.0)
    load = (idx.reshape(-1, 1) + 1).flatten().long()
    load = torch.zeros(case["experts"] + 1, dtype=torch.int64, device=x.device).index_add_(
        0, load, torch.ones_like(load))[1:]
    return {"idx": idx, "w": w, "load": load.to(torch.int32)}


def _ratio(case, xk):
    """Scores of the chosen over their sum: a softmax of the logits, or of log sigmoid of them."""
    f = xk if case["score"] == "softmax" else torch.clamp(xk, max=0) - torch.log1p(torch.exp(-xk.abs()))
    q = torch.exp(f - f.amax(1, keepdim=True))
    return q / q.sum(1, keepdim=True)


def _route_bwd(st):
    case, idx = st["case"], st["idx"]
    if own:
        import combine_router_top_schedule_amd as mok
        mok.mok_route_bwd(st["desc"], st["x"], idx, st["dw"], st["dx"])
        return {"dx": st["dx"]}
    x, c = st["x"].float(), case["scale"]
    xk, some = _chosen(x, idx)
    dw = torch.where(some, st["dw"], 0.0)
    if case["renorm"]:
        q = torch.where(some, _ratio(case, xk), 0.0)
        d = c * q * (dw - (dw * q).sum(1, keepdim=True))
        d = d if case["score"] == "softmax" else d / (1 + torch.exp(xk))
    elif case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-xk))
        d = c * dw * s / (1 + torch.exp(xk))
    else:
        top = x.amax(1, keepdim=True)
        s = torch.exp(x - top)
        s = s / s.sum(1, keepdim=True)
        sk = torch.where(some, s.gather(1, idx.clamp_min(0).long()), 0.0)
        d = c * dw * sk
        rest = torch.where(some.any(1, keepdim=True), s * d.sum(1, keepdim=True), 0.0)
    dx = torch.zeros_like(x).scatter_add_(1, idx.clamp_min(0).long(), torch.where(some, d, 0.0))
    if not case["renorm"] and case["score"] == "softmax":
        dx = dx - rest
    return {"dx": dx.to(st["dx"].dtype)}


def _sumsq(st):
    if own:
        import combine_router_top_schedule_amd as mok
        mok.mok_grad_sumsq(st["plan"], st["out"])
        return {"sumsq": st["out"]}
    return {"sumsq": st["g"].double().square().sum().reshape(1)}


def _mix(h):
    h = h ^ (h >> 16)
    h = (h * 0x6A09E667) & M32
    h = h ^ (h >> 15)
    h = (h * 0xBB67AE85) & M32
    return h ^ (h >> 16)


def _bits(st):
    """32 random bits for every element: a hash of the seed, the tensor's number and the element's."""
    dev = st["p"].device
    lens = torch.tensor(st["padded"], device=dev)
    number = torch.arange(len(st["sizes"]), device=dev)
    base = _mix(_mix((st["hyper"]["seed"] + number * 0x9E3779B1) & M32))
    begin = torch.tensor(st["starts"], device=dev)
    at = torch.arange(st["p"].numel(), device=dev) - begin.repeat_interleave(lens)
    return _mix((at & M32) ^ base.repeat_interleave(lens))


def _pow2(e):
    return torch.ldexp(torch.ones((), device=e.device), e)


def _encode(x, u, positive):
    """E4M3 codes and UE8M0 scales, one for 32 values: the smallest power of two that keeps the
    block's largest value at most 448. Rounds up where the rest is over 1 - u / 65536; with
    `positive`, what is not zero does not become zero."""
    blocks = x.view(-1, 32)
    amax = blocks.abs().amax(1)
    man, ex = torch.frexp(amax)                       # amax = man 2^ex, man in [0.5, 1)
    ex = (ex - 9 + (man > 0.875)).clamp(-127, 127)
    ex = torch.where(amax > 0, ex, -127)
    a = blocks.abs() * _pow2(-ex)[:, None]
    q = torch.frexp(a)[1].clamp_min(-5) - 4           # a code's step is 2^q
    k = torch.floor(a * _pow2(-q) + u.view(-1, 32).float() * 2.0 ** -16)
    if positive:
        k = torch.where(a > 0, k.clamp_min(1), k)
    code = torch.copysign(k * _pow2(q), blocks).to(torch.float8_e4m3fn)
    return code.view(torch.uint8).view(-1), (ex + 127).to(torch.uint8)


def _decode(code, scale):
    v = code.view(torch.float8_e4m3fn).float().view(-1, 32)
    return (v * _pow2(scale.int() - 127)[:, None]).view(-1)


def _adamw(st):
    case, h = st["case"], st["hyper"]
    if own:
        import combine_router_top_schedule_amd as mok
        mok.mok_adamw(st["plan"], lr=h["lr"], beta1=h["beta1"], beta2=h["beta2"], eps=h["eps"],
                      weight_decay=h["weight_decay"], step=h["step"], seed=h["seed"], sumsq=st["sumsq"],
                      max_norm=h["max_norm"] if case["clip"] else None)
        return _outputs(st)
    g, p = st["g"].float(), st["p"].float()
    if case["clip"]:
        g = g * torch.clamp(h["max_norm"] / st["sumsq"].sqrt(), max=1.0).float()
    mx = case["state"] == "mx8"
    r0 = _decode(st["v"], st["vs"]) if mx else None
    m = (_decode(st["m"], st["ms"]) if mx else st["m"]) * h["beta1"] + g * (1 - h["beta1"])
    v = (r0 * r0 if mx else st["v"]) * h["beta2"] + (g * g) * (1 - h["beta2"])
    r = torch.sqrt(v)
    down1, down2 = 1 - h["beta1"] ** h["step"], 1 - h["beta2"] ** h["step"]
    den = r * (1 / math.sqrt(down2)) + h["eps"]
    p = p * (1 - h["lr"] * h["weight_decay"]) - (m / den) * (h["lr"] / down1)
    bits = _bits(st) if mx or case["param"] == "bfloat16" else None
    if case["param"] == "bfloat16":
        up = p.view(torch.int32).long() + (_mix(bits ^ 0x3C6EF372) & 0xFFFF)
        st["p"].copy_((up & ~0xFFFF).to(torch.int32).view(torch.float32))
    else:
        st["p"].copy_(p)
        if case["copy"]:
            st["copy"].copy_(p)
    if mx:
        for code, scale, x, u in (("m", "ms", m, bits & 0xFFFF), ("v", "vs", r, bits >> 16)):
            c, s = _encode(x, u, code == "v")
            st[code].copy_(c)
            st[scale].copy_(s)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    return _outputs(st)


def _outputs(st):
    """Parameters and states; 8-bit codes and scales as the float8 values that they are."""
    out = {"p": st["p"]}
    if st["case"]["copy"]:
        out["copy"] = st["copy"]
    if st["case"]["state"] == "mx8":
        for k, t in (("m", torch.float8_e4m3fn), ("v", torch.float8_e4m3fn), ("ms", torch.float8_e8m0fnu),
                     ("vs", torch.float8_e8m0fnu)):
            out[k] = st[k].view(t)
    else:
        out["m"], out["v"] = st["m"], st["v"]
    return out


# -------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route_fwd":
        return _exact_fwd(case, st)
    if case["op"] == "route_bwd":
        return _exact_bwd(case, st)
    if case["op"] == "sumsq":
        parts = [torch.dot(a, a) for a in st["g"].double().split(1 << 20)]
        return {"sumsq": torch.stack(parts).sum().reshape(1)}
    return _exact_adamw(case, st)


def _exact_fwd(case, st):
    """Choice by taking the largest key away K times; weights as quotients of scores."""
    n, e, k = case["tokens"], case["experts"], case["top_k"]
    x = st["x"].to(torch.float64)
    live = torch.ones(n, 1, dtype=torch.bool, device=x.device) if st["mask"] is None else st["mask"].bool()[:, None]
    x = x.masked_fill(~live, -INF)
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    s = torch.where(live, s, 0.0)
    key = (s + st["bias"].double()) if case["bias"] else s.clone()
    rank = key if case["bias"] else x
    dead = ~((x > -INF) & (rank > -INF))
    number = torch.arange(e, device=x.device)
    if case["groups"] > 1:
        size = e // case["groups"]
        by = (key if case["group_score"] == "top2" else rank).masked_fill(dead, -INF).view(n, case["groups"], size)
        one, at = by.max(-1)
        if case["group_score"] == "top2":
            first = (by == one[..., None]).to(torch.int8).argmax(-1, keepdim=True)
            two = by.scatter(-1, first, -INF).amax(-1)
            one = one + torch.where(two > -INF, two, 0.0)
        order = torch.argsort(-one, dim=1, stable=True)
        place = torch.empty_like(order).scatter_(1, order, torch.arange(case["groups"], device=x.device).expand(n, -1).contiguous())
        dead = dead | (place >= case["top_groups"]).unsqueeze(-1).expand(-1, -1, size).reshape(n, e)
    left = rank.masked_fill(dead, -INF)
    picks = []
    for _ in range(k):
        top = left.amax(1, keepdim=True)
        i = torch.where(left == top, number, e).amin(1, keepdim=True)
        picks.append(torch.where(top > -INF, i, -1))
        left = left.scatter(1, i.clamp(max=e - 1), -INF)
    idx = torch.cat(picks, 1)
    w = torch.where(idx >= 0, s.gather(1, idx.clamp_min(0)), 0.0)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    w = w * case["scale"]
    load = torch.bincount(idx[idx >= 0].reshape(-1), minlength=e)
    return {"idx": idx, "w": w, "load": load}


def _exact_bwd(case, st):
    """Quotient rule on the scores, then the scores' own derivatives."""
    n, e = case["tokens"], case["experts"]
    hit = torch.zeros(n, e + 1, dtype=torch.float64, device="cuda").scatter_(1, torch.where(st["idx"] < 0, e, st["idx"]).long(), 1.0)[:, :e]
    dw = torch.zeros(n, e + 1, dtype=torch.float64, device="cuda").scatter_(1, torch.where(st["idx"] < 0, e, st["idx"]).long(), st["dw"].double())[:, :e]
    any_ = hit.sum(1, keepdim=True) > 0
    x = torch.where(any_, st["x"].double(), 0.0)
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    ds = dw * hit * case["scale"]
    if case["renorm"]:
        z = (s * hit).sum(1, keepdim=True)
        z = torch.where(z > 0, z, 1.0)
        ds = hit * (ds * z - (ds * s).sum(1, keepdim=True)) / z ** 2
    if case["score"] == "sigmoid":
        dx = ds * s * (1 - s)
    else:
        dx = s * (ds - (s * ds).sum(1, keepdim=True))
    return {"dx": torch.where(any_, dx, 0.0)}


def _exact_adamw(case, st):
    h, f64 = st["hyper"], torch.float64
    mx = case["state"] == "mx8"
    g = st["g"].to(f64)
    if case["clip"]:
        g = g * min(1.0, h["max_norm"] / math.sqrt(float(st["sumsq"])))
    if mx:
        widen = lambda c, s: (st[c].view(torch.float8_e4m3fn).to(f64).view(-1, 32) * torch.pow(
            torch.tensor(2.0, dtype=f64, device="cuda"), st[s].to(f64) - 127)[:, None]).view(-1)
        m, v = widen("m", "ms"), widen("v", "vs") ** 2
    else:
        m, v = st["m"].to(f64), st["v"].to(f64)
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
    mhat = m / (1 - h["beta1"] ** h["step"])
    vhat = v / (1 - h["beta2"] ** h["step"])
    p = st["p"].to(f64)
    p = p - h["lr"] * h["weight_decay"] * p - h["lr"] * mhat / (vhat.sqrt() + h["eps"])
    out = {"p": p}
    bits = None
    if mx or case["param"] == "bfloat16":
        bits = torch.empty(p.numel(), dtype=torch.int64, device="cuda")
        for t, (a, n) in enumerate(zip(st["starts"], st["padded"])):
            salt = _mix(_mix(torch.tensor((h["seed"] + t * 0x9E3779B1) % 2 ** 32, device="cuda")))
            bits[a:a + n] = _mix(torch.arange(n, device="cuda") ^ salt)
    if case["param"] == "bfloat16":
        ulp = torch.pow(torch.tensor(2.0, dtype=f64, device="cuda"), torch.floor(torch.log2(p.abs().clamp_min(1e-38))) - 7)
        u = (_mix(bits ^ 0x3C6EF372) % 65536).to(f64) / 65536
        out["p"] = torch.sign(p) * torch.floor(p.abs() / ulp + u) * ulp
    if case["copy"]:
        out["copy"] = p
    if not mx:
        out["m"], out["v"] = m, v
        return out
    for c, s, x, u in (("m", "ms", m, bits % 65536), ("v", "vs", v.sqrt(), bits // 65536)):
        b = x.view(-1, 32)
        top = b.abs().amax(1, keepdim=True)
        e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp_min(1e-300) / 448)), -127.0)
        e = torch.where(top > 448 * torch.exp2(e), e + 1, e)      # (a logarithm may be off by its last bit)
        e = torch.where((top > 0) & (top <= 448 * torch.exp2(e - 1)), e - 1, e).clamp(-127, 127)
        a = b.abs() / torch.exp2(e)
        step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
        k = torch.floor(a / step + u.view(-1, 32).to(f64) / 65536)
        k = torch.where((a > 0) & (k < 1) & (c == "v"), 1.0, k)
        out[c] = (torch.sign(b) * k * step).view(-1)
        out[s] = torch.exp2(e).view(-1)
    return out
