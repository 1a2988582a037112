"""Cases that measure the experts' linear maps in block-scaled FP8 and their optimizer: quantising with
one scale for 128 values (rows, rows turned to columns for the weight gradient, weights in blocks of
128 x 128), the product of token rows sorted by expert with the experts' weights, the weight gradient,
and Muon's orthogonalised update.

`run` computes an operator in elementary torch operations, or, with `own` true, by the framework's
calls. Shapes are those of this repository's workloads (its tiny test layer, the DeepSeek-V3- and
Kimi-K2-shaped shares) and generic odd ones.
"""
import math

import torch

own = False

B = 128                       # values a scale stands for, along the product's sum
TOP = 448.0                   # largest E4M3 value
LEAST = 2.0 ** -100           # smaller largest values of a block count as this
JORDAN = (3.4445, -4.7750, 2.0315)


# ------------------------------------------------------------------------------------- the cases

def _case(name, op, **kw):
    case = dict(op=op, rows=0, groups=1, tail=0, n=0, k=0, dtype="bfloat16", both=False, accumulate=False)
    case.update(kw)
    return dict(case, name=name) if name else case


def _muon(name, op, shapes, **kw):
    """`shapes`: batch x rows x cols of each tensor, separated by spaces."""
    case = dict(op=op, shapes=shapes, grad="float32", copy=True, clip=False, nesterov=True,
                adjust="rms", dtype="bfloat16")
    case.update(kw)
    return dict(case, name=name) if name else case


TINY = "8x256x128 8x256x128 8x128x256 1x8x128"                      # the tiny test layer and its router
DSV3 = "4x2048x7168 4x2048x7168 4x7168x2048 1x256x7168"             # one GPU's share, DeepSeek-V3 shapes


def listed():
    return [
        # one token on its way into an FP8 product: latency
        _case("quant_one", "quant", rows=1, k=7168),
        # the rows that the DeepSeek-V3-shaped share of 4 experts gets of 131,072 tokens, for the forward
        # product (along the row) and the weight gradient (along the tokens of each expert) at once
        _case("quant_dsv3", "quant", rows=16384, groups=4, k=7168, both=True),
        # that share's gate and up weights after an optimizer step, fp32 masters, for both products
        _case("quant_weights_dsv3", "quant_w", groups=4, n=4096, k=7168, dtype="float32", both=True),
        # one token through one expert's gate and up: decoding alone
        _case("gemm_one", "gemm", rows=1, n=4096, k=7168),
        # a decoding batch over the Kimi-K2-shaped share of 6 experts, down product
        _case("gemm_decode_kimi", "gemm", rows=44, groups=6, n=7168, k=2048),
        # gate and up of the DeepSeek-V3-shaped share in training
        _case("gemm_dsv3", "gemm", rows=16384, groups=4, n=4096, k=7168),
        # odd sizes everywhere, an expert without rows, rows behind the last expert, fp32 out
        _case("gemm_odd", "gemm", rows=5003, groups=7, tail=17, n=1001, k=1416, dtype="float32"),
        # weight gradient of the DeepSeek-V3-shaped share's down projection
        _case("wgrad_dsv3", "wgrad", rows=16384, groups=4, n=7168, k=2048),
        # odd sizes, added to the gradient of an earlier micro-batch
        _case("wgrad_odd", "wgrad", rows=3001, groups=7, tail=17, n=1001, k=712, accumulate=True),
        # the optimizer step of the tiny test layer: latency
        _muon("muon_tiny", "muon", TINY),
        # the optimizer step of one GPU's share, clipped by the norm of all gradients
        _muon("muon_dsv3", "muon", DSV3, clip=True),
        # updates of many odd shapes orthogonalised alone, as a sharded optimizer does
        _muon("orthogonalize_odd", "orth", "3x333x129 1x60x1000 2x700x701 1x1x500 5x129x64 1x1500x130"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "quant_w", "gemm", "gemm", "gemm", "wgrad", "wgrad", "muon", "muon", "orth"])
    if op in ("muon", "orth"):
        shapes, left = [], 60_000_000_000 if rng.random() < 0.3 else 4_000_000_000
        for _ in range(rng.choice([1, 2, 3, 6, 12])):
            r, c, b = _log(rng, 1, 2500), _log(rng, 1, 5000), _log(rng, 1, 8)
            cost = b * min(r, c) ** 2 * max(r, c)
            if cost <= left:
                left -= cost
                shapes.append(f"{b}x{r}x{c}")
        shapes = " ".join(shapes) or f"{rng.randint(1, 5)}x{_log(rng, 2, 900)}x{_log(rng, 2, 900)}"
        if op == "orth":
            return _muon(None, op, shapes, dtype=rng.choice(["bfloat16", "float32"]))
        return _muon(None, op, shapes, grad=rng.choice(["float32", "bfloat16"]), copy=rng.random() < 0.7,
                     clip=rng.random() < 0.5, nesterov=rng.random() < 0.7,
                     adjust=rng.choice(["rms", "spectral", "none"]))
    groups = rng.choice([1, 1, 2, 4, 6, 16, 64])
    wide = lambda: rng.choice([_log(rng, 1, 8000), 128 * _log(rng, 1, 60)])
    n, k = wide(), wide()
    if op == "quant_w":
        while groups * n * k > 4 * 4096 * 7168:
            groups = max(1, groups // 2)
            n = max(1, n // 2)
        return _case(None, op, groups=groups, n=n, k=k, dtype=rng.choice(["bfloat16", "float32"]),
                     both=rng.random() < 0.6)
    while groups * n * k > 16 * 2048 * 7168:
        groups = max(1, groups // 2)
        n = max(1, n // 2)
    rows = _log(rng, 1, max(1, min(16384, 16384 * 4096 * 7168 // (n * k))))
    tail = rng.choice([0, 0, 0, 5]) if rows > 8 else 0
    if op == "quant":
        return _case(None, op, rows=rows, groups=groups, tail=tail, k=k, both=rng.random() < 0.6,
                     dtype=rng.choice(["bfloat16", "float32"]))
    return _case(None, op, rows=rows, groups=groups, tail=tail, n=n, k=k,
                 dtype=rng.choice(["bfloat16", "float32"]) if op == "gemm" else "float32",
                 accumulate=op == "wgrad" and rng.random() < 0.4)


def _up(n):
    return -(-n // B) * B


def _counts(case):
    """Rows of each group: uneven, one of more than three groups without any."""
    g, rows = case["groups"], case["rows"] - case["tail"]
    part = [1.0 + 0.5 * math.sin(2.4 * i + 1.0) for i in range(g)]
    if g > 3:
        part[g // 2] = 0.0
    cuts = [0] + [int(round(rows * sum(part[:i + 1]) / sum(part))) for i in range(g)]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split()]


def work(case):
    if case["op"] in ("muon", "orth"):
        flops = size = 0
        for b, r, c in _shapes(case):
            m, n = min(r, c), max(r, c)
            # X X^T and A A^T are symmetric: half of each is enough
            flops += b * 5 * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)
            size += b * r * c
        if case["op"] == "orth":
            return {"bytes": size * (4 + 2 * (case["dtype"] == "float32")), "flops": flops}
        g = 4 if case["grad"] == "float32" else 2
        return {"bytes": size * (g + 8 + 8 + 2 * case["copy"]), "flops": flops}
    n, k, counts = case["n"], case["k"], _counts(case)
    kp, rows = _up(k), sum(counts)
    e = 2 if case["dtype"] == "bfloat16" else 4
    if case["op"] == "quant":
        side = kp + kp // B * 4
        if case["both"]:
            return {"bytes": case["rows"] * k * e + case["rows"] * side + sum(map(_up, counts)) * (k + k / 32),
                    "flops": 6 * case["rows"] * k}
        return {"bytes": case["rows"] * k * e + case["rows"] * side, "flops": 3 * case["rows"] * k}
    if case["op"] == "quant_w":
        out = n * kp + (k * _up(n) if case["both"] else 0)
        return {"bytes": case["groups"] * (n * k * e + out), "flops": 3 * case["groups"] * n * k}
    if case["op"] == "gemm":
        live = sum(c > 0 for c in counts)
        return {"bytes": rows * (kp + kp // 32) + live * n * kp + rows * n * e, "flops": 2 * rows * n * k}
    tokens = sum(map(_up, counts))
    return {"bytes": (n + k) * (tokens + tokens // 32) + 4 * case["groups"] * n * k * (1 + case["accumulate"]),
            "flops": 2 * rows * n * k}


# ----------------------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _features(g, rows, k):
    """Activations: features of different sizes, a few of them large."""
    size = torch.exp(0.5 * _rand(g, k))
    return _rand(g, rows, k) * torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 20 * size, size)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("muon", "orth"):
        return _prepare_muon(case, g)
    n, k, counts = case["n"], case["k"], _counts(case)
    starts = [sum(counts[:i]) for i in range(len(counts) + 1)]
    empty = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")
    u8, dt = torch.uint8, getattr(torch, case["dtype"])
    st = dict(case=case, counts=counts, starts=starts)
    if case["op"] == "quant_w":
        gr = case["groups"]
        st["x"] = (0.02 * _rand(g, gr, n, k)).to(dt)
        st["codes"], st["scales"] = empty(gr, n, _up(k), dt=u8), empty(gr, _up(n) // B, _up(k) // B)
        if case["both"]:
            st["codes_t"], st["scales_t"] = empty(gr, k, _up(n), dt=u8), empty(gr, _up(k) // B, _up(n) // B)
        return st
    rows = case["rows"]
    st["offsets"] = torch.tensor(starts, dtype=torch.int32, device="cuda") if case["groups"] > 1 or case["tail"] else None
    padded = (rows + (B - 1) * case["groups"]) // B * B
    if case["op"] == "quant":
        st["x"] = _features(g, rows, k).to(dt)
        st["codes"], st["scales"] = empty(rows, _up(k), dt=u8), empty(_up(k) // B, rows)
        if case["both"]:
            st["codes_t"], st["scales_t"] = empty(k, padded, dt=u8), empty(padded // B, k)
        return st
    if case["op"] == "gemm":
        st["x"], st["xs"] = _quant(_features(g, rows, k))
        st["w"] = empty(case["groups"], n, _up(k), dt=u8)
        st["ws"] = empty(case["groups"], _up(n) // B, _up(k) // B)
        for e in range(case["groups"]):
            st["w"][e], st["ws"][e] = _quant_square(0.02 * _rand(g, n, k))
        st["out"] = empty(rows, n, dt=dt)
        return st
    for name, width, rnd in (("dy", n, lambda: _rand(g, rows, n) * 1e-3), ("x", k, lambda: _features(g, rows, k))):
        st[name], st[name + "s"] = empty(width, padded, dt=u8), empty(padded // B, width)
        _columns(rnd(), counts, starts, st[name], st[name + "s"])
    st["dw"] = empty(case["groups"], n, k)
    if case["accumulate"]:
        st["dw"].copy_(0.1 * _rand(g, case["groups"], n, k))
    return st


def _prepare_muon(case, g):
    shapes = _shapes(case)
    # gradients whose rows and columns differ in size, as experts' features do
    grad = lambda b, r, c: _rand(g, b, r, c) * torch.exp(0.5 * _rand(g, b, r, 1)) * torch.exp(0.5 * _rand(g, b, 1, c)) * 1e-3
    st = dict(case=case)
    if case["op"] == "orth":
        st["src"] = [grad(*s).to(getattr(torch, case["dtype"])) for s in shapes]
        st["out"] = [torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in shapes]
        if own:
            import combine_router_top_schedule_amd as mok
            st["plan"] = mok.orthogonalize_plan(st["src"], st["out"])
        return st
    st["g"] = [grad(*s).to(getattr(torch, case["grad"])) for s in shapes]
    st["m"] = [grad(*s) * 3 for s in shapes]
    st["p"] = [0.02 * _rand(g, *s) for s in shapes]
    st["copy"] = [p.bfloat16() for p in st["p"]] if case["copy"] else None
    st["sumsq"] = sum(t.double().square().sum() for t in st["g"]).reshape(1) if case["clip"] else None
    st["hyper"] = dict(lr=2e-4, momentum=0.95, weight_decay=0.1, eps=1e-7, max_norm=1.0)
    if own:
        import combine_router_top_schedule_amd as mok
        st["plan"] = mok.muon_plan(p=st["p"], g=st["g"], m=st["m"], copy=st["copy"])
    return st


# ------------------------------------------------------------------------------ the plain forms

def _encode(x, axes):
    """E4M3 codes and scales: one scale for all of `axes`."""
    amax = x.abs().amax(axes, keepdim=True).clamp_min(LEAST)
    return (x * (TOP / amax)).to(torch.float8_e4m3fn).view(torch.uint8), amax / TOP


def _quant(x):
    """Blocks along the row: codes [rows][up(k)], scales [up(k) / 128][rows]."""
    r, k = x.shape
    c, s = _encode(torch.nn.functional.pad(x.float(), (0, _up(k) - k)).view(r, -1, B), (2,))
    return c.view(r, -1), s.view(r, -1).t().contiguous()


def _quant_square(w):
    """Blocks of 128 x 128: codes [n][up(k)], scales [up(n) / 128][up(k) / 128]."""
    n, k = w.shape
    w = torch.nn.functional.pad(w.float(), (0, _up(k) - k, 0, _up(n) - n))
    c, s = _encode(w.view(_up(n) // B, B, _up(k) // B, B), (1, 3))
    return c.view(_up(n), _up(k))[:n], s.view(_up(n) // B, _up(k) // B)


def _columns(x, counts, starts, codes, scales):
    """Each group's rows turned to columns from a multiple of 128 on, blocks along the rows."""
    at = 0
    for c, a in zip(counts, starts):
        if c:
            codes[:, at:at + _up(c)], scales[at // B:(at + _up(c)) // B] = _quant(x[a:a + c].t())
        at += _up(c)


def _decode(codes, scales):
    """Rows of codes with scales [blocks][rows]."""
    r = codes.shape[0]
    v = codes.view(torch.float8_e4m3fn).float().view(r, -1, B)
    return (v * scales.t().unsqueeze(2)).view(r, -1)


def _decode_square(codes, scales):
    n = codes.shape[0]
    s = scales.repeat_interleave(B, 0)[:n].repeat_interleave(B, 1)
    return codes.view(torch.float8_e4m3fn).float() * s


def _values(t):
    return t.view(torch.float8_e4m3fn)


# -------------------------------------------------------------------------------- the operators

def run(st):
    return {"quant": _run_quant, "quant_w": _run_quant_w, "gemm": _run_gemm, "wgrad": _run_wgrad,
            "muon": _run_muon, "orth": _run_orth}[st["case"]["op"]](st)


def _run_quant(st):
    out = {"codes": _values(st["codes"]), "scales": st["scales"]}
    if "codes_t" in st:
        out["codes_t"], out["scales_t"] = _values(st["codes_t"]), st["scales_t"]
    if own:
        import combine_router_top_schedule_amd as mok
        mok.mok_block_quantize(st["x"], st["codes"], st["scales"], codes_t=st.get("codes_t"),
                               scales_t=st.get("scales_t"), offsets=st["offsets"])
        return out
    c, s = _quant(st["x"])
    st["codes"].copy_(c)
    st["scales"].copy_(s)
    if "codes_t" in st:
        _columns(st["x"], st["counts"], st["starts"], st["codes_t"], st["scales_t"])
    return out


def _run_quant_w(st):
    out = {"codes": _values(st["codes"]), "scales": st["scales"]}
    if "codes_t" in st:
        out["codes_t"], out["scales_t"] = _values(st["codes_t"]), st["scales_t"]
    if own:
        import combine_router_top_schedule_amd as mok
        mok.mok_block_quantize_weights(st["x"], st["codes"], st["scales"], codes_t=st.get("codes_t"),
                                       scales_t=st.get("scales_t"))
        return out
    for e, w in enumerate(st["x"]):
        st["codes"][e], st["scales"][e] = _quant_square(w)
        if "codes_t" in st:
            st["codes_t"][e], st["scales_t"][e] = _quant_square(w.t())
    return out


def _run_gemm(st):
    if own:
        import combine_router_top_schedule_amd as mok
        mok.mok_block_gemm(st["x"], st["xs"], st["w"], st["ws"], st["out"], offsets=st["offsets"])
        return st["out"]
    for e, (c, a) in enumerate(zip(st["counts"], st["starts"])):
        if c:
            x = _decode(st["x"][a:a + c], st["xs"][:, a:a + c])
            st["out"][a:a + c] = torch.mm(x, _decode_square(st["w"][e], st["ws"][e]).t())
    return st["out"]


def _run_wgrad(st):
    if own:
        import combine_router_top_schedule_amd as mok
        mok.mok_block_wgrad(st["dy"], st["dys"], st["x"], st["xs"], st["dw"], offsets=st["offsets"],
                            accumulate=st["case"]["accumulate"])
        return st["dw"]
    at = 0
    for e, c in enumerate(st["counts"]):
        cols, blocks = slice(at, at + _up(c)), slice(at // B, (at + _up(c)) // B)
        dw = torch.mm(_decode(st["dy"][:, cols], st["dys"][blocks]), _decode(st["x"][:, cols], st["xs"][blocks]).t())
        st["dw"][e] = st["dw"][e] + dw if st["case"]["accumulate"] else dw
        at += _up(c)
    return st["dw"]


def _newton_schulz(u, eps):
    """Five steps towards the nearest matrix with orthonormal rows (or columns), batched."""
    x = u.float()
    turn = x.shape[1] > x.shape[2]
    if turn:
        x = x.transpose(1, 2)
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    a, b, c = JORDAN
    for _ in range(5):
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x.contiguous())
    return x.transpose(1, 2) if turn else x


def _adjust(case, rows, cols):
    return {"rms": 0.2 * math.sqrt(max(rows, cols)), "spectral": math.sqrt(max(1.0, rows / cols)), "none": 1.0}[case["adjust"]]


def _run_muon(st):
    case, h = st["case"], st["hyper"]
    if own:
        import combine_router_top_schedule_amd as mok
        mok.mok_muon(st["plan"], lr=h["lr"], momentum=h["momentum"], nesterov=case["nesterov"],
                     weight_decay=h["weight_decay"], eps=h["eps"], adjust=case["adjust"],
                     sumsq=st["sumsq"], max_norm=h["max_norm"] if case["clip"] else None)
        return _muon_outputs(st)
    clip = torch.clamp(h["max_norm"] / st["sumsq"].sqrt(), max=1.0).float() if case["clip"] else 1.0
    for t, (g, m, p) in enumerate(zip(st["g"], st["m"], st["p"])):
        g = g.float() * clip
        m.mul_(h["momentum"]).add_(g)
        u = g + h["momentum"] * m if case["nesterov"] else m
        o = _newton_schulz(u, h["eps"])
        p.copy_(p * (1 - h["lr"] * h["weight_decay"]) - o * (h["lr"] * _adjust(case, *p.shape[1:])))
        if case["copy"]:
            st["copy"][t].copy_(p)
    return _muon_outputs(st)


def _muon_outputs(st):
    out = {"p": st["p"], "m": st["m"]}
    if st["copy"] is not None:
        out["copy"] = st["copy"]
    return out


def _run_orth(st):
    if own:
        import combine_router_top_schedule_amd as mok
        mok.mok_orthogonalize(st["plan"], eps=1e-7)
        return st["out"]
    for s, o in zip(st["src"], st["out"]):
        o.copy_(_newton_schulz(s, 1e-7))
    return st["out"]


# -------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] in ("muon", "orth"):
        return _exact_muon(case, st)
    if case["op"] == "quant":
        out = dict(zip(("codes", "scales"), _exact_rows(st["x"].to(f64))))
        if case["both"]:
            out["codes_t"], out["scales_t"] = st["codes_t"].to(f64), st["scales_t"].to(f64)
            at = 0
            for c, a in zip(st["counts"], st["starts"]):
                if c:
                    v, s = _exact_rows(st["x"][a:a + c].to(f64).t())
                    out["codes_t"][:, at:at + v.shape[1]] = v
                    out["scales_t"][at // B:at // B + s.shape[0]] = s
                at += _up(c)
        return out
    if case["op"] == "quant_w":
        two = [_exact_blocks(w.to(f64)) for w in st["x"]]
        out = {"codes": torch.stack([v for v, _ in two]), "scales": torch.stack([s for _, s in two])}
        if case["both"]:
            two = [_exact_blocks(w.to(f64).t()) for w in st["x"]]
            out["codes_t"], out["scales_t"] = torch.stack([v for v, _ in two]), torch.stack([s for _, s in two])
        return out
    wide = lambda c: c.view(torch.float8_e4m3fn).to(f64)
    if case["op"] == "gemm":
        out = st["out"].to(f64)
        for e, (c, a) in enumerate(zip(st["counts"], st["starts"])):
            for j in range(st["x"].shape[1] // B) if c else ():
                cols = slice(j * B, (j + 1) * B)
                part = wide(st["x"][a:a + c, cols]) @ wide(st["w"][e, :, cols]).t().contiguous()
                out[a:a + c] += part * st["xs"][j, a:a + c, None].to(f64) * st["ws"][e, :, j].to(f64).repeat_interleave(B)[:case["n"]]
        return out
    out, at = st["dw"].to(f64) * (1 if case["accumulate"] else 0), 0
    for e, c in enumerate(st["counts"]):
        for j in range(at // B, (at + _up(c)) // B):
            cols = slice(j * B, (j + 1) * B)
            part = wide(st["dy"][:, cols]) @ wide(st["x"][:, cols]).t().contiguous()
            out[e] += part * st["dys"][j, :, None].to(f64) * st["xs"][j].to(f64)
        at += _up(c)
    return out


def _nearest_e4m3(a):
    """E4M3 value nearest to a, ties to the even one."""
    mag = a.abs()
    step = torch.exp2(torch.floor(torch.log2(mag.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(a) * torch.clamp(torch.round(mag / step) * step, max=TOP)


def _exact_rows(x):
    r, k = x.shape
    values, scales = torch.zeros(r, _up(k), dtype=x.dtype, device=x.device), []
    for j in range(0, k, B):
        v = x[:, j:j + B]
        s = v.abs().max(1).values.clamp(min=LEAST) / TOP
        values[:, j:min(j + B, k)] = _nearest_e4m3(v / s[:, None])
        scales.append(s)
    return values, torch.stack(scales)


def _exact_blocks(w):
    n, k = w.shape
    values = torch.zeros(n, _up(k), dtype=w.dtype, device=w.device)
    scales = torch.zeros(_up(n) // B, _up(k) // B, dtype=w.dtype, device=w.device)
    for j in range(0, k, B):
        strip = w[:, j:j + B]
        top = torch.nn.functional.pad(strip.abs().max(1).values, (0, _up(n) - n)).view(-1, B).max(1).values
        s = top.clamp(min=LEAST) / TOP
        values[:, j:min(j + B, k)] = _nearest_e4m3(strip / s.repeat_interleave(B)[:n, None])
        scales[:, j // B] = s
    return values, scales


def _polynomial(u):
    """The same polynomial of u, as a function of its smaller Gram matrix times u / |u|."""
    u = u.to(torch.float64)
    if u.shape[0] > u.shape[1]:
        return _polynomial(u.t().contiguous()).t()
    x = u / (torch.linalg.vector_norm(u) + 1e-7)
    gram = x @ x.t().contiguous()
    eye = torch.eye(gram.shape[0], dtype=gram.dtype, device=gram.device)
    left, now = eye, gram                       # iterate = left x, now = its Gram matrix
    for _ in range(5):
        f = JORDAN[0] * eye + JORDAN[1] * now + JORDAN[2] * (now @ now)
        left = f @ left
        now = f @ now @ f
    return left @ x


def _exact_muon(case, st):
    each = lambda t: torch.stack([_polynomial(u) for u in t])
    if case["op"] == "orth":
        return [each(s) for s in st["src"]]
    h, out = st["hyper"], {"p": [], "m": []}
    down = min(1.0, h["max_norm"] / math.sqrt(float(st["sumsq"]))) if case["clip"] else 1.0
    for g, m, p in zip(st["g"], st["m"], st["p"]):
        g = g.to(torch.float64) * down
        m = m.to(torch.float64) * h["momentum"] + g
        o = each(m * h["momentum"] + g if case["nesterov"] else m)
        p = p.to(torch.float64)
        out["m"].append(m)
        out["p"].append(p - h["lr"] * (h["weight_decay"] * p + _adjust(case, *p.shape[1:]) * o))
    if case["copy"]:
        out["copy"] = out["p"]
    return out
