"""What the operators around the mixer cost: states in a pool, slot maps, the output norm, the prologue.

Each case is one call (or one direction of a call) as a serving loop or a training step makes it:

* ``step``      the gated delta rule token by token over a pool of state slots (``step_slots``)
* ``slot_map``  slot maps of a batch from its request lengths (``slot_map``)
* ``norm``      the output norm, grouped by head, with an activation (``group_norm_fwd`` / ``group_norm_bwd``)
* ``prologue``  raw projections to normalised q, k and gates, and back (``prologue_fwd`` / ``prologue_bwd``)

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits; with ``own`` true it calls
the package.  ``exact`` computes the same values in 64 bits.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
NORM_EPS = 1e-6  # of the L2 normalisation of q and k
GROUP_EPS = 1e-5  # of the output norm


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's next token: 16 heads, the smallest call of a decode loop
        dict(name="step, 1 request", op="step", R=1, most=1, Hk=16, H=16, dk=128, dv=128, dtype="bf16",
             gate="scalar", raw=True, fused=True, keep="last"),
        # a full decode batch: 256 requests, 16 heads of 128
        dict(name="step, 256 requests", op="step", R=256, most=1, Hk=16, H=16, dk=128, dv=128, dtype="bf16",
             gate="scalar", raw=True, fused=True, keep="last"),
        # checking up to five drafted tokens a request, the state kept after each; two value heads share a key head
        dict(name="step, drafts kept", op="step", R=48, most=5, Hk=16, H=32, dk=128, dv=128, dtype="bf16",
             gate="scalar", raw=True, fused=True, keep="all"),
        # a ragged batch in fp32 with gates per key channel, mapped beforehand; only the last state is kept
        dict(name="step, ragged fp32 channel", op="step", R=37, most=12, Hk=5, H=5, dk=64, dv=128, dtype="fp32",
             gate="channel", raw=False, fused=False, keep="last"),
        # the maps of a small batch with drafts
        dict(name="map, 9 requests", op="slot_map", R=9, W=4, tokens=64, keep="all"),
        # the maps of the largest batch: thousands of requests, a few drafts each
        dict(name="map, 4096 requests", op="slot_map", R=4096, W=8, tokens=32768, keep="all"),
        # output norm of a decode batch (256 requests, 16 heads of 128), SiLU gate from a fused projection
        dict(name="norm, decode", op="norm", way="fwd", rows=256, G=16, D=128, dtype="bf16", gate=True, act="silu",
             center=False, affine="group", bias=False, fused=True),
        # output norm of a training batch (8 x 4096 tokens, 16 heads of 128) and its gradient
        dict(name="norm, training", op="norm", way="fwd", rows=32768, G=16, D=128, dtype="bf16", gate=True, act="silu",
             center=False, affine="group", bias=False, fused=True),
        dict(name="norm, training gradient", op="norm", way="bwd", rows=32768, G=16, D=128, dtype="bf16", gate=True,
             act="silu", center=False, affine="group", bias=False, fused=True),
        # an odd width in fp32, centred, with weights and biases for every channel, the activation on the norm itself
        dict(name="norm, odd gradient", op="norm", way="bwd", rows=2003, G=7, D=100, dtype="fp32", gate=False, act="silu",
             center=True, affine="channel", bias=True, fused=False),
        # a training batch's raw projections to the mixer's inputs; two value heads share a key head
        dict(name="prologue, training", op="prologue", way="fwd", tokens=32768, Hk=8, H=16, dk=128, dtype="bf16",
             gate="scalar", fused=True),
        # the gradient of an odd batch with gates per key channel; three value heads share a key head
        dict(name="prologue, odd gradient", op="prologue", way="bwd", tokens=3331, Hk=4, H=12, dk=64, dtype="bf16",
             gate="channel", fused=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("step", "step", "slot_map", "norm", "norm", "prologue"))
    if op == "step":
        case = dict(op=op, R=_log(rng, 1, 256), most=rng.choice((1, 1, 2, 3, 4, 6, 8, 32)), Hk=rng.choice((1, 2, 3, 4, 8, 16)),
                    dk=rng.choice((32, 64, 128)), dv=rng.choice((32, 64, 128)), dtype=rng.choice(("bf16", "bf16", "fp32")),
                    gate=rng.choice(("scalar", "scalar", "channel")), raw=rng.random() < 0.6, fused=rng.random() < 0.5,
                    keep=rng.choice(("last", "all")))
        case["H"] = case["Hk"] * rng.choice((1, 1, 2, 3))
        while work(case)["bytes"] > 4e8:  # (states of 64 KB add up quickly)
            case["R"] = max(1, case["R"] * 2 // 3)
            if case["R"] == 1:
                break
        return case
    if op == "slot_map":
        R, W = _log(rng, 1, 4096), rng.randint(1, 8)
        keep = rng.choice(("last", "all"))
        return dict(op=op, R=R, W=W, tokens=R * W + rng.randint(0, 300), keep=keep)
    if op == "norm":
        G, D = rng.randint(1, 32), rng.choice((32, 33, 48, 64, 80, 100, 128, 128, 192, 256, 513))
        rows = min(_log(rng, 1, 32768), 48_000_000 // (G * D))
        gate = rng.random() < 0.7
        return dict(op=op, way=rng.choice(("fwd", "bwd")), rows=rows, G=G, D=D, dtype=rng.choice(("bf16", "bf16", "fp32")),
                    gate=gate, act=rng.choice(("silu", "silu", "sigmoid")) if gate else rng.choice(("silu", "none")),
                    center=rng.random() < 0.4, affine=rng.choice(("group", "channel", "none")), bias=rng.random() < 0.4,
                    fused=gate and rng.random() < 0.5)
    Hk, dk = rng.choice((1, 2, 3, 4, 6, 8, 16)), rng.choice((32, 64, 128))
    H = Hk * rng.choice((1, 1, 2, 3, 4))
    tokens = min(_log(rng, 1, 32768), 32_000_000 // (H * dk))
    return dict(op=op, way=rng.choice(("fwd", "bwd")), tokens=tokens, Hk=Hk, H=H, dk=dk,
                dtype=rng.choice(("bf16", "bf16", "fp32")), gate=rng.choice(("scalar", "scalar", "channel")),
                fused=rng.random() < 0.5)


def _lengths(case):
    """New tokens of each request: every length up to ``most`` as often as the others (in an order that the seed gives)."""
    return [1 + r % case["most"] for r in range(case["R"])]


def work(case):
    e = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "step":
        lens = _lengths(case)
        t, R, Hk, H, dk, dv = sum(lens), case["R"], case["Hk"], case["H"], case["dk"], case["dv"]
        kept = t if case["keep"] == "all" else R
        gates = t * H * (dk if case["gate"] == "channel" else 1) + t * H + (H if case["raw"] else 0)
        maps = R if case["most"] == 1 and case["keep"] == "last" else 2 * R + 1 + t
        return {"bytes": 4 * H * dk * dv * (R + kept) + e * t * (2 * Hk * dk + 2 * H * dv) + 4 * gates + 4 * maps,
                "flops": 7 * t * H * dk * dv}
    if case["op"] == "slot_map":
        R, W, t = case["R"], case["W"], case["tokens"]
        return {"bytes": 4 * (R + R + R * W + (R + 1) + R + 2 * t), "flops": 4 * t}
    if case["op"] == "norm":
        n = case["rows"] * case["G"] * case["D"]
        w = {"group": case["D"], "channel": case["G"] * case["D"], "none": 0}[case["affine"]] * (2 if case["bias"] else 1)
        if case["way"] == "fwd":
            return {"bytes": n * e * (3 if case["gate"] else 2) + 4 * w, "flops": 12 * n}
        return {"bytes": n * e * (4 if case["gate"] else 2) + 4 * n + 8 * w, "flops": 30 * n}
    t, Hk, H, dk = case["tokens"], case["Hk"], case["H"], case["dk"]
    gates = t * H * (dk if case["gate"] == "channel" else 1) + t * H
    if case["way"] == "fwd":
        return {"bytes": e * 2 * t * dk * (Hk + H) + 8 * gates + 4 * H, "flops": 8 * t * dk * (Hk + H) + 10 * gates}
    return {"bytes": e * 4 * t * Hk * dk + 8 * t * H * dk + 12 * gates + 8 * H, "flops": 12 * t * dk * (Hk + H) + 20 * gates}


# ------------------------------------------------------------------ the inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device)


def _rows(gen, n, widths, dtype, fused):
    """[n, w] tensors of N(0, 1): slices of one projection's rows (fused), or each on its own."""
    if not fused:
        return [_normal(gen, n, w).to(dtype) for w in widths]
    return list(_normal(gen, n, sum(widths)).to(dtype).split(widths, dim=1))


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _prepare_step(case, gen):
    R, most, Hk, H, dk, dv = (case[k] for k in ("R", "most", "Hk", "H", "dk", "dv"))
    dev, dtype = gen.device, DTYPES[case["dtype"]]
    lens = torch.tensor(_lengths(case), device=dev)[torch.randperm(R, generator=gen, device=dev)]
    total = sum(_lengths(case))
    W = most if case["keep"] == "all" else 1
    slots = R * W + 3  # a few slots belong to requests that are not in this batch
    q, k, v = _rows(gen, total, [Hk * dk, Hk * dk, H * dv], dtype, case["fused"])
    q, k, v = q.unflatten(1, (Hk, dk)), k.unflatten(1, (Hk, dk)), v.unflatten(1, (H, dv))
    logits = _normal(gen, total, H, dk) if case["gate"] == "channel" else _normal(gen, total, H)
    writes = _normal(gen, total, H)
    s = {"case": case, "v": v, "slots": slots}
    if case["raw"]:
        s |= {"q": q, "k": k, "g": logits, "beta": writes, "gate_scale": 0.05 + 0.1 * torch.rand(H, generator=gen, device=dev)}
    else:
        s |= {"q": _unit(q.float()).to(dtype), "k": _unit(k.float()).to(dtype), "g": -0.1 * torch.log1p(torch.exp(logits)),
              "beta": 1 / (1 + torch.exp(-writes)), "gate_scale": None}
    # one more slot than the pool has: the plain form's place for what nobody keeps
    s["buffer"] = 0.1 * _normal(gen, slots + 1, H, dv, dk)
    s["pool"] = s["buffer"][:slots]
    table = torch.randperm(slots, generator=gen, device=dev)[: R * W].view(R, W)
    row = torch.arange(R, device=dev)
    src = table[row, torch.randint(0, W, (R,), generator=gen, device=dev)]
    s["dst"] = s["cu"] = None
    if most > 1 or case["keep"] == "all":
        src = torch.where(row % 16 == 5, -1, src)  # a few requests are new: they start from nothing
        cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)])
        dst = torch.full((total,), -1, device=dev)
        if case["keep"] == "all":
            for j in range(most):
                has = lens > j
                dst[cu[:-1][has] + j] = table[has, j]
        else:
            dst[cu[1:] - 1] = table[:, 0]
        s["dst"], s["cu"] = dst.int(), cu.int()
    s["src"] = src.int()
    return s


def _prepare_map(case, gen):
    R, W, dev = case["R"], case["W"], gen.device
    lens = torch.randint(0, W + 1, (R,), generator=gen, device=dev, dtype=torch.int32)
    kept = torch.randint(0, W + 1, (R,), generator=gen, device=dev, dtype=torch.int32)
    slots = R * W + 16
    table = torch.randperm(slots, generator=gen, device=dev)[: R * W].view(R, W).int()
    return {"case": case, "lens": lens, "kept": kept, "table": table, "slots": slots}


def _prepare_norm(case, gen):
    rows, G, D, dtype, dev = case["rows"], case["G"], case["D"], DTYPES[case["dtype"]], gen.device
    scale = 0.2 + torch.rand(G, 1, generator=gen, device=dev)  # heads answer at their own scale
    x = (_normal(gen, rows, G, D) * scale + 0.1).to(dtype)
    s = {"case": case, "x": x, "z": None, "weight": None, "bias": None, "dy": None}
    if case["gate"]:  # beside another projection's columns where one product makes both
        s["z"] = _rows(gen, rows, [G * D, G * D] if case["fused"] else [G * D], dtype, case["fused"])[-1].unflatten(1, (G, D))
    if case["affine"] != "none":
        shape = (D,) if case["affine"] == "group" else (G, D)
        s["weight"] = 1 + 0.2 * _normal(gen, *shape)
        s["bias"] = 0.2 * _normal(gen, *shape) if case["bias"] else None
    if case["way"] == "bwd":
        s["dy"] = _normal(gen, rows, G, D).to(dtype)
    return s


def _prepare_prologue(case, gen):
    t, Hk, H, dk, dtype, dev = case["tokens"], case["Hk"], case["H"], case["dk"], DTYPES[case["dtype"]], gen.device
    q, k = (x.unflatten(1, (Hk, dk)) for x in _rows(gen, t, [Hk * dk, Hk * dk], dtype, case["fused"]))
    a = _normal(gen, t, H, dk) if case["gate"] == "channel" else _normal(gen, t, H)
    s = {"case": case, "q": q, "k": k, "a": a, "b": _normal(gen, t, H), "scale": 0.05 + 0.1 * torch.rand(H, generator=gen, device=dev)}
    if case["way"] == "bwd":
        s |= {"dq": _normal(gen, t, H, dk), "dk": _normal(gen, t, H, dk), "dg": torch.randn(a.shape, generator=gen, device=dev),
              "dbeta": _normal(gen, t, H)}
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"step": _prepare_step, "slot_map": _prepare_map, "norm": _prepare_norm, "prologue": _prepare_prologue}[case["op"]](case, gen)


# ------------------------------------------------------------------ the plain forms
def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_step(s):
    case = s["case"]
    most, H, dtype = case["most"], case["H"], DTYPES[case["dtype"]]
    q, k, v, g, beta, src = s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["beta"], s["src"].long()
    if case["raw"]:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + NORM_EPS)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + NORM_EPS)
        g = -s["gate_scale"].view(H, *[1] * (g.dim() - 2)) * _softplus(g)
        beta = _sigmoid(beta)
    alpha = torch.exp(g if g.dim() == 3 else g[..., None])
    if s["cu"] is None:
        first, lens = torch.arange(case["R"], device=q.device), torch.ones_like(src)
        dst = src
    else:
        cu = s["cu"].long()
        first, lens, dst = cu[:-1], cu[1:] - cu[:-1], s["dst"].long()
    total = v.shape[0]
    state = s["buffer"][src.clamp(min=0)] * (src >= 0).view(-1, 1, 1, 1)
    o = v.new_zeros(total + 1, *v.shape[1:])
    for j in range(most):  # a recurrence: one token of every request after the other
        live = lens > j
        t = torch.where(live, first + j, 0)
        qt, kt = (x[t].repeat_interleave(H // case["Hk"], dim=1)[..., None] for x in (q, k))
        new = state * alpha[t][:, :, None]
        u = beta[t][..., None] * (v[t] - torch.matmul(new, kt)[..., 0])
        new = new + u[..., None] * kt.transpose(-1, -2)
        o[torch.where(live, t, total)] = torch.matmul(new, qt)[..., 0]
        state = new if most == 1 else torch.where(live.view(-1, 1, 1, 1), new, state)
        to = dst[t]
        s["buffer"][torch.where(live & (to >= 0), to, s["slots"])] = state
    return {"o": o[:total].to(dtype), "pool": s["pool"]}


def _plain_map(s):
    case = s["case"]
    R, W, T, dev = case["R"], case["W"], case["tokens"], s["lens"].device
    lens, kept, table, row = s["lens"].long(), s["kept"].long(), s["table"], torch.arange(case["R"], device=s["lens"].device)
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)])
    starts = torch.zeros(T + 1, dtype=torch.long, device=dev).index_add_(0, cu[1:].clamp(max=T), torch.ones_like(row))
    request = starts.cumsum(0)[:T]
    token = torch.arange(T, device=dev)
    real = token < cu[-1]
    request = torch.where(real, request, 0)
    at = token - cu[request]
    src = torch.where(lens > 0, torch.where(kept > 0, table[row, (kept - 1).clamp(min=0)], -1), -2)
    if case["keep"] == "all":
        dst = torch.where(real, table[request, at.clamp(0, W - 1)], -1)
    else:
        dst = torch.where(real & (at == lens[request] - 1), table[request, 0], -1)
    return {"cu_seqlens": cu.int(), "request": torch.where(real, request, -1).int(), "src": src.int(), "dst": dst.int()}


def _plain_norm(s):
    case = s["case"]
    x, z, w, b = s["x"].float(), s["z"], s["weight"], s["bias"]
    dtype = DTYPES[case["dtype"]]
    x = x - x.mean(-1, keepdim=True) if case["center"] else x
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + GROUP_EPS)
    n = x * rstd
    lin = n if w is None else n * w if b is None else n * w + b
    on = lin if z is None else z.float()  # what the activation acts on
    sg = None if case["act"] == "none" else _sigmoid(on)
    act = on if sg is None else sg if case["act"] == "sigmoid" else on * sg
    if case["way"] == "fwd":
        return {"y": (act if z is None else act * lin).to(dtype)}
    slope = 1 if sg is None else sg * (1 - sg) if case["act"] == "sigmoid" else sg * (1 + on * (1 - sg))
    dy = s["dy"].float()
    dlin = dy * slope if z is None else dy * act
    out = {"dz": None if z is None else (dy * lin * slope).to(dtype), "dweight": None, "dbias": None}
    if w is not None:
        over = (0, 1) if w.dim() == 1 else (0,)
        out["dweight"] = (dlin * n).sum(over)
        out["dbias"] = None if b is None else dlin.sum(over)
        dlin = dlin * w
    dx = dlin - n * (dlin * n).mean(-1, keepdim=True)
    out["dx"] = rstd * (dx - dlin.mean(-1, keepdim=True) if case["center"] else dx)
    return out


def _plain_prologue(s):
    case = s["case"]
    H, Hk, dtype = case["H"], case["Hk"], DTYPES[case["dtype"]]
    q, k, a, b = s["q"].float(), s["k"].float(), s["a"], s["b"]
    scale = s["scale"].view(H, *[1] * (a.dim() - 2))
    rq, rk = (torch.rsqrt((x * x).sum(-1, keepdim=True) + NORM_EPS) for x in (q, k))
    beta = _sigmoid(b)
    if case["way"] == "fwd":
        share = lambda x: x.to(dtype).repeat_interleave(H // Hk, dim=1)  # noqa: E731
        return {"q": share(q * rq), "k": share(k * rk), "g": -scale * _softplus(a), "beta": beta}
    out = {}
    for name, x, r, d in (("dq", q, rq, s["dq"]), ("dk", k, rk, s["dk"])):
        d = d.unflatten(1, (Hk, H // Hk)).sum(2)
        n = x * r
        out[name] = (r * (d - n * (n * d).sum(-1, keepdim=True))).to(dtype)
    out["da"] = -scale * _sigmoid(a) * s["dg"]
    out["db"] = beta * (1 - beta) * s["dbeta"]
    ds = -s["dg"] * _softplus(a)
    out["dgate_scale"] = ds.sum((0, 2) if a.dim() == 3 else 0)
    return out


# ------------------------------------------------------------------ the package's operators
def _own_step(s):
    import gated_delta_rule_93_b200 as gdr

    raw = s["gate_scale"] is not None
    o = gdr.step_slots(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s["src"], dst=s["dst"],
                       cu_seqlens=s["cu"], gate_scale=s["gate_scale"], norm_q=raw, norm_k=raw)
    return {"o": o, "pool": s["pool"]}


def _own_map(s):
    import gated_delta_rule_93_b200 as gdr

    return gdr.slot_map(s["lens"], s["kept"], s["table"], s["slots"], s["case"]["tokens"], keep_all=s["case"]["keep"] == "all")


def _own_norm(s):
    import gated_delta_rule_93_b200 as gdr

    case = s["case"]
    how = dict(act=case["act"], center=case["center"], eps=GROUP_EPS)
    if case["way"] == "fwd":
        return {"y": gdr.group_norm_fwd(s["x"], s["z"], s["weight"], s["bias"], **how)}
    return gdr.group_norm_bwd(s["dy"], s["x"], s["z"], s["weight"], s["bias"], **how)


def _own_prologue(s):
    import gated_delta_rule_93_b200 as gdr

    if s["case"]["way"] == "fwd":
        q, k, g, beta = gdr.prologue_fwd(s["q"], s["k"], s["a"], s["b"], s["scale"])
        return {"q": q, "k": k, "g": g, "beta": beta}
    return gdr.prologue_bwd(s["q"], s["k"], s["a"], s["b"], s["scale"], s["dq"], s["dk"], s["dg"], s["dbeta"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"step": _own_step, "slot_map": _own_map, "norm": _own_norm, "prologue": _own_prologue}[op](state)
    return {"step": _plain_step, "slot_map": _plain_map, "norm": _plain_norm, "prologue": _plain_prologue}[op](state)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_step(s):
    """Every token as a product with its transition matrix, S (Diag(alpha) (I - beta k k^T)) + beta v k^T."""
    case = s["case"]
    H, dk = case["H"], case["dk"]
    share = lambda x: x.repeat_interleave(H // case["Hk"], dim=1)  # noqa: E731
    q, k, v, g, beta = (s[n].double() for n in ("q", "k", "v", "g", "beta"))
    if case["raw"]:
        q = q * (q.square().sum(-1, keepdim=True) + NORM_EPS).pow(-0.5)
        k = k * (k.square().sum(-1, keepdim=True) + NORM_EPS).pow(-0.5)
        scale = s["gate_scale"].double()
        g = -torch.logaddexp(g, torch.zeros_like(g)) * (scale[:, None] if g.dim() == 3 else scale)
        beta = torch.special.expit(beta)
    q, k = share(q), share(k)
    alpha = g.exp() if g.dim() == 3 else g.exp()[..., None].expand(-1, -1, dk)
    pool, src = s["pool"].double(), s["src"].tolist()
    R, total = len(src), v.shape[0]
    cu = list(range(R + 1)) if s["cu"] is None else s["cu"].tolist()
    dst = src if s["dst"] is None else s["dst"].tolist()
    state = torch.stack([pool[n] if n >= 0 else torch.zeros_like(pool[0]) for n in src])
    o, eye, kept = torch.zeros_like(v), torch.eye(dk, dtype=torch.float64, device=v.device), {}
    for j in range(case["most"]):
        at = [r for r in range(R) if cu[r] + j < cu[r + 1]]
        t = [cu[r] + j for r in at]
        if not at:
            break
        kt, bt = k[t], beta[t][..., None, None]
        through = alpha[t][..., None] * (eye - bt * kt[..., :, None] * kt[..., None, :])
        new = state[at] @ through + bt * v[t][..., :, None] * kt[..., None, :]
        state[at] = new
        o[t] = torch.einsum("rhij,rhj->rhi", new, q[t])
        to = [n for n, x in enumerate(t) if dst[x] >= 0]
        if to:
            pool[[dst[t[n]] for n in to]] = new[to]
    return {"o": o, "pool": pool}


def _exact_norm(s):
    """The definition, and its gradients by differentiation in 64 bits."""
    case = s["case"]
    up = lambda x: None if x is None else x.detach().double().requires_grad_(case["way"] == "bwd")  # noqa: E731
    x, z, w, b = (up(s[n]) for n in ("x", "z", "weight", "bias"))
    var = x.var(-1, unbiased=False, keepdim=True) if case["center"] else x.square().mean(-1, keepdim=True)
    lin = (x - x.mean(-1, keepdim=True) if case["center"] else x) / torch.sqrt(var + GROUP_EPS)
    lin = lin if w is None else lin * w
    lin = lin if b is None else lin + b
    on = lin if z is None else z
    act = {"none": lambda u: u, "silu": lambda u: u * torch.special.expit(u), "sigmoid": torch.special.expit}[case["act"]](on)
    y = act if z is None else act * lin
    if case["way"] == "fwd":
        return {"y": y}
    wrt = {"dx": x, "dz": z, "dweight": w, "dbias": b}
    have = [n for n in wrt if wrt[n] is not None]
    got = dict(zip(have, torch.autograd.grad(y, [wrt[n] for n in have], s["dy"].double())))
    return {n: got.get(n) for n in wrt}


def _exact_prologue(s):
    case = s["case"]
    up = lambda n: s[n].detach().double().requires_grad_(case["way"] == "bwd")  # noqa: E731
    q, k, a, b, scale = (up(n) for n in ("q", "k", "a", "b", "scale"))
    share = lambda x: (x / torch.sqrt(x.square().sum(-1, keepdim=True) + NORM_EPS)).repeat_interleave(case["H"] // case["Hk"], dim=1)  # noqa: E731
    out = {"q": share(q), "k": share(k), "g": -torch.logaddexp(a, torch.zeros_like(a)) * (scale[:, None] if a.dim() == 3 else scale),
           "beta": torch.special.expit(b)}
    if case["way"] == "fwd":
        return out
    names = ("dq", "dk", "da", "db", "dgate_scale")
    return dict(zip(names, torch.autograd.grad([out[n] for n in ("q", "k", "g", "beta")], [q, k, a, b, scale],
                                               [s[n].double() for n in ("dq", "dk", "dg", "dbeta")])))


def exact(case, seed):
    if case["op"] == "slot_map":
        return None  # whole numbers: they have to be equal
    return {"step": _exact_step, "norm": _exact_norm, "prologue": _exact_prologue}[case["op"]](prepare(case, seed))
