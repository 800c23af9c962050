"""Cases of the operators on grouped rows and 8-bit features: the index of rows by group, the
channel mixing with weights per group and its gradients, the normalisation of x + residual with
its gradients and with an output in 8 bits, and the channel mixing of 8-bit features.

``run`` computes a case in its plain form (elementary torch operations), or, where ``own`` is
true, through the package's entry points.  Inputs come from the seed alone.  Features are laid out
[rows][components][channels], an irrep of degree l having 2l+1 components; weights are
[groups][pairs][Cin][Cout], a pair for every input and output block of equal degree and parity.
A group is a chemical element (a row is an atom) or, for wide scalars, an expert.
"""
import functools
import math

import torch

own = False

EPS = 1e-5
RUN, TOP = 128, 448.0  # channels that share a scale, largest 8-bit value
LEAST = 2.0 ** -126    # of a scale
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HIGH = "0e+1o+2e+3o"


def listed():
    return [
        # the elements of the 64,000-atom system, as a simulation sorts its atoms at the start
        {"name": "index mace64k", "op": "index", "rows": 64000, "groups": 10, "stray": 0.0},
        # millions of atoms of any element, padding among them
        {"name": "index large", "op": "index", "rows": 4000003, "groups": 118, "stray": 0.01},
        # one atom: latency of a call
        {"name": "mix fwd one row", "op": "mix", "backward": False, "rows": 1, "groups": 10,
         "stray": 0.0, "cin": 128, "cout": 128, "in": HIGH, "out": HIGH, "dtype": "f32"},
        # the messages of the 64,000-atom system, weights for each of ten elements
        {"name": "mix fwd mace64k", "op": "mix", "backward": False, "rows": 64000, "groups": 10,
         "stray": 0.0, "cin": 128, "cout": 128, "in": HIGH, "out": HIGH, "dtype": "f32"},
        {"name": "mix bwd mace64k", "op": "mix", "backward": True, "rows": 64000, "groups": 10,
         "stray": 0.0, "cin": 128, "cout": 128, "in": HIGH, "out": HIGH, "dtype": "f32"},
        # wide scalars in bf16 shared out over 16 experts, an uneven number of rows each
        {"name": "mix bwd experts bf16", "op": "mix", "backward": True, "rows": 16411, "groups": 16,
         "stray": 0.0, "cin": 1024, "cout": 2048, "in": "0e", "out": "0e", "dtype": "bf16"},
        # the residual update and normalisation of the 3,000-atom box
        {"name": "norm fwd water3k", "op": "norm", "pass": "fwd", "rows": 3000, "channels": 128,
         "irreps": HIGH, "dtype": "f32", "centered": True},
        # its gradients for the 64,000-atom system, with what comes back along the residual
        {"name": "norm bwd mace64k", "op": "norm", "pass": "bwd", "rows": 64000, "channels": 128,
         "irreps": HIGH, "dtype": "f32", "centered": True},
        # the same system in simulation: bf16 features, the normalised ones in 8 bits
        {"name": "norm fp8 mace64k", "op": "norm", "pass": "fp8", "rows": 64000, "channels": 128,
         "irreps": HIGH, "dtype": "bf16", "centered": False},
        # one row of wide scalars: the weights are what is read
        {"name": "fp8 one row", "op": "fp8", "rows": 1, "groups": 1, "stray": 0.0, "cin": 1024,
         "cout": 4096, "in": "0e", "out": "0e", "given": "bf16", "dtype": "bf16"},
        # channel mixing of the 64,000-atom system's features as the normalisation leaves them
        {"name": "fp8 mace64k", "op": "fp8", "rows": 64000, "groups": 1, "stray": 0.0, "cin": 128,
         "cout": 128, "in": HIGH, "out": HIGH, "given": "codes", "dtype": "bf16"},
        # 16 experts on wide scalars, quantised in the call
        {"name": "fp8 experts", "op": "fp8", "rows": 16411, "groups": 16, "stray": 0.0,
         "cin": 2048, "cout": 1024, "in": "0e", "out": "0e", "given": "bf16", "dtype": "bf16"},
    ]


def _span(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step))


def draw(rng):
    op = rng.choice(("index", "mix", "mix", "norm", "norm", "fp8", "fp8"))
    if op == "index":
        return {"op": op, "rows": _span(rng, 1, 4000000), "groups": _span(rng, 1, 1000),
                "stray": rng.choice((0.0, 0.01, 0.3))}
    if op == "norm":
        way = rng.choice(("fwd", "bwd", "fp8"))
        irreps = rng.choice(("0e", "0e", "1o", "0e+1o", "0e+1o+2e", HIGH, "0e+0o+0e+1e",
                             "0e+1o+1e+2e+2o+3o+3e", "0e+1o+2e+3o+4e+5o+6e"))
        channels = _span(rng, 16, 1024, 16) if way == "fp8" else _span(rng, 1, 1024)
        rows = _span(rng, 1, max(1, min(400000, 60_000_000 // (channels * _dim(irreps)))))
        return {"op": op, "pass": way, "rows": rows, "channels": channels, "irreps": irreps,
                "dtype": rng.choice(("f32", "bf16")), "centered": rng.random() < 0.6}
    case = {"op": op}
    if op == "mix":
        case["backward"] = rng.random() < 0.5
    wide = rng.random() < 0.4
    into, out = rng.choice((("0e", "0e"),) if wide else (
        ("0e+1o", "0e+1o"), (HIGH, HIGH), (HIGH, "0e+1o"), ("0e+0e+1o", "0e+1o+2e"),
        ("0e+1o+1e", "1e+0e+0e"), ("0e+1o+2e", "0e+1o+2e")))
    step = 8 if op == "mix" else 16
    cin, cout = (_span(rng, *((128, 2048) if wide else (step, 256)), step) for _ in range(2))
    size = max(cin * _dim(into), cout * _dim(out))
    rows = _span(rng, 1, max(1, min(100000, 60_000_000 // size, 30_000_000_000 // (cin * size))))
    groups = _span(rng, 1, max(1, min(100, 60_000_000 // (cin * cout * len(_pairs(into, out))))))
    case |= {"rows": rows, "groups": groups, "stray": rng.choice((0.0, 0.0, 0.05)), "cin": cin,
             "cout": cout, "in": into, "out": out, "dtype": rng.choice(("f32", "bf16"))}
    if op == "fp8":
        case["given"] = rng.choice(("codes", case["dtype"]))
    return case


# ------------------------------------------------------------------ inputs

@functools.cache
def _blocks(irreps):
    """[(degree, parity)] of a text such as 0e+1o."""
    return [(int(b[:-1]), 1 if b[-1] == "e" else -1) for b in irreps.split("+")]


def _dim(irreps):
    return sum(2 * l + 1 for l, _ in _blocks(irreps))


def _starts(irreps):
    """First component of every block."""
    return [sum(2 * l + 1 for l, _ in _blocks(irreps)[:i]) for i in range(len(_blocks(irreps)))]


def _pairs(into, out):
    """(input block, output block) of every weight matrix, input block by input block."""
    return [(i, o) for i, a in enumerate(_blocks(into)) for o, b in enumerate(_blocks(out))
            if a == b]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    if case["op"] == "norm":
        return _prepare_norm(case, rand)
    s = {"case": case}
    if case["op"] == "index" or case["groups"] > 1:
        # group g is about 1 / (g + 1) as frequent as group 0; what has no group is padding
        rows, groups = case["rows"], case["groups"]
        u = torch.rand(rows, device="cuda", generator=gen)
        ids = ((groups + 1.0) ** u - 1).long().clamp(max=groups - 1)
        ids = (ids * 7919 + seed) % groups
        stray = torch.rand(rows, device="cuda", generator=gen) < case["stray"]
        s["ids"] = torch.where(stray, -1, ids).int()
    return s if case["op"] == "index" else _prepare_mix(s, case, rand)


def _prepare_norm(case, rand):
    blocks, C, rows = _blocks(case["irreps"]), case["channels"], case["rows"]
    dtype, dim = TYPES[case["dtype"]], _dim(case["irreps"])
    scalars = sum(b == (0, 1) for b in blocks)
    # features of differing size from row to row, off zero, and an update of them
    x = rand(rows, dim, C) * (0.2 + rand(rows, 1, 1).square()) + 0.3
    s = {"case": case, "x": x.to(dtype), "w": 1 + 0.1 * rand(len(blocks), C),
         "b": 0.1 * rand(scalars, C)}
    s["r" if case["pass"] != "bwd" else "dh"] = rand(rows, dim, C).to(dtype)
    if case["pass"] == "bwd":
        s["dy"] = rand(rows, dim, C).to(dtype)
    # the plain form's maps: block of each component, the mean over a block's components,
    # the scalars
    of = torch.tensor([i for i, (l, _) in enumerate(blocks) for _ in range(2 * l + 1)],
                      device="cuda")
    s["of"] = of
    s["one"] = (of[None, :] == torch.arange(len(blocks), device="cuda")[:, None]).float()
    same = (of[:, None] == of[None, :]).float()
    s["share"] = same / same.sum(0, keepdim=True)
    s["scalar"] = torch.tensor([i for i, k in enumerate(of.tolist()) if blocks[k] == (0, 1)],
                               dtype=torch.long, device="cuda")
    s["center"] = torch.zeros(dim, 1, device="cuda")
    if case["centered"]:
        s["center"][s["scalar"]] = 1.0
    return s


def _prepare_mix(s, case, rand):
    rows, groups, cin, cout = (case[k] for k in ("rows", "groups", "cin", "cout"))
    into, out, dtype = _blocks(case["in"]), _blocks(case["out"]), TYPES[case["dtype"]]
    pairs = _pairs(case["in"], case["out"])
    s["W"] = rand(groups, len(pairs), cin, cout) / math.sqrt(cin)
    x = rand(rows, _dim(case["in"]), cin) * (0.2 + rand(rows, 1, 1).square())
    if case["op"] == "mix":
        s["W"], s["x"] = s["W"].to(dtype), x.to(dtype)
        if case["backward"]:
            s["dy"] = rand(rows, _dim(case["out"]), cout).to(dtype)
    elif case["given"] == "codes":
        s["q"], s["scale"] = _quantize(x)
    else:
        s["x"] = x.to(TYPES[case["given"]])
    if own:
        from clebsch_gordan_tensor_amd import api

        s["index"] = api.group_rows(s["ids"], groups) if groups > 1 else None
        if case["op"] == "fp8":
            s["packed"] = api.linear_fp8_pack(into, out, s["W"])
        return s
    if case["op"] == "fp8":
        s["W"] = _rounded_weights(s["W"])
    # the plain form's plan: the rows of every group in pieces of equal size, the last ones filled
    # up with an empty row; the components that every pair joins
    ids = s["ids"] if groups > 1 else torch.zeros(rows, dtype=torch.int32, device="cuda")
    order, start = _index(ids, groups)
    n = start[1:] - start[:-1]
    size = max(32, min(512, rows // groups))
    count = (n + size - 1) // size
    of = torch.repeat_interleave(torch.arange(groups, device="cuda"), count)
    first = (torch.cumsum(count, 0) - count)[of]
    at = (torch.arange(len(of), device="cuda") - first)[:, None] * size + torch.arange(
        size, device="cuda")
    place = (start[of.long()][:, None] + at).clamp(max=rows - 1)
    s["rows"] = torch.where(at < n[of][:, None], order[place.long()].long(), rows)
    s["of"] = of
    comps = [(p, _starts(case["in"])[i] + m, _starts(case["out"])[o] + m)
             for p, (i, o) in enumerate(pairs) for m in range(2 * into[i][0] + 1)]
    s["pair"], s["ic"], s["oc"] = (torch.tensor(t, device="cuda") for t in zip(*comps))
    return s


def _runs(x):
    """The runs of 128 channels of the last axis, the last one filled up with zeros."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % RUN)).unflatten(-1, (-1, RUN))


def _codes(x, scale):
    return (x / scale).to(torch.float8_e4m3fn)


def _quantize(x):
    """8-bit values and the scales of runs of 128 channels."""
    x = x.float()
    scale = (_runs(x.abs()).amax(-1) / TOP).clamp(min=LEAST)
    q = _codes(_runs(x), scale[..., None])
    return q.view(torch.uint8).flatten(-2)[..., :x.shape[-1]].contiguous().view(q.dtype), scale


def _values(q, scale):
    """What 8-bit features stand for."""
    return (_runs(q.float()) * scale[..., None]).flatten(-2)[..., :q.shape[-1]]


def _rounded_weights(W):
    """What the 8-bit form of weights [..][Cin][Cout] stands for: a scale for 128 x 128 of them."""
    cin, cout = W.shape[-2:]
    t = torch.nn.functional.pad(W, (0, -cout % RUN, 0, -cin % RUN))
    t = t.unflatten(-1, (-1, RUN)).unflatten(-3, (-1, RUN))  # [..][in runs][128][out runs][128]
    scale = (t.abs().amax((-1, -3), keepdim=True) / TOP).clamp(min=LEAST)
    t = _codes(t, scale).float() * scale
    return t.flatten(-4, -3).flatten(-2, -1)[..., :cin, :cout].contiguous()


def _index(ids, groups):
    """(rows by group, what has none last; where each group's rows start)."""
    key = torch.where((ids >= 0) & (ids < groups), ids, groups)
    order = torch.sort(key, stable=True).indices.int()
    n = torch.bincount(key, minlength=groups + 1)[:groups]
    return order, torch.nn.functional.pad(torch.cumsum(n, 0), (1, 0)).int()


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if op == "index":
        if own:
            from clebsch_gordan_tensor_amd import api

            index = api.group_rows(state["ids"], state["case"]["groups"])
            return index.order, index.offsets
        return _index(state["ids"], state["case"]["groups"])
    return {"mix": _run_mix, "norm": _run_norm, "fp8": _run_fp8}[op](state)


def _pieces(s, t, comps):
    """[pieces x component pairs][rows][channels] of the rows of every piece."""
    t = torch.cat([t, t.new_zeros(1, *t.shape[1:])])[s["rows"]][:, :, comps]
    return t.transpose(1, 2).flatten(0, 1).contiguous()


def _back(s, t, comps, dim):
    """_pieces' results summed over the pairs of each component, at their rows."""
    t = t.unflatten(0, (len(s["of"]), len(comps))).transpose(1, 2)
    sums = t.new_zeros(*t.shape[:2], dim, t.shape[3]).index_add_(2, comps, t)
    out = t.new_zeros(s["case"]["rows"] + 1, dim, t.shape[3])
    out[s["rows"]] = sums
    return out[:-1]


def _weights(s):
    """The matrix of every (piece, component pair)."""
    return s["W"].float()[s["of"][:, None], s["pair"]].flatten(0, 1)


def _run_mix(s):
    case = s["case"]
    if own:
        from clebsch_gordan_tensor_amd import api

        into, out = _blocks(case["in"]), _blocks(case["out"])
        if not case["backward"]:
            return api.linear_grouped(into, out, s["index"], s["x"], s["W"])
        return api.linear_grouped_backward(into, out, s["index"], s["x"], s["W"], s["dy"])
    dtype, x, W = s["x"].dtype, _pieces(s, s["x"].float(), s["ic"]), _weights(s)
    if not case["backward"]:
        return _back(s, torch.bmm(x, W), s["oc"], _dim(case["out"])).to(dtype)
    dy = _pieces(s, s["dy"].float(), s["oc"])
    dx = _back(s, torch.bmm(dy, W.transpose(1, 2).contiguous()), s["ic"], _dim(case["in"]))
    parts = torch.bmm(x.transpose(1, 2).contiguous(), dy)
    pairs = s["W"].shape[1]
    dW = x.new_zeros(case["groups"] * pairs, *parts.shape[1:])
    dW.index_add_(0, (s["of"][:, None] * pairs + s["pair"]).flatten(), parts)
    return dx.to(dtype), dW.view(s["W"].shape)


def _run_norm(s):
    case = s["case"]
    if own:
        from clebsch_gordan_tensor_amd import api

        irreps, flags = _blocks(case["irreps"]), 0 if case["centered"] else api.E3_NORM_UNCENTERED
        if case["pass"] == "bwd":
            return api.layer_norm_residual_backward(irreps, s["x"], s["w"], s["dy"], s["dh"],
                                                    eps=EPS, flags=flags)
        call = api.layer_norm_residual if case["pass"] == "fwd" else api.layer_norm_fp8
        return call(irreps, s["x"], s["r"], s["w"], s["b"], eps=EPS, flags=flags)
    h = s["x"]
    if case["pass"] != "bwd":
        h = (h.float() + s["r"].float()).to(h.dtype)
    x, w = h.float(), s["w"][s["of"]]
    xc = x - x.mean(-1, keepdim=True) * s["center"]
    var = xc.square().mean(-1) @ s["share"]
    rstd = (1 / (var + EPS).sqrt())[..., None]
    if case["pass"] != "bwd":
        y = xc * rstd * w
        y[:, s["scalar"]] += s["b"]
        return (y.to(h.dtype), h) if case["pass"] == "fwd" else (*_quantize(y), h)
    dy = s["dy"].float()
    xh, g = xc * rstd, dy * w
    along = ((g * xh).mean(-1) @ s["share"])[..., None]
    dx = rstd * (g - g.mean(-1, keepdim=True) * s["center"] - xh * along) + s["dh"].float()
    return dx.to(h.dtype), s["one"] @ (dy * xh).sum(0), dy[:, s["scalar"]].sum(0)


def _run_fp8(s):
    case = s["case"]
    if own:
        from clebsch_gordan_tensor_amd import api

        q, scale = (s["q"], s["scale"]) if "q" in s else api.quantize_fp8(s["x"])
        return api.linear_fp8(_blocks(case["in"]), _blocks(case["out"]), q, scale, s["packed"],
                              index=s["index"], dtype=TYPES[case["dtype"]])
    q, scale = (s["q"], s["scale"]) if "q" in s else _quantize(s["x"])
    x = _pieces(s, _values(q, scale), s["ic"])
    y = _back(s, torch.bmm(x, _weights(s)), s["oc"], _dim(case["out"]))
    return y.to(TYPES[case["dtype"]])


# ------------------------------------------------------------------ what a pass needs

def work(case):
    rows = case["rows"]
    if case["op"] == "index":
        return {"bytes": 8 * rows + 4 * case["groups"], "flops": rows}
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        blocks = _blocks(case["irreps"])
        n = rows * _dim(case["irreps"]) * case["channels"]
        weights = 4 * case["channels"] * (len(blocks) + sum(b == (0, 1) for b in blocks))
        if case["pass"] == "bwd":
            return {"bytes": 4 * e * n + 2 * weights, "flops": 17 * n}
        if case["pass"] == "fwd":
            return {"bytes": 4 * e * n + weights, "flops": 9 * n}
        return {"bytes": (3 * e + 1 + 4 / RUN) * n + weights, "flops": 12 * n}
    cin, cout = case["cin"], case["cout"]
    into, out = rows * _dim(case["in"]) * cin, rows * _dim(case["out"]) * cout
    pairs = _pairs(case["in"], case["out"])
    flops = 2 * rows * cin * cout * sum(2 * _blocks(case["in"])[i][0] + 1 for i, _ in pairs)
    weights = min(rows, case["groups"]) * len(pairs) * cin * cout
    if case["op"] == "mix":
        if case["backward"]:
            return {"bytes": e * (2 * into + out) + (e + 4) * weights, "flops": 2 * flops}
        return {"bytes": e * (into + out + weights), "flops": flops}
    given = 1 + 4 / RUN if case["given"] == "codes" else 4 if case["given"] == "f32" else 2
    return {"bytes": given * into + e * out + weights, "flops": flops}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "index":
        return None
    if case["op"] == "norm":
        return _exact_norm(case, s)
    W = s["W"].double()
    if case["op"] == "mix":
        x = s["x"].double()
    else:
        x = _exact_values(s["x"].double()) if "x" in s else torch.cat(
            [c.double() * a[..., None].double() for c, a in zip(
                s["q"].float().split(RUN, -1), s["scale"].unbind(-1))], -1)
    y = x.new_zeros(case["rows"], _dim(case["out"]), case["cout"])
    dx, dW = torch.zeros_like(x), torch.zeros_like(W)
    dy = s["dy"].double() if "dy" in s else None
    for g in range(case["groups"]):
        of = torch.nonzero(s["ids"] == g)[:, 0] if "ids" in s else torch.arange(
            case["rows"], device="cuda")
        for p, (i, o) in enumerate(_pairs(case["in"], case["out"])):
            for m in range(2 * _blocks(case["in"])[i][0] + 1):
                a, b = _starts(case["in"])[i] + m, _starts(case["out"])[o] + m
                if dy is None:
                    y[of, b] += x[of, a] @ W[g, p]
                else:
                    dx[of, a] += dy[of, b] @ W[g, p].T
                    dW[g, p] += x[of, a].T @ dy[of, b]
    return y if dy is None else (dx, dW)


def _exact_values(v):
    """The 8-bit form of 64-bit values, read back."""
    out = []
    for run in v.split(RUN, -1):
        scale = (run.abs().max(-1, keepdim=True).values.float() / 448).clamp(min=2 ** -126).double()
        out.append((run / scale).to(torch.float8_e4m3fn).double() * scale)
    return torch.cat(out, -1)


def _exact_norm(case, s):
    x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
    back = case["pass"] == "bwd"
    if not back:
        x = (x + s["r"].double()).to(s["x"].dtype).double()  # held in the storage type
    at, scalar, ys, dxs, dws, dbs = 0, 0, [], [], [], []
    for i, (l, parity) in enumerate(_blocks(case["irreps"])):
        seg = x[:, at:at + 2 * l + 1]
        bias = (l, parity) == (0, 1)
        if bias and case["centered"]:
            seg = seg - seg.mean(2, keepdim=True)
        size = (seg.square().mean((1, 2), keepdim=True) + EPS).sqrt()
        unit = seg / size
        if not back:
            ys.append(unit * w[i] + (b[scalar] if bias else 0.0))
        else:
            d = s["dy"][:, at:at + 2 * l + 1].double()
            g = d * w[i]
            t = g - unit * (g * unit).mean((1, 2), keepdim=True)
            if bias and case["centered"]:
                t = t - g.mean(2, keepdim=True)
            dxs.append(t / size + s["dh"][:, at:at + 2 * l + 1].double())
            dws.append((d * unit).sum((0, 1)))
            if bias:
                dbs.append(d.sum((0, 1)))
        at, scalar = at + 2 * l + 1, scalar + bias
    if back:
        return torch.cat(dxs, 1), torch.stack(dws), (
            torch.stack(dbs) if dbs else x.new_zeros((0, x.shape[2])))
    y = torch.cat(ys, 1)
    if case["pass"] == "fwd":
        return y, x
    scale = torch.stack([r.abs().amax(-1) / TOP for r in y.split(RUN, -1)], -1).clamp(min=LEAST)
    q = torch.cat([r / a[..., None] for r, a in zip(y.split(RUN, -1), scale.unbind(-1))], -1)
    return q, scale, x
