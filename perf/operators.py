"""Cases of the training operators: normalisation of irreps features with its
gradients, the norm of all gradients with its clip factor, and the AdamW step
over many tensors with moments in 32 or in 8 bits.

``run`` computes a case in its plain form (elementary torch operations), or,
where ``own`` is true, through the package's entry points.  Inputs come from
the seed alone.  Features are laid out [rows][components][channels], an irrep
of degree l having 2l+1 components; parameters are tensors of one flat buffer
each, so that a case of many tensors gives back one buffer for all of them.
"""
import math

import torch

own = False

EPS_NORM = 1e-5
BETA1, BETA2, EPS_ADAM, LR, DECAY, MAX_NORM = 0.9, 0.999, 1e-8, 1e-3, 0.01, 1.0
BLOCK = 256  # consecutive elements of a tensor that share the scale of their 8-bit moments
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# The weights of a network of these layers at 128 channels: per layer the channel mixing of
# 0e+1o+2e+3o (4 x 128 x 128), of 0e+1o (2 x 128 x 128), the radial MLP (8 x 64, 64 x 1280) and,
# without decay, the normalisation's weights and biases.
LAYER = "65536 32768 512 81920"
NORMS = "512 128"


def listed():
    return [
        # the tiny configuration's features: latency of one call, gradients included
        {"name": "norm bwd tiny", "op": "norm", "backward": True, "rows": 64, "channels": 8,
         "irreps": "0e+1o", "dtype": "f32", "centered": True},
        # the messages of the 3,000-atom box, as the network normalises them after a convolution
        {"name": "norm fwd water3k", "op": "norm", "backward": False, "rows": 3000,
         "channels": 128, "irreps": "0e+1o+2e+3o", "dtype": "f32", "centered": True},
        # the messages of the 64,000-atom system
        {"name": "norm fwd mace64k", "op": "norm", "backward": False, "rows": 64000,
         "channels": 128, "irreps": "0e+1o+2e+3o", "dtype": "f32", "centered": True},
        {"name": "norm bwd mace64k", "op": "norm", "backward": True, "rows": 64000,
         "channels": 128, "irreps": "0e+1o+2e+3o", "dtype": "f32", "centered": True},
        # the higher-order configuration: bf16 storage, 64 channels, scalars not centred
        {"name": "norm bwd ho20k bf16", "op": "norm", "backward": True, "rows": 20000,
         "channels": 64, "irreps": "0e+1o+2e+3o", "dtype": "bf16", "centered": False},
        # ordinary layer norm of wide scalars, an odd width and a ragged count of rows
        {"name": "norm bwd scalars odd", "op": "norm", "backward": True, "rows": 20011,
         "channels": 1001, "irreps": "0e", "dtype": "f32", "centered": True},
        # all gradients of a two-layer network, and of a large one with bf16 gradients
        {"name": "grad norm network", "op": "grad_norm", "grad": "f32", "pad": 256,
         "sizes": " ".join([LAYER, LAYER, NORMS, NORMS])},
        {"name": "grad norm large bf16", "op": "grad_norm", "grad": "bf16", "pad": 256,
         "sizes": "100000007 30000001 65536 129"},
        # clipped update of the two-layer network's weights, moments in 32 bits
        {"name": "adamw network", "op": "adamw", "bits": 32, "grad": "f32", "pad": 256, "clip": True,
         "copy": False, "sizes": " ".join([LAYER, LAYER, NORMS, NORMS]), "undecayed": 4, "step": 10},
        # a large update with tensors packed end to end (any alignment) and bf16 copies
        {"name": "adamw large packed", "op": "adamw", "bits": 32, "grad": "f32", "pad": 1,
         "clip": False, "copy": True, "sizes": "40000001 20000003 999999 333 77", "undecayed": 2,
         "step": 1000},
        # twelve layers, moments in 8 bits, clipped
        {"name": "adamw8 network", "op": "adamw", "bits": 8, "grad": "f32", "pad": 256, "clip": True,
         "copy": False, "sizes": " ".join([LAYER] * 12 + [NORMS] * 12), "undecayed": 24,
         "step": 10},
        # a large update, moments in 8 bits, gradients in bf16
        {"name": "adamw8 large", "op": "adamw", "bits": 8, "grad": "bf16", "pad": 256, "clip": False,
         "copy": False, "sizes": "67108864 30000001 4194304 1000 1", "undecayed": 2, "step": 1000},
    ]


def _span(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm", "grad_norm", "adamw", "adamw8"))
    if op == "norm":
        irreps = rng.choice(("0e", "0e", "1o", "0e+1o", "0e+1o+2e", "0e+1o+2e+3o", "0e+0o+0e+1e",
                             "0e+1o+1e+2e+2o+3o+3e", "0e+1o+2e+3o+4e+5o+6e"))
        channels = _span(rng, 1, 1024)
        rows = _span(rng, 1, max(1, min(400000, 100_000_000 // (channels * _dim(irreps)))))
        return {"op": op, "backward": rng.random() < 0.6, "rows": rows, "channels": channels,
                "irreps": irreps, "dtype": rng.choice(("f32", "f32", "bf16")),
                "centered": rng.random() < 0.8}
    n = _span(rng, 1, 150)
    total = _span(rng, 1000, 50_000_000)
    parts = [rng.random() ** 4 + 1e-4 for _ in range(n)]
    sizes = [max(1, round(total * q / sum(parts))) for q in parts]
    case = {"op": op[:9], "grad": rng.choice(("f32", "bf16")), "pad": rng.choice((1, 4, 256)),
            "sizes": " ".join(map(str, sizes))}
    if op == "grad_norm":
        return case
    bits = 8 if op == "adamw8" else 32
    return {**case, "op": "adamw", "bits": bits, "pad": 256 if bits == 8 else case["pad"],
            "clip": rng.random() < 0.5, "copy": rng.random() < 0.3,
            "undecayed": rng.randrange(n + 1), "step": _span(rng, 1, 100000)}


# ------------------------------------------------------------------ inputs

def _blocks(irreps):
    """[(degree, parity)] of a text such as 0e+1o."""
    return [(int(b[:-1]), 1 if b[-1] == "e" else -1) for b in irreps.split("+")]


def _dim(irreps):
    return sum(2 * l + 1 for l, _ in _blocks(irreps))


def _offsets(case):
    """Where each tensor starts in the flat buffers, and how long these are."""
    at, starts = 0, []
    for n in map(int, case["sizes"].split()):
        starts.append((at, n))
        at += -(-n // case["pad"]) * case["pad"]
    return starts, at


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    return _prepare_norm(case, rand) if case["op"] == "norm" else _prepare_params(case, rand)


def _prepare_norm(case, rand):
    blocks, C, rows = _blocks(case["irreps"]), case["channels"], case["rows"]
    dtype, dim = TYPES[case["dtype"]], _dim(case["irreps"])
    scalars = sum(b == (0, 1) for b in blocks)
    # features of differing size from row to row, off zero
    x = rand(rows, dim, C) * (0.2 + rand(rows, 1, 1).square()) + 0.3
    s = {"case": case, "x": x.to(dtype), "w": 1 + 0.1 * rand(len(blocks), C),
         "b": 0.1 * rand(scalars, C)}
    if case["backward"]:
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


def _prepare_params(case, rand):
    starts, total = _offsets(case)
    ends = [at + n for at, n in starts]
    inside = torch.zeros(total + 1, device="cuda", dtype=torch.int32)
    inside[torch.tensor([at for at, _ in starts], device="cuda")] += 1
    inside[torch.tensor(ends, device="cuda")] -= 1
    inside = (inside.cumsum(0)[:total] > 0).float()
    s = {"case": case, "starts": starts,
         "g": (rand(total) * torch.exp(1.5 * rand(total)) * 1e-3 * inside).to(TYPES[case["grad"]])}
    if case["op"] == "grad_norm":
        if own:
            s["params"] = _params(s)
        return s
    s["t"] = case["step"] - 1
    # the tensors without decay come last
    s["decayed"] = starts[len(starts) - case["undecayed"]][0] if case["undecayed"] else total
    s["p"] = 0.1 * rand(total) * inside
    # what earlier steps with gradients of this size leave
    m, v = 3e-4 * rand(total) * inside, (1e-3 * rand(total)).square() * inside
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        s["m"], s["ms"] = _encode_m(m.double())
        s["v"], s["vs"] = _encode_v(v.double())
    if case["copy"]:
        s["copy"] = s["p"].to(torch.bfloat16)
    if own:
        s["params"] = _params(s)
        if case["bits"] == 8:
            s["mv"] = tuple(torch.zeros(total, device="cuda") for _ in range(2))
            s["views"] = [[t[at:at + n] for at, n in starts] for t in s["mv"]]
    return s


def _params(s):
    """The package's handle on the tensors of a case."""
    from clebsch_gordan_tensor_amd import api

    views = lambda key: [s[key][at:at + n] for at, n in s["starts"]] if key in s else None  # noqa: E731
    scales = lambda key: ([s[key][at // BLOCK:-(-(at + n) // BLOCK)] for at, n in s["starts"]]  # noqa: E731
                          if key in s else None)
    if "p" not in s:
        return api.Params(grads=views("g"))
    k = len(s["starts"]) - s["case"]["undecayed"]
    return api.Params(params=views("p"), grads=views("g"), m=views("m"), v=views("v"),
                      m_scale=scales("ms"), v_scale=scales("vs"), copies=views("copy"),
                      weight_decay=[DECAY if i < k else 0.0 for i in range(len(s["starts"]))])


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return _run_norm(state)
    return _run_grad_norm(state) if op == "grad_norm" else _run_adamw(state)


def _run_norm(s):
    case = s["case"]
    if own:
        from clebsch_gordan_tensor_amd import api

        irreps, flags = _blocks(case["irreps"]), 0 if case["centered"] else api.E3_NORM_UNCENTERED
        if not case["backward"]:
            return api.layer_norm(irreps, s["x"], s["w"], s["b"], eps=EPS_NORM, flags=flags)
        return api.layer_norm_backward(irreps, s["x"], s["w"], s["dy"], eps=EPS_NORM, flags=flags)
    x, w = s["x"].float(), s["w"][s["of"]]
    xc = x - x.mean(-1, keepdim=True) * s["center"]
    var = xc.square().mean(-1) @ s["share"]
    rstd = (1 / (var + EPS_NORM).sqrt())[..., None]
    if not case["backward"]:
        y = xc * rstd * w
        y[:, s["scalar"]] += s["b"]
        return y.to(s["x"].dtype)
    dy = s["dy"].float()
    xh, g = xc * rstd, dy * w
    along = ((g * xh).mean(-1) @ s["share"])[..., None]
    dx = rstd * (g - g.mean(-1, keepdim=True) * s["center"] - xh * along)
    return (dx.to(s["x"].dtype), s["one"] @ (dy * xh).sum(0), dy[:, s["scalar"]].sum(0))


def _run_grad_norm(s):
    if own:
        from clebsch_gordan_tensor_amd import api

        return api.grad_norm(s["params"], max_norm=MAX_NORM)
    return _norm_and_factor(s["g"])


def _norm_and_factor(g):
    # a long sum, and the factor decides between 8-bit codes: 64 bits, rounded once
    norm = g.double().square().sum().sqrt()
    return torch.stack([norm, (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)]).float()


def _run_adamw(s):
    case = s["case"]
    s["t"] += 1
    out = {"p": s["p"]}
    if own:
        from clebsch_gordan_tensor_amd import api

        if case["clip"]:
            out["norm"] = api.grad_norm(s["params"], max_norm=MAX_NORM)
        api.adamw(s["params"], s["t"], LR, beta1=BETA1, beta2=BETA2, eps=EPS_ADAM,
                  grad_scale=out["norm"][1:] if case["clip"] else None)
        if case["bits"] == 8:
            api.adamw_moments(s["params"], *s["views"])
            out["m"], out["v"] = s["mv"]
    elif case["bits"] == 32:
        g = s["g"].float()
        if case["clip"]:
            out["norm"] = _norm_and_factor(s["g"])
            g = g * out["norm"][1]
        s["m"].mul_(BETA1).add_(g * (1 - BETA1))
        s["v"].mul_(BETA2).add_(g * g * (1 - BETA2))
        _update(s, s["m"], s["v"])
    else:
        # which 8-bit code a moment takes must not hang on its 32-bit rounding: 64 bits
        g = s["g"].double()
        if case["clip"]:
            out["norm"] = _norm_and_factor(s["g"])
            g = g * out["norm"][1].double()
        m = BETA1 * _decode_m(s["m"], s["ms"]) + (1 - BETA1) * g
        v = BETA2 * _decode_v(s["v"], s["vs"]) + (1 - BETA2) * g * g
        s["m"], s["ms"] = _encode_m(m)
        s["v"], s["vs"] = _encode_v(v)
        _update(s, m.float(), v.float())
        out["m"] = _decode_m(s["m"], s["ms"]).float()
        out["v"] = _decode_v(s["v"], s["vs"]).float()
    if case["bits"] == 32:
        out["m"], out["v"] = s["m"], s["v"]
    if case["copy"]:
        if not own:
            s["copy"] = s["p"].to(torch.bfloat16)
        out["copy"] = s["copy"]
    return out


def _update(s, m, v):
    c1, c2 = 1 - BETA1 ** s["t"], 1 - BETA2 ** s["t"]
    s["p"][:s["decayed"]] *= 1 - LR * DECAY
    s["p"] -= LR * (m / c1) / ((v / c2).sqrt() + EPS_ADAM)


def _encode_m(m):
    """Codes in [-127, 127] and scales of blocks of first moments: value = scale c |c|."""
    a = m.abs().view(-1, BLOCK)
    scale = (a.amax(1, keepdim=True).float().double() / 127 ** 2).float()
    s = scale.double()
    c = (a / s).sqrt().nan_to_num(0.0).round().clamp(max=127)
    # the border between two codes belongs to the lower one
    c = c - (s * (c - 0.5).square() >= a).double() * (c > 0)
    c = (c + (s * (c + 0.5).square() < a).double()).clamp(max=127)
    return (c.view(-1) * m.sign()).to(torch.int8), scale.view(-1)


def _decode_m(code, scale):
    c = code.double()
    return (scale.double()[:, None] * (c * c.abs()).view(-1, BLOCK)).view(-1)


def _encode_v(v):
    """Codes in [0, 255] and scales of blocks of second moments: value = (scale c^2)^2, and what
    is not zero has a code of 1 at least."""
    v = v.view(-1, BLOCK)
    scale = (v.amax(1, keepdim=True).float().double().sqrt() / 255 ** 2).float()
    s = scale.double()
    c = (v.sqrt() / s).sqrt().nan_to_num(0.0).round().clamp(max=255)
    c = c - ((s * (c - 0.5).square()).square() >= v).double() * (c > 0)
    c = (c + ((s * (c + 0.5).square()).square() < v).double()).clamp(max=255)
    return torch.maximum(c, (v > 0).double()).to(torch.uint8).view(-1), scale.view(-1)


def _decode_v(code, scale):
    c = code.double()
    return (scale.double()[:, None] * c.square().view(-1, BLOCK)).square().view(-1)


# ------------------------------------------------------------------ what a pass needs

def work(case):
    if case["op"] == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        blocks = _blocks(case["irreps"])
        n = case["rows"] * _dim(case["irreps"]) * case["channels"]
        weights = 4 * case["channels"] * (len(blocks) + sum(b == (0, 1) for b in blocks))
        if case["backward"]:
            return {"bytes": 3 * e * n + 2 * weights, "flops": 16 * n}
        return {"bytes": 2 * e * n + weights, "flops": 8 * n}
    n = sum(map(int, case["sizes"].split()))
    g = 2 if case["grad"] == "bf16" else 4
    if case["op"] == "grad_norm":
        return {"bytes": g * n + 8, "flops": 2 * n}
    b = g + 8 + (2 if case["copy"] else 0)
    # 8 bits: codes and scales read and written, and the moments given back as values
    b += 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 8
    return {"bytes": b * n, "flops": (15 if case["bits"] == 32 else 40) * n}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm":
        return _exact_norm(case, s)
    g = s["g"].double()
    norm = torch.linalg.vector_norm(g)
    factor = min(1.0, MAX_NORM / (float(norm) + 1e-6))
    both = torch.stack([norm, norm.new_tensor(factor)])
    if case["op"] == "grad_norm":
        return both
    out = {"norm": both} if case["clip"] else {}
    if case["clip"]:
        g *= float(both.float()[1])  # the factor is held in 32 bits
    if case["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        k = torch.arange(0, 256, device="cuda", dtype=torch.float64)
        cm, cv = s["m"].reshape(-1).long(), s["v"].reshape(-1).long()
        m = (k ** 2)[cm.abs()] * cm.sign() * s["ms"].double().repeat_interleave(BLOCK)
        v = (k ** 4)[cv] * s["vs"].double().repeat_interleave(BLOCK) ** 2
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g ** 2, v, BETA2)
    t = case["step"]
    decay = torch.ones_like(m)
    decay[:s["decayed"]] -= LR * DECAY
    out["p"] = decay * s["p"].double() - LR / (1 - BETA1 ** t) * m / (
        torch.sqrt(v / (1 - BETA2 ** t)) + EPS_ADAM)
    if case["copy"]:
        out["copy"] = out["p"]
    if case["bits"] == 32:
        return {**out, "m": m, "v": v}
    k = torch.arange(0.5, 255, 1, device="cuda", dtype=torch.float64)
    top = lambda t: t.view(-1, BLOCK).max(1, keepdim=True).values.float().double()  # noqa: E731
    sm = (top(m.abs()) * (1.0 / 16129)).float().double()
    sv = (top(v).sqrt() * (1.0 / 65025)).float().double()
    cm = torch.searchsorted(k[:127] ** 2, m.abs().view(-1, BLOCK) / sm)
    cv = torch.searchsorted(k ** 4, v.view(-1, BLOCK) / sv ** 2)
    cv = torch.where(v.view(-1, BLOCK) > 0, cv.clamp(min=1), 0)
    out["m"] = torch.where(sm > 0, sm * cm ** 2, 0.0).view(-1) * m.sign()
    out["v"] = torch.where(sv > 0, sv ** 2 * cv.double() ** 4, 0.0).view(-1)
    return out


def _exact_norm(case, s):
    x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
    dy = s["dy"].double() if case["backward"] else None
    at, scalar, ys, dxs, dws, dbs = 0, 0, [], [], [], []
    for i, (l, parity) in enumerate(_blocks(case["irreps"])):
        seg = x[:, at:at + 2 * l + 1]
        bias = (l, parity) == (0, 1)
        if bias and case["centered"]:
            seg = seg - seg.mean(2, keepdim=True)
        size = (seg.square().mean((1, 2), keepdim=True) + EPS_NORM).sqrt()
        unit = seg / size
        if dy is None:
            ys.append(unit * w[i] + (b[scalar] if bias else 0.0))
        else:
            d = dy[:, at:at + 2 * l + 1]
            g = d * w[i]
            back = g - unit * (g * unit).mean((1, 2), keepdim=True)
            if bias and case["centered"]:
                back = back - g.mean(2, keepdim=True)
            dxs.append(back / size)
            dws.append((d * unit).sum((0, 1)))
            if bias:
                dbs.append(d.sum((0, 1)))
        at, scalar = at + 2 * l + 1, scalar + bias
    if dy is None:
        return torch.cat(ys, 1)
    return torch.cat(dxs, 1), torch.stack(dws), torch.stack(dbs) if dbs else x.new_zeros((0, x.shape[2]))
