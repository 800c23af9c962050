"""Plain 64-bit forms of the normalisation of irreps features, of its
gradients and of the AdamW step (numpy), with the error that float32
arithmetic may make in each result, element by element."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24       # half a step of float32, relative
U_BF16 = 2.0 ** -8   # of bfloat16

# Operations a float32 sum over a segment passes a value through: at most 17 x 4
# products added in one lane, 6 + 4 joining steps of lanes and wavefronts, and
# the handful of products, divisions and roots before and after.
SEGMENT = 96


def blocks_of(irreps):
    at, scalar, out = 0, 0, []
    for l, p in irreps:
        bias = scalar if (l, p) == (0, 1) else -1
        scalar += bias >= 0
        out.append((at, 2 * l + 1, bias))
        at += 2 * l + 1
    return out


def _block(x, at, nc, centered, eps):
    seg = x[:, at:at + nc].astype(np.float64)
    xc = seg - seg.mean((1, 2), keepdims=True) if centered else seg
    rstd = 1.0 / np.sqrt((xc ** 2).mean((1, 2), keepdims=True) + eps)
    # error of xh = xc rstd in units of SEGMENT * U
    e = rstd * np.abs(seg).mean((1, 2), keepdims=True) * centered + np.abs(xc * rstd)
    return xc * rstd, rstd, e


def norm_forward(irreps, x, w, b, eps, centered=True):
    """(y, bound)"""
    y, tol = np.zeros(x.shape), np.zeros(x.shape)
    for i, (at, nc, bias) in enumerate(blocks_of(irreps)):
        xh, _, e = _block(x, at, nc, centered and bias >= 0, eps)
        y[:, at:at + nc] = xh * w[i] + (b[bias] if bias >= 0 else 0.0)
        tol[:, at:at + nc] = SEGMENT * U * e * np.abs(w[i])
    return y, tol + U * np.abs(y)


def norm_backward(irreps, x, w, dy, eps, centered=True):
    """((dx, dweight, dbias), their bounds)"""
    rows, _, C = x.shape
    blocks = blocks_of(irreps)
    scalars = sum(b >= 0 for _, _, b in blocks)
    dx, tx = np.zeros(x.shape), np.zeros(x.shape)
    dw, tw = np.zeros((len(blocks), C)), np.zeros((len(blocks), C))
    db, tb = np.zeros((scalars, C)), np.zeros((scalars, C))
    for i, (at, nc, bias) in enumerate(blocks):
        c = centered and bias >= 0
        xh, rstd, e = _block(x, at, nc, c, eps)
        d = dy[:, at:at + nc].astype(np.float64)
        g = d * w[i]
        mean = lambda t: t.mean((1, 2), keepdims=True)  # noqa: E731
        along, mg = mean(g * xh), mean(g) * c
        dx[:, at:at + nc] = rstd * (g - mg - xh * along)
        tx[:, at:at + nc] = SEGMENT * U * rstd * (
            np.abs(g) + mean(np.abs(g)) + np.abs(xh) * (mean(np.abs(g * xh)) + mean(np.abs(g) * e))
            + e * np.abs(along) + np.abs(g - mg - xh * along))
        n = rows * nc + SEGMENT  # values a sum over rows passes through, at most
        dw[i] = (d * xh).sum((0, 1))
        tw[i] = n * U * np.abs(d * xh).sum((0, 1)) + SEGMENT * U * (np.abs(d) * e).sum((0, 1))
        if bias >= 0:
            db[bias], tb[bias] = d.sum((0, 1)), n * U * np.abs(d).sum((0, 1))
    return (dx, dw, db), (tx + U * np.abs(dx), tw, tb)


# dweight and dbias over many rows, each workgroup taking several turns over them:
# (irreps, channels, storage type, rows, channels of a component row that a lane holds, roundings
# that a term of the sums passes through, at most).  The last, term by term: adds of a lane over
# its rows and components, joins of lanes and teams, adds of every 64th partial, 32 + 1 last ones.
LONG_SUMS = [
    # a block a workgroup: 170, 512 and 853 of them, 8 teams of 32 lanes; 8, 9, 10 + 1 + 4 + 14 + 33
    ("0e+1o+2e", 128, "f32", 10007, 4, 62),
    # scalars: 256 workgroups, 8 teams of two rows; 10 + 1 + 4 + 4 + 33
    ("0e", 128, "f32", 20011, 4, 52),
    # four vectors a lane, 4 teams; 5 + 4 + 4 + 33
    ("0e", 1001, "f32", 5003, 16, 46),
    # a team of four wavefronts; 12 + 4 + 33
    ("0e", 2050, "bf16", 3001, 16, 49),
    # whole rows: 2048 workgroups, 16 or 8 teams, two turns; 3 + 2 + 4 + 4 + 32 + 33
    ("0e+1o", 60, "f32", 40003, 4, 78),
    ("0e+1o", 100, "bf16", 20011, 4, 78),
    # staged rows, 64 (128 in bf16) a piece in 9 groups: 8 (15) + 3 + 1 + 6 + 16 + 33
    ("0e+1o+2e", 3, "f32", 70001, 4, 67),
    ("0e+1o+2e", 3, "bf16", 140003, 4, 74),
]


def long_sums(irreps, x, dy, eps, lane, depth, centered=True):
    """[(dweight terms of every row [rows][C], dweight, its bound)] of the
    blocks and the same of dbias for the 0e ones."""
    dw, db = [], []
    for at, nc, bias in blocks_of(irreps):
        c = centered and bias >= 0
        xh, _, e = _block(x, at, nc, c, eps)
        d = dy[:, at:at + nc].astype(np.float64)
        # xh: sums over what a lane holds of the segment, then at most 6 + 4 joins and 6 other
        # roundings (the root halves the error of its argument)
        segment = lane * nc + 16
        tol = depth * U * np.abs(d * xh).sum((0, 1)) + segment * U * (np.abs(d) * e).sum((0, 1))
        terms = (d * xh).sum(1)
        dw.append((terms, terms.sum(0), tol))
        if bias >= 0:
            db.append((d[:, 0], d.sum((0, 1)), depth * U * np.abs(d).sum((0, 1))))
    return dw, db


def long_case(irreps, C, dtype, rows):
    """x and dy of a case of LONG_SUMS."""
    from clebsch_gordan_tensor_amd import synth as S
    rng = np.random.default_rng(rows + C)
    dim = sum(2 * l + 1 for l, _ in irreps)
    x = rng.standard_normal((rows, dim, C)) * rng.uniform(0.1, 3.0, (rows, 1, 1)) + 0.2
    x, dy = x.astype(np.float32), rng.standard_normal((rows, dim, C)).astype(np.float32)
    return (S.round_bf16(x), S.round_bf16(dy)) if dtype == "bf16" else (x, dy)


# ------------------------------------------------------------------ optimizer

def decode(m, v, ms, vs):
    """The moments that 8-bit codes and scales of one tensor stand for."""
    n = m.size
    sm = np.repeat(ms.astype(np.float64), 256)[:n]
    sv = np.repeat(vs.astype(np.float64), 256)[:n]
    cm, cv = m.astype(np.float64), v.astype(np.float64)
    return sm * (cm * np.abs(cm)), (sv * cv ** 2) ** 2


def _runs(x):
    n = x.size
    return np.concatenate([x, np.zeros(-n % 256)]).reshape(-1, 256)


def scales(m, v):
    """float32 scales of the runs of 256 of a tensor's moments."""
    a = np.abs(_runs(m)).max(1).astype(np.float32).astype(np.float64)
    b = _runs(v).max(1).astype(np.float32).astype(np.float64)
    return (a / 127 ** 2).astype(np.float32), (np.sqrt(b) / 255 ** 2).astype(np.float32)


def borders(top, scale, power):
    """Borders between the codes 0..top of one run."""
    k = np.arange(top) + 0.5
    return scale * k ** 2 if power == 1 else (scale * k ** 2) ** 2


def codes(value, scale, top, power):
    """Codes of the values of one tensor under given scales; and whether a
    value is so near a border (1e-13 of it) that 64 bits do not decide."""
    out, near = [np.zeros(0, np.int64)], [np.zeros(0, bool)]
    for run, s in zip(_runs(value), scale.astype(np.float64)):
        b = borders(top, s, power)
        c = np.searchsorted(b, run, side="left")
        out.append(c)
        near.append((np.abs(run[:, None] - b[None, :]) <= 1e-13 * b[None, :]).any(1))
    return (np.concatenate(out)[:value.size], np.concatenate(near)[:value.size])


def adamw(p, g, m, v, t, lr, wd, b1=0.9, b2=0.999, eps=1e-8, scale=1.0):
    """(p, m, v) after the step, and the bounds of the float32 forms."""
    p, g, m, v = (a.astype(np.float64) for a in (p, g, m, v))
    g = g * scale
    gm, gv = (1 - b1) * g, (1 - b2) * g * g
    nm, nv = b1 * m + gm, b2 * v + gv
    # the betas, their complements, the scaled gradient and the products are rounded once each
    tm = 5 * U * (np.abs(b1 * m) + np.abs(gm))
    tv = 8 * U * (b2 * v + gv)
    size, c2 = lr / (1 - b1 ** t), 1 - b2 ** t
    d = np.sqrt(nv / c2) + eps
    new = p - lr * wd * p - size * nm / d
    # root and reciprocal are off by a step (2 U) each, v by tv, the rest rounds once
    tp = U * np.abs(new) + 4 * U * np.abs(lr * wd * p) + size / d * tm + 16 * U * np.abs(
        size * nm / d)
    return (new, nm, nv), (tp, tm, tv)
