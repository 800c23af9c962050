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
