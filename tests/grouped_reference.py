"""Plain 64-bit forms of the operators on grouped rows and on 8-bit features
(numpy), and the error that the kernels' arithmetic may make in them."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24       # half a step of float32, relative
U_BF16 = 2.0 ** -8   # of bfloat16
# A product of float32 values on the matrix cores is six products of bf16
# parts, so that a sum over K terms is one of 6 K; what the parts leave out is
# below 2^-26 of a product, less than one rounding.
ADDS = 6


def blocks(irreps):
    """[(first component, components)]"""
    at, out = 0, []
    for l, _ in irreps:
        out.append((at, 2 * l + 1))
        at += 2 * l + 1
    return out


def pairs(into, out):
    return [(i, o) for i, a in enumerate(into) for o, b in enumerate(out) if a == b]


def index(group, n_groups):
    """(order, offsets)"""
    key = np.where((group >= 0) & (group < n_groups), group, n_groups)
    n = np.bincount(key, minlength=n_groups + 1)[:n_groups]
    return np.argsort(key, kind="stable"), np.concatenate([[0], np.cumsum(n)])


def mix(into, out, group, x, W):
    """(y, sum of the terms' sizes, largest number of terms)"""
    x, W = x.astype(np.float64), W.astype(np.float64)
    bi, bo = blocks(into), blocks(out)
    y = np.zeros((x.shape[0], sum(n for _, n in bo), W.shape[3]))
    size, terms = np.zeros_like(y), np.zeros(len(out), int)
    for p, (i, o) in enumerate(pairs(into, out)):
        terms[o] += x.shape[2]
        for g in range(W.shape[0]):
            r = np.nonzero(group == g)[0]
            a = x[r, bi[i][0]:bi[i][0] + bi[i][1]]
            y[r, bo[o][0]:bo[o][0] + bo[o][1]] += a @ W[g, p]
            size[r, bo[o][0]:bo[o][0] + bo[o][1]] += np.abs(a) @ np.abs(W[g, p])
    return y, size, terms.max()


def mix_backward(into, out, group, x, W, dy):
    """((dx, sizes, terms), (dW, sizes, terms))"""
    x, W, dy = (t.astype(np.float64) for t in (x, W, dy))
    bi, bo = blocks(into), blocks(out)
    dx, sx, tx = np.zeros_like(x), np.zeros_like(x), np.zeros(len(into), int)
    dW, sW, tW = np.zeros_like(W), np.zeros_like(W), 0
    for p, (i, o) in enumerate(pairs(into, out)):
        tx[i] += W.shape[3]
        (a, n), (b, _) = bi[i], bo[o]
        for g in range(W.shape[0]):
            r = np.nonzero(group == g)[0]
            d, v = dy[r, b:b + n], x[r, a:a + n]
            dx[r, a:a + n] += d @ W[g, p].T
            sx[r, a:a + n] += np.abs(d) @ np.abs(W[g, p].T)
            d, v = d.reshape(-1, d.shape[2]), v.reshape(-1, v.shape[2])
            dW[g, p] = v.T @ d
            sW[g, p] = np.abs(v).T @ np.abs(d)
            tW = max(tW, len(v))
    return (dx, sx, tx.max()), (dW, sW, tW)


# What the 8-bit matrix cores drop of a sum: below 2^-13 of the largest of 8
# consecutive products, of each of the other 7.
EIGHTS = 7 * 2.0 ** -13


def check(got, ref, what, bf16=False, adds=ADDS, drops=0.0):
    """Every element within one rounding for each add of its terms' sizes
    (and half a step of bf16), and float32 results within what independent
    roundings of their partial sums come to together: the sum of n terms of
    size s passes through partial sums of size s sqrt(j), each rounded by U at
    most, so its error is U s n / 2 at most in the root mean square, for a
    result of s sqrt(n).  drops: of the terms' sizes, besides; results in bf16
    are then held in the root mean square as well, to that of the rounding to
    bf16 (half a step at most, even spread) and an eighth of it."""
    y, size, terms = ref
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == y.shape, what
    err = np.abs(got - y)
    n = adds * terms + 16
    tol = (n * U + drops) * size + (U_BF16 * np.maximum(np.abs(y), np.abs(got)) if bf16 else U * np.abs(y))
    worst = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
    rms = float(np.sqrt((err ** 2).mean())) if err.size else 0.0
    most = float(U * np.sqrt(n + 48) / 2 * np.sqrt((y ** 2).mean())) if err.size else 0.0
    print(f"[err] {what}: {worst:.4f} of the bound, rms {rms:.3e} of {most:.3e}", flush=True)
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} outside, worst {worst:.2f}"
    # (the rows' sizes differ and so do the groups' lengths: a factor of 2)
    if drops:
        most = U_BF16 / 3 ** 0.5 * float(np.sqrt((y ** 2).mean())) * 1.125 / 2
    assert (bf16 and not drops) or rms <= 2 * most, f"{what}: rms {rms:.3e} over {2 * most:.3e}"


# ------------------------------------------------------------------ 8 bits

def e4m3(t):
    """float32 values of at most 448 (1 + 2^-20) rounded to e4m3, ties to even."""
    t = np.asarray(t, dtype=np.float64)
    _, e = np.frexp(t)  # |t| in [2^(e-1), 2^e)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(t / step) * step


def runs(v):
    """[(slice, run)] of the last axis."""
    return [slice(k, min(k + 128, v.shape[-1])) for k in range(0, v.shape[-1], 128)]


def _scale(top):
    with np.errstate(invalid="ignore", over="ignore"):
        s = (top * (np.float32(1) / np.float32(448))).astype(np.float32)
    return np.where(s < np.float32(2.0 ** -126), np.float32(2.0 ** -126), s)


def quantize(x):
    """(codes' values, scales) of float32 x [...][C], as e3_quantize_fp8 defines them."""
    q = np.zeros(x.shape)
    scale = np.zeros((*x.shape[:-1], len(runs(x))), np.float32)
    for b, k in enumerate(runs(x)):
        v = x[..., k]
        s = _scale(np.abs(v).max(-1))
        bad = ~np.isfinite(v).all(-1)
        scale[..., b] = np.where(bad, np.float32(np.nan), s)
        with np.errstate(invalid="ignore"):
            q[..., k] = np.where(bad[..., None], np.nan, e4m3(v / s[..., None]))
    return q, scale


def quantize_weights(W):
    """The same of the 128 x 128 blocks of W [...][Cin][Cout]."""
    q = np.zeros(W.shape)
    scale = np.zeros((*W.shape[:-2], -(-W.shape[-1] // 128), -(-W.shape[-2] // 128)), np.float32)
    for a in range(scale.shape[-1]):
        for b in range(scale.shape[-2]):
            at = (..., slice(128 * a, 128 * a + 128), slice(128 * b, 128 * b + 128))
            s = _scale(np.abs(W[at]).max((-1, -2)))
            scale[..., b, a] = s
            q[at] = e4m3(W[at] / s[..., None, None])
    return q, scale


def values(q, scale):
    out = np.zeros(q.shape)
    for b, k in enumerate(runs(q)):
        out[..., k] = q[..., k] * scale[..., b, None].astype(np.float64)
    return out


def weight_values(q, scale):
    s = np.repeat(np.repeat(scale.astype(np.float64).swapaxes(-1, -2), 128, -2), 128, -1)
    return q * s[..., :q.shape[-2], :q.shape[-1]]
