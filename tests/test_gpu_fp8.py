"""8-bit features on the GPU: the quantisation of features and weights and
their channel mixing, code for code and against 64-bit forms
(tests/grouped_reference.py)."""
import numpy as np
import pytest

from clebsch_gordan_tensor_amd import synth as S
from tests import grouped_reference as R
from tests import norm_reference as N
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    from clebsch_gordan_tensor_amd import api
    api.lib()
    return api


def _ir(s):
    return S.parse_irreps(s)[1]


def _q(t):
    return host(t.float()).astype(np.float64)


def _same(got, ref, what):
    assert got.shape == ref.shape, what
    assert np.array_equal(got, ref, equal_nan=True), \
        f"{what}: {int((~((got == ref) | (np.isnan(got) & np.isnan(ref)))).sum())} differ"


# ------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", [(1, 16), (3, 48), (700, 128), (257, 144), (5, 1024),
                                    (33, 8192), (20011, 64), (0, 128)])
def test_quantize(gpu, rows, C, dtype):
    rng = np.random.default_rng(rows + C)
    x = (rng.standard_normal((rows, 3, C)) * 10.0 ** rng.uniform(-6, 6, (rows, 3, 1)) *
         np.exp(3 * rng.standard_normal((rows, 3, C)))).astype(np.float32)
    if dtype == "bf16":
        x = S.round_bf16(x)
    q, scale = gpu.quantize_fp8(dev(x, dtype))
    assert q.dtype == torch.float8_e4m3fn
    rq, rs = R.quantize(x)
    _same(host(scale), rs, "scale")
    _same(_q(q), rq, "codes")


def test_quantize_borders(gpu):
    # every border between two codes (a tie goes to the even one), and its neighbours
    top = np.float32(448 * 0.37)
    codes = np.unique(R.e4m3(np.exp2(np.linspace(-12, 8.9, 20000)).astype(np.float32)))
    codes = np.concatenate([[0.0], codes[codes <= 448]])
    mid = ((codes[1:] + codes[:-1]) / 2).astype(np.float32)
    s = np.float32(top * (np.float32(1) / np.float32(448)))
    v = np.concatenate([mid * s, np.nextafter(mid * s, np.float32(0)),
                        np.nextafter(mid * s, np.float32(1e9))]).astype(np.float32)
    v = np.concatenate([v, -v])
    v = v[np.abs(v) <= top]
    rows = -(-v.size // 127)
    x = np.zeros((rows, 128), np.float32)
    x[:, 0] = top
    x[:, 1:].reshape(-1)[:] = 0
    flat = np.zeros(rows * 127, np.float32)
    flat[:v.size] = v
    x[:, 1:] = flat.reshape(rows, 127)
    q, scale = gpu.quantize_fp8(dev(x))
    rq, rs = R.quantize(x)
    _same(host(scale), rs, "scale")
    _same(_q(q), rq, "codes")


def test_quantize_extremes(gpu):
    # zeros, the smallest and largest floats, and runs that are not finite
    x = np.zeros((9, 256), np.float32)
    x[1, 5] = 1e-45
    x[2, 5:9] = (1e-39, -1e-40, 3e-38, 1e-45)
    x[3] = 3.4e38
    x[4, 130] = np.inf
    x[5, 3] = np.nan
    x[6, 7], x[6, 8] = -np.inf, np.inf
    x[7, 0], x[7, 1] = 3.4e38, 1e-3
    x[8] = np.linspace(-1, 1, 256)
    q, scale = gpu.quantize_fp8(dev(x))
    rq, rs = R.quantize(x)
    _same(host(scale), rs, "scale")
    _same(_q(q), rq, "codes")
    assert np.isnan(rs[4, 1]) and np.isfinite(rs[4, 0])


# ------------------------------------------------ normalisation with residual

def _norm_case(irreps, rows, C, dtype, seed=0):
    rng = np.random.default_rng(rows * 3 + C + seed)
    shape = (rows, S.dim(irreps), C)
    scalars = sum(b == (0, 1) for b in irreps)
    x = rng.standard_normal(shape) * rng.uniform(0.1, 3.0, (rows, 1, 1)) + 0.5
    x, r, dy, dh = (t.astype(np.float32) for t in (x, *rng.standard_normal((3, *shape))))
    if dtype == "bf16":
        x, r, dy, dh = map(S.round_bf16, (x, r, dy, dh))
    w = (1 + 0.3 * rng.standard_normal((len(irreps), C))).astype(np.float32)
    b = rng.standard_normal((scalars, C)).astype(np.float32)
    h = x + r
    return x, r, dy, dh, w, b, S.round_bf16(h) if dtype == "bf16" else h


def _within(got, ref, tol, what, bf16=False):
    got = host(got).astype(np.float64)
    assert got.shape == ref.shape, what
    tol = tol + (R.U_BF16 * np.maximum(np.abs(ref), np.abs(got)) if bf16 else 0.0)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside"


SHAPES = [("0e", 1), ("0e", 3), ("0e", 128), ("0e", 1001), ("0e", 4096), ("0e+1o+2e+3o", 128),
          ("0e+1o", 2), ("0e+1o", 8), ("0o+0e+0e+1o", 37), ("0e+1o+2e+3o", 24), ("1o+2e", 100),
          ("0e+1o+2e", 300), ("8e+0e", 64), ("0e+4e+1o", 20), ("1o", 600), ("0e+1o+2e", 3)]


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("irreps,C", SHAPES)
@pytest.mark.parametrize("rows", [1, 67, 1500])
def test_residual(gpu, irreps, C, rows, dtype, flags):
    if rows == 1500 and C * S.dim(_ir(irreps)) > 3000:
        rows = 300
    ir, bf16 = _ir(irreps), dtype == "bf16"
    x, r, dy, dh, w, b, h = _norm_case(ir, rows, C, dtype)
    X, Rd, D, H, W, B = dev(x, dtype), dev(r, dtype), dev(dy, dtype), dev(dh, dtype), dev(w), dev(b)
    y, gh = gpu.layer_norm_residual(ir, X, Rd, W, B, eps=EPS, flags=flags)
    assert np.array_equal(host(gh), h)
    # bitwise the normalisation of the same h
    assert torch.equal(y, gpu.layer_norm(ir, gh, W, B, eps=EPS, flags=flags))
    ref, tol = N.norm_forward(ir, h, w, b, EPS, not flags)
    _within(y, ref, tol, "y", bf16)
    dx, dw, db = gpu.layer_norm_residual_backward(ir, gh, W, D, H, eps=EPS, flags=flags)
    _, pw, pb = gpu.layer_norm_backward(ir, gh, W, D, eps=EPS, flags=flags)
    assert torch.equal(dw, pw) and torch.equal(db, pb)
    (rx, _, _), (tx, _, _) = N.norm_backward(ir, h, w, dy, EPS, not flags)
    _within(dx, rx + dh, tx + R.U * np.abs(rx + dh), "dx", bf16)


def test_residual_in_place(gpu):
    ir = _ir("0e+1o+2e")
    for C in (2, 24, 64):
        x, r, dy, dh, w, b, _ = _norm_case(ir, 900, C, "f32")
        W, B = dev(w), dev(b)
        y, h = gpu.layer_norm_residual(ir, dev(x), dev(r), W, B)
        for hx, yx in ((0, 1), (1, 0), (0, None), (None, 1), (None, 0)):
            t = [dev(x), dev(r)]
            gy, gh = gpu.layer_norm_residual(ir, t[0], t[1], W, B,
                                             h=None if hx is None else t[hx],
                                             out=None if yx is None else t[yx])
            assert torch.equal(gy, y) and torch.equal(gh, h), (C, hx, yx)
        ref = gpu.layer_norm_residual_backward(ir, h, W, dev(dy), dev(dh))[0]
        for k in range(3):
            t = [h.clone(), dev(dy), dev(dh)]
            got = gpu.layer_norm_residual_backward(ir, t[0], W, t[1], t[2], dx=t[k])[0]
            assert torch.equal(got, ref), (C, k)


# widths whose last vector is moved back over the channels of another wavefront's (257 to 259 of
# every 256 in lists with a degree above 0; of scalars 1025 and up), and their neighbours
@pytest.mark.parametrize("irreps,C,dtype", [
    ("0e+1o", 257, "f32"), ("0e+1o+2e", 258, "bf16"), ("1o", 259, "f32"), ("0e+1o", 260, "f32"),
    ("4e+0e", 257, "f32"), ("0e+1o", 514, "f32"), ("0e+5o", 513, "bf16"), ("1o+0e", 771, "f32"),
    ("0e+1o", 1025, "f32"), ("1o", 2049, "bf16"), ("0e", 1025, "f32"), ("0e", 1027, "f32"),
    ("0e", 1281, "f32"), ("0e", 2049, "f32"), ("0e", 1025, "bf16"), ("0e", 1031, "bf16"),
    ("0o", 1537, "bf16"), ("0e", 1300, "f32")])
def test_residual_in_place_wide(gpu, irreps, C, dtype):
    ir, rows = _ir(irreps), 2003
    x, r, dy, dh, w, b, _ = _norm_case(ir, rows, C, dtype)
    X, Rd, D, H = (dev(t, dtype) for t in (x, r, dy, dh))
    W, B = dev(w), dev(b)
    y, h = gpu.layer_norm_residual(ir, X, Rd, W, B)
    assert torch.equal(h, (X.float() + Rd.float()).to(X.dtype))
    assert torch.equal(y, gpu.layer_norm(ir, h, W, B))
    ref = gpu.layer_norm_residual_backward(ir, h, W, D, H)
    for _ in range(3):
        for hx, yx in ((0, 1), (1, 0), (0, None), (1, None), (None, 1), (None, 0)):
            t = [X.clone(), Rd.clone()]
            gy, gh = gpu.layer_norm_residual(ir, t[0], t[1], W, B,
                                             h=None if hx is None else t[hx],
                                             out=None if yx is None else t[yx])
            assert torch.equal(gh, h) and torch.equal(gy, y), (hx, yx)
        for k in range(3):
            t = [h.clone(), D.clone(), H.clone()]
            got = gpu.layer_norm_residual_backward(ir, t[0], W, t[1], t[2], dx=t[k])
            for a, c in zip(got, ref):
                assert torch.equal(a, c), k


def test_residual_without_weights_and_rows(gpu):
    ir = _ir("0e+1o")
    x, r, dy, dh, w, b, h = _norm_case(ir, 40, 64, "f32")
    y, gh = gpu.layer_norm_residual(ir, dev(x), dev(r))
    assert torch.equal(y, gpu.layer_norm(ir, gh))
    e = torch.empty((0, 4, 64), device="cuda")
    y, gh = gpu.layer_norm_residual(ir, e, e.clone(), dev(w), dev(b))
    dx, dw, db = gpu.layer_norm_residual_backward(ir, e, dev(w), e, e)
    assert y.shape == gh.shape == dx.shape == (0, 4, 64) and not dw.any() and not db.any()
    q, s, gh = gpu.layer_norm_fp8(ir, e, e.clone(), dev(w), dev(b))
    assert q.shape == (0, 4, 64) and s.shape == (0, 4, 1)


def test_residual_gradient_against_differences(gpu):
    ir = _ir("0e+1o")
    x, r, dy, dh, w, b, _ = _norm_case(ir, 30, 32, "f32")
    X, W, B, D, H = dev(x), dev(w), dev(b), dev(dy), dev(dh)
    rng = np.random.default_rng(3)
    d = rng.standard_normal(x.shape)

    def loss(t):  # in 64 bits from the plain form
        h = x.astype(np.float64) + r + t * d
        y, _ = N.norm_forward(ir, h, w, b, EPS)
        return (y * dy).sum() + (h * dh).sum()
    _, h = gpu.layer_norm_residual(ir, X, dev(r), W, B, eps=EPS)
    dx = gpu.layer_norm_residual_backward(ir, h, W, D, H, eps=EPS)[0]
    t = 1e-4
    num = (loss(t) - loss(-t)) / (2 * t)
    ana = (host(dx).astype(np.float64) * d).sum()
    # differences: third derivatives x t^2, 1e-8 of the terms' sizes; float32: 1e-6 of them
    assert abs(num - ana) <= 2e-6 * np.abs(host(dx) * d).sum()


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("irreps,C", [
    ("0e", 16), ("0e", 128), ("0e", 144), ("0e", 1008), ("0e", 2048), ("0e", 4096),
    ("0e+1o+2e+3o", 128), ("0e+1o", 16), ("0e+1o+2e+3o", 48), ("1o+2e", 112), ("0e+1o+2e", 304),
    ("8e+0e", 64), ("0e+4e+1o", 32), ("1o", 608), ("8e+0e", 1024), ("0e+3o", 4096)])
@pytest.mark.parametrize("rows", [1, 67])
def test_norm_in_8_bits(gpu, irreps, C, rows, dtype, flags):
    ir = _ir(irreps)
    x, r, _, _, w, b, h = _norm_case(ir, rows, C, dtype)
    X, Rd, W, B = dev(x, dtype), dev(r, dtype), dev(w), dev(b)
    q, scale, gh = gpu.layer_norm_fp8(ir, X, Rd, W, B, eps=EPS, flags=flags)
    assert np.array_equal(host(gh), h)
    q1, scale1 = gpu.layer_norm_fp8(ir, gh, None, W, B, eps=EPS, flags=flags)
    assert torch.equal(q1.view(torch.uint8), q.view(torch.uint8)) and torch.equal(scale1, scale)
    if dtype == "f32":  # code for code the quantised result of the normalisation
        rq, rs = R.quantize(host(gpu.layer_norm(ir, gh, W, B, eps=EPS, flags=flags)))
        _same(host(scale), rs, "scale")
        _same(_q(q), rq, "codes")
    y, tol = N.norm_forward(ir, h, w, b, EPS, not flags)
    s = host(scale)
    for k, run in enumerate(R.runs(y)):
        # the largest value's error, a division; the codes: half a step of 8 bits
        top, off = np.abs(y[..., run]).max(-1), tol[..., run].max(-1)
        assert np.all(np.abs(s[..., k] - top / 448) <= (off + 2 * R.U * top) / 448)
        step = np.maximum(2.0 ** -4 * np.abs(y[..., run]), s[..., k, None] * 2.0 ** -10)
        err = np.abs(_q(q)[..., run] * s[..., k, None] - y[..., run])
        assert np.all(err <= step * (1 + 1e-5) + tol[..., run] * 1.1)


def test_norm_in_8_bits_not_finite(gpu):
    ir = _ir("0e+1o")
    x, r, _, _, w, b, _ = _norm_case(ir, 20, 256, "f32")
    ref = gpu.layer_norm_fp8(ir, dev(x), dev(r), dev(w), dev(b))
    x[3, 0, 200], x[4, 2, 7] = np.nan, np.inf
    q, scale, h = gpu.layer_norm_fp8(ir, dev(x), dev(r), dev(w), dev(b))
    bad = torch.zeros((20, 4), dtype=torch.bool, device="cuda")
    bad[3, 0], bad[4, 1:] = True, True  # the whole block of the row
    assert torch.isnan(scale[bad]).all()
    assert torch.equal(scale[~bad], ref[1][~bad])
    assert torch.equal(q.view(torch.uint8)[~bad], ref[0].view(torch.uint8)[~bad])


# ------------------------------------------------------------------- mixing

def _mix_case(into, out, rows, groups, cin, cout, stray=0.1):
    rng = np.random.default_rng(rows * 31 + groups * 7 + cin + cout)
    group = (rng.random(rows) ** 2 * groups).astype(np.int32)
    group[rng.random(rows) < stray] = -1
    x = (rng.standard_normal((rows, S.dim(into), cin)) * rng.uniform(0.1, 3, (rows, 1, 1)))
    W = rng.standard_normal((groups, len(R.pairs(into, out)), cin, cout)) / np.sqrt(cin)
    return group, x.astype(np.float32), W.astype(np.float32)


MIXES = [
    ("0e+1o+2e+3o", "0e+1o+2e+3o", 301, 1, 128, 128), ("0e+1o+2e+3o", "0e+1o+2e+3o", 1, 10, 128, 128),
    ("0e+1o", "0e+1o", 64, 3, 16, 16), ("0e+1o", "0e+1o+2e+3o", 77, 4, 64, 96),
    ("0e+0e+1o+2e", "1o+0e", 130, 7, 48, 32), ("1o+0e", "0e+1o+1o", 90, 6, 32, 208),
    ("0e", "0e", 333, 16, 528, 272), ("0e", "0e", 3, 2, 2048, 144), ("0e", "0e", 700, 1, 144, 1008),
    ("0e", "0e", 1, 1, 1024, 512), ("8e+0e", "8e", 40, 100, 16, 16), ("1o", "1o", 2100, 2, 256, 256),
    ("0e+1o+2e", "0e+1o+2e", 1200, 300, 32, 48)]


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("xs,os_,rows,groups,cin,cout", MIXES)
def test_mixing(gpu, xs, os_, rows, groups, cin, cout, out_dtype):
    into, out = _ir(xs), _ir(os_)
    group, x, W = _mix_case(into, out, rows, groups, cin, cout, stray=0.1 if groups > 1 else 0.0)
    index = gpu.group_rows(dev(group), groups) if groups > 1 else None
    q, scale = gpu.quantize_fp8(dev(x))
    packed = gpu.linear_fp8_pack(into, out, dev(W))
    rq, rs = R.quantize_weights(W)
    # the packed form: a header, scales [..][out blocks][in blocks], codes [..][cout][cin to 128]
    buf, mats = packed.buffer.cpu(), W.shape[0] * W.shape[1]
    blocks_in, n_scales = -(-cin // 128), rs.size
    codes_at = 64 + -(-4 * n_scales // 64) * 64
    _same(buf[64:64 + 4 * n_scales].view(torch.float32).numpy().reshape(rs.shape), rs, "scales of W")
    codes = buf[codes_at:codes_at + mats * cout * blocks_in * 128].view(torch.float8_e4m3fn)
    codes = codes.float().numpy().reshape(*W.shape[:2], cout, blocks_in * 128)
    _same(codes[..., :cin].swapaxes(-1, -2), rq.astype(np.float32), "codes of W")
    assert not codes[..., cin:].any()
    y = gpu.linear_fp8(into, out, q, scale, packed, index=index,
                       dtype=torch.float32 if out_dtype == "f32" else None)
    ref = R.mix(into, out, group, R.values(_q(q), host(scale)), R.weight_values(rq, rs))
    # a rounding for each of the products' adds at most, and two for the scales
    bf16 = out_dtype == "bf16"
    R.check(host(y), ref, "y", bf16, adds=1, drops=R.EIGHTS if bf16 else 0.0)
    if groups > 1:
        assert not host(y)[group < 0].any()


@pytest.mark.parametrize("xs,os_,rows,groups,cin,cout", MIXES[:8])
def test_mixing_of_whole_numbers_is_exact(gpu, xs, os_, rows, groups, cin, cout):
    # codes of small whole numbers and scales of powers of two: every sum is exact
    into, out = _ir(xs), _ir(os_)
    group, x, W = _mix_case(into, out, rows, groups, cin, cout, stray=0.0)
    rng = np.random.default_rng(1)
    q = rng.integers(-8, 9, x.shape).astype(np.float32)
    scale = np.exp2(rng.integers(-2, 3, (*x.shape[:-1], -(-cin // 128)))).astype(np.float32)
    Wv = rng.integers(-8, 9, W.shape).astype(np.float32)
    Wv[..., ::128, ::128] = 14.0  # every block's scale is 2^-5
    index = gpu.group_rows(dev(group), groups) if groups > 1 else None
    y = gpu.linear_fp8(into, out, dev(q).to(torch.float8_e4m3fn), dev(scale),
                       gpu.linear_fp8_pack(into, out, dev(Wv)), index=index, dtype=torch.float32)
    ref, _, _ = R.mix(into, out, group, R.values(q, scale), Wv)
    assert np.array_equal(host(y), ref)


# results a hundredth of their terms and less: float32 keeps them, bf16 is off by what the 8-bit
# matrix cores drop of the terms
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cin,cout", [(3, 256, 64), (900, 128, 128), (3000, 512, 272)])
def test_small_differences_of_large_terms(gpu, rows, cin, cout, out_dtype):
    into = out = _ir("0e")
    _, x, W = _mix_case(into, out, rows, 1, cin, cout, stray=0.0)
    x[..., 1::2] = -x[..., ::2]  # pairs of terms that cancel but for a few
    x[..., 1::16] *= np.float32(0.9)
    W[..., 1::2, :] = W[..., ::2, :]
    q, scale = gpu.quantize_fp8(dev(x))
    y = gpu.linear_fp8(into, out, q, scale, gpu.linear_fp8_pack(into, out, dev(W)),
                       dtype=torch.float32 if out_dtype == "f32" else None)
    ref, size, terms = R.mix(into, out, np.zeros(rows, int), R.values(_q(q), host(scale)),
                             R.weight_values(*R.quantize_weights(W)))
    assert np.sqrt((ref ** 2).mean()) < 0.02 * size.mean()
    got = host(y).astype(np.float64)
    tol = (terms + 16) * R.U * size + R.U * np.abs(ref)
    if out_dtype == "bf16":
        tol += R.EIGHTS * size + R.U_BF16 * np.maximum(np.abs(ref), np.abs(got))
    assert np.all(np.abs(got - ref) <= tol)


def test_mixing_keeps_rows_apart(gpu):
    # a row that is not finite, and a row's result alone and among others
    into = out = _ir("0e+1o")
    group, x, W = _mix_case(into, out, 300, 3, 144, 80, stray=0.0)
    packed, Gd = gpu.linear_fp8_pack(into, out, dev(W)), dev(group)
    ref = gpu.linear_fp8(into, out, *gpu.quantize_fp8(dev(x)), packed, index=gpu.group_rows(Gd, 3))
    x[7, 2, 140] = np.inf
    y = gpu.linear_fp8(into, out, *gpu.quantize_fp8(dev(x)), packed, index=gpu.group_rows(Gd, 3))
    keep = torch.ones((300, 4), dtype=torch.bool, device="cuda")
    keep[7, 2] = False
    assert torch.isnan(y[7, 2]).all() and torch.equal(y[keep], ref[keep])
    for n in (1, 7, 130):
        some = gpu.linear_fp8(into, out, *gpu.quantize_fp8(dev(x[:n])), packed,
                              index=gpu.group_rows(Gd[:n].contiguous(), 3))
        assert torch.equal(some[:7], ref[:7][:n])


def test_weights_packed_for_other_sizes_change_nothing(gpu):
    into = out = _ir("0e+1o")
    _, x, W = _mix_case(into, out, 30, 1, 64, 64)
    packed = gpu.linear_fp8_pack(into, out, dev(W))
    big = torch.zeros(gpu._pack_size(tuple(into), tuple(out), 128, 128, 1), device="cuda",
                      dtype=torch.uint8)
    big[:packed.buffer.numel()] = packed.buffer
    q, scale = gpu.quantize_fp8(torch.randn((30, 4, 128), device="cuda"))
    keep = torch.full((30, 4, 128), 3.0, device="cuda")
    y = gpu.linear_fp8(into, out, q, scale, gpu.Fp8Weights(big, 1, 2, 128, 128), out=keep.clone())
    assert torch.equal(y, keep)


@pytest.mark.parametrize("rows", [1, 1700])
def test_layer_captured_and_on_another_stream(gpu, rows):
    # as a simulation runs them: normalise x + update in 8 bits, mix by element
    ir = _ir("0e+1o+2e+3o")
    C, G = 128, 4
    x, r, _, _, w, b, _ = _norm_case(ir, rows, C, "bf16")
    group, _, W = _mix_case(ir, ir, rows, G, C, C)
    X, Rd, Wn, B, Gd = dev(x, "bf16"), dev(r, "bf16"), dev(w), dev(b), dev(group)
    packed = gpu.linear_fp8_pack(ir, ir, dev(W))

    def layer(stream=None, **mem):
        index = gpu.group_rows(Gd, G, index=mem.get("index"), stream=stream)
        q, s, h = gpu.layer_norm_fp8(ir, X, Rd, Wn, B, h=mem.get("h"), q=mem.get("q"),
                                     scale=mem.get("scale"), stream=stream)
        y = gpu.linear_fp8(ir, ir, q, s, packed, index=index, out=mem.get("y"), stream=stream)
        return dict(index=index, h=h, q=q, scale=s, y=y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mem = layer(stream=side)
    side.synchronize()
    ref = layer()
    for k in ("h", "scale", "y"):
        assert torch.equal(mem[k], ref[k]), k
    # what the 8-bit layer computes, against the plain forms of its steps
    hq, hs = _q(ref["q"]), host(ref["scale"])
    wq, ws = R.quantize_weights(W)
    R.check(host(ref["y"]), R.mix(ir, ir, group, R.values(hq, hs), R.weight_values(wq, ws)), "layer",
            True, adds=1, drops=R.EIGHTS)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(**mem)
    for seed in range(3):
        x, r, _, _, _, _, _ = _norm_case(ir, rows, C, "bf16", seed=seed + 1)
        X.copy_(torch.from_numpy(x))
        Rd.copy_(torch.from_numpy(r))
        Gd.copy_(Gd.roll(1))
        mem["y"].fill_(1.0)
        g.replay()
        torch.cuda.synchronize()
        ref = layer()
        for k in ("h", "scale", "y"):
            assert torch.equal(mem[k], ref[k]), k
