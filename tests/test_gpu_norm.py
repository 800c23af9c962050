"""The normalisation of irreps features and its gradients on the GPU against
their 64-bit forms.  Every element is held to the error its own float32
arithmetic may make (tests/norm_reference.py), plus half a step of the storage
type."""
import numpy as np
import pytest

from clebsch_gordan_tensor_amd import synth as S
from tests import norm_reference as R
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


def _case(irreps, rows, C, seed, dtype="f32", shift=0.5):
    rng = np.random.default_rng(seed)
    shape = (rows, S.dim(irreps), C)
    scalars = sum(b == (0, 1) for b in irreps)
    x = (rng.standard_normal(shape) * rng.uniform(0.1, 3.0, (rows, 1, 1)) + shift)
    dy = rng.standard_normal(shape)
    x, dy = x.astype(np.float32), dy.astype(np.float32)
    if dtype == "bf16":
        x, dy = S.round_bf16(x), S.round_bf16(dy)
    w = (1 + 0.3 * rng.standard_normal((len(irreps), C))).astype(np.float32)
    b = rng.standard_normal((scalars, C)).astype(np.float32)
    return x, dy, w, b


def _within(got, ref, tol, what, dtype="f32"):
    got = host(got).astype(np.float64)
    assert got.shape == ref.shape, what
    if dtype == "bf16":
        tol = tol + R.U_BF16 * np.maximum(np.abs(ref), np.abs(got))
    bad = ~(np.abs(got - ref) <= tol)
    worst = float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-300))) if got.size else 0.0
    print(f"[err] {what}: {worst:.3f} of the bound", flush=True)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {worst:.2f}"


def _check(gpu, irreps, x, dy, w, b, dtype="f32", flags=0, forward=True):
    centered = not flags & gpu.E3_NORM_UNCENTERED
    X, D = dev(x, dtype), dev(dy, dtype)
    W, B = dev(w), dev(b)
    if forward:
        y = gpu.layer_norm(irreps, X, W, B, eps=EPS, flags=flags)
        _within(y, *R.norm_forward(irreps, x, w, b, EPS, centered), "y", dtype)
    got = gpu.layer_norm_backward(irreps, X, W, D, eps=EPS, flags=flags)
    ref, tol = R.norm_backward(irreps, x, w, dy, EPS, centered)
    for g, r, t, name in zip(got, ref, tol, ("dx", "dweight", "dbias")):
        _within(g, r, t, name, dtype if name == "dx" else "f32")


@pytest.mark.parametrize("rows", [1, 2, 300])
@pytest.mark.parametrize("C", [1, 2, 3, 4, 5, 7, 8, 31, 64, 100, 128, 255, 256, 257, 1000, 1025,
                               4095, 4096])
def test_layer_norm_of_scalars(gpu, C, rows):
    irreps = _ir("0e")
    _check(gpu, irreps, *_case(irreps, rows, C, C + rows))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("irreps,C", [
    ("0e+1o+2e+3o", 128), ("0e+1o", 8), ("0e+1o+1e+2e+2o+3o+3e", 64), ("0o+0e+0e+1o", 37),
    ("3o+0e", 3), ("2e", 1), ("0e+1o+2e+3o", 300), ("1o+0e", 2050),
    ("0e+1o+2e+3o", 24), ("0e+1o", 50), ("1o+2e", 100), ("0e+4e+1o", 20), ("0e+1o+2e+3o", 1500),
    ("0e+1o+2e+3o", 2), ("0e+3o", 4096), ("8e+0e", 1024), ("0e", 1100), ("0e", 2500), ("0e", 6), ("1o", 600),
    ("0e+1o+2e+3o+4e+5o+6e+7o+8e", 16), ("8e+0e", 5), ("7o+4e+1o", 512), ("5o+6e", 1024),
])
@pytest.mark.parametrize("rows", [1, 53])
def test_irreps(gpu, irreps, C, rows, dtype):
    irreps = _ir(irreps)
    _check(gpu, irreps, *_case(irreps, rows, C, 7 * C + rows, dtype), dtype=dtype)


@pytest.mark.parametrize("C", [6, 128, 700])
def test_uncentered(gpu, C):
    irreps = _ir("0e+1o+0e")
    _check(gpu, irreps, *_case(irreps, 77, C, C), flags=gpu.E3_NORM_UNCENTERED)


def test_many_rows(gpu):
    # every workgroup takes several rows, the last ones are ragged
    irreps = _ir("0e+1o+2e")
    _check(gpu, irreps, *_case(irreps, 5003, 48, 3))


@pytest.mark.parametrize("case", R.LONG_SUMS, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}")
def test_long_sums(gpu, case):
    # every kernel over more rows than its workgroups take in one turn, bounds that see a lost row
    ir, C, dtype, rows, lane, depth = case
    irreps = _ir(ir)
    x, dy = R.long_case(irreps, C, dtype, rows)
    w = (1 + 0.3 * np.random.default_rng(C).standard_normal((len(irreps), C))).astype(np.float32)
    dx, dweight, dbias = gpu.layer_norm_backward(irreps, dev(x, dtype), dev(w), dev(dy, dtype),
                                                 eps=EPS)
    dw, db = R.long_sums(irreps, x, dy, EPS, lane, depth)
    for got, sums, what in ((dweight, dw, "dweight"), (dbias, db, "dbias")):
        _within(got, *(np.stack([s[k] for s in sums]) for k in (1, 2)), what)
    (ref, _, _), (tol, _, _) = R.norm_backward(irreps, x, w, dy, EPS)
    _within(dx, ref, tol, "dx", dtype)


@pytest.mark.parametrize("C", [3, 4, 64])
def test_many_blocks(gpu, C):
    # more blocks than one launch takes, low and high degrees mixed
    irreps = _ir("0e+1o+4e") * 45
    _check(gpu, irreps, *_case(irreps, 9, C, 4))


@pytest.mark.parametrize("irreps,C,rows", [("0e", 64, 40), ("0e", 64, 4000), ("0e+1o", 9, 700),
                                           ("0e+1o", 2, 3000), ("0e+1o+2e", 64, 900)])
def test_gradients_not_wanted(gpu, irreps, C, rows):
    # dweight, dbias or both left out (NULL): the others are the same
    import ctypes
    irreps = _ir(irreps)
    x, dy, w, _ = (dev(a) for a in _case(irreps, rows, C, 16))
    ref = gpu.layer_norm_backward(irreps, x, w, dy)
    st = gpu._irreps_struct(irreps, C)
    ws = torch.empty(gpu.layer_norm_workspace_size(irreps, rows, C), device="cuda",
                     dtype=torch.uint8)
    for want_w, want_b in ((0, 1), (1, 0), (0, 0)):
        got = [torch.full_like(t, 3.0) for t in ref]
        at = [got[0].data_ptr(), got[1].data_ptr() if want_w else None,
              got[2].data_ptr() if want_b else None]
        assert gpu.lib().e3_layer_norm_backward(
            ctypes.byref(st), rows, x.data_ptr(), w.data_ptr(), dy.data_ptr(), EPS, 0, *at,
            ws.data_ptr(), ws.numel(), 0, torch.cuda.current_stream().cuda_stream) == 0
        for t, r, want in zip(got, ref, (1, want_w, want_b)):
            assert torch.equal(t, r) if want else torch.all(t == 3.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("irreps,C", [("0e", 128), ("0e", 13), ("0e", 700), ("0e+1o+2e+3o", 128),
                                      ("0e+1o", 9), ("0e+1o", 3), ("0e+1o", 300), ("4e+0e", 64),
                                      ("4e+0e", 9), ("6e+0e", 300)])
def test_a_row_by_itself(gpu, irreps, C, dtype):
    # a row's result is the same wherever it stands, alone or among others, bit for bit
    irreps = _ir(irreps)
    x, dy, w, b = _case(irreps, 1030, C, C, dtype)
    X, D, W, B = dev(x, dtype), dev(dy, dtype), dev(w), dev(b)
    y, dx = gpu.layer_norm(irreps, X, W, B), gpu.layer_norm_backward(irreps, X, W, D)[0]
    for rows in ([0], [1029], [3, 700, 1028]):
        at = torch.tensor(rows, device="cuda")
        part, dpart = X[at].contiguous(), D[at].contiguous()
        assert torch.equal(gpu.layer_norm(irreps, part, W, B), y[at])
        assert torch.equal(gpu.layer_norm_backward(irreps, part, W, dpart)[0], dx[at])


@pytest.mark.parametrize("irreps", ["0e", "0e+1o", "0e+0e"])
def test_a_single_channel(gpu, irreps):
    # a centred scalar of one channel is its own mean: y is the bias and dx zero, exactly
    irreps = _ir(irreps)
    x, dy, w, b = _case(irreps, 70, 1, 15)
    y = host(gpu.layer_norm(irreps, dev(x), dev(w), dev(b)))
    dx, dw, _ = (host(t) for t in gpu.layer_norm_backward(irreps, dev(x), dev(w), dev(dy)))
    for i, (at, _, bias) in enumerate(R.blocks_of(irreps)):
        if bias >= 0:
            assert np.all(y[:, at] == b[bias]) and np.all(dx[:, at] == 0) and np.all(dw[i] == 0)


def test_mean_far_from_zero(gpu):
    irreps = _ir("0e+1o")
    _check(gpu, irreps, *_case(irreps, 40, 128, 5, shift=30.0))


def test_without_weight_and_bias(gpu):
    irreps = _ir("0e+1o")
    x, dy, w, b = _case(irreps, 20, 32, 6)
    one, zero = np.ones_like(w), np.zeros_like(b)
    X, D, W, B = dev(x), dev(dy), dev(one), dev(zero)
    assert torch.equal(gpu.layer_norm(irreps, X), gpu.layer_norm(irreps, X, W, B))
    for a, c in zip(gpu.layer_norm_backward(irreps, X, None, D),
                    gpu.layer_norm_backward(irreps, X, W, D)):
        assert torch.equal(a, c)


def test_gradient_against_differences(gpu):
    # <dx, d> and the weight gradients against central differences of the 64-bit forward: step
    # 1e-4 of the values, error of order 1e-8 of the sums, float32 gradients 1e-6 of them
    irreps = _ir("0e+1o+2e")
    x, dy, w, b = _case(irreps, 11, 24, 8)
    dx, dw, db = (host(t).astype(np.float64) for t in gpu.layer_norm_backward(
        irreps, dev(x), dev(w), dev(dy), eps=EPS))
    f = lambda x, w, b: float((R.norm_forward(irreps, x, w, b, EPS)[0] * dy).sum())  # noqa: E731
    rng = np.random.default_rng(9)
    x, w, b = (a.astype(np.float64) for a in (x, w, b))
    h = 1e-4
    for grad, at in ((dx, 0), (dw, 1), (db, 2)):
        d = rng.standard_normal(grad.shape)
        args = [x, w, b]
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + h * d, args[at] - h * d
        num, ref = (f(*up) - f(*down)) / (2 * h), float((grad * d).sum())
        assert abs(num - ref) <= 1e-5 * np.abs(grad * d).sum(), at


@pytest.mark.parametrize("irreps,C", [(ir, C) for ir in ("0e+1o", "4e+0e") for C in (2, 5, 50, 128, 300, 1000)] +
                         [("0e+1o", 2050)])
def test_in_place(gpu, C, irreps):
    irreps = _ir(irreps)
    x, dy, w, b = _case(irreps, 33, C, 10 + C)
    X, D, W, B = dev(x), dev(dy), dev(w), dev(b)
    y = gpu.layer_norm(irreps, X, W, B)
    ref = gpu.layer_norm_backward(irreps, X, W, D)
    x2, d2 = X.clone(), D.clone()
    for over in (x2, d2):
        args = (x2 if over is x2 else X, W, d2 if over is d2 else D)
        got = gpu.layer_norm_backward(irreps, *args, dx=over)
        for a, c in zip(got, ref):
            assert torch.equal(a, c)
    x2 = X.clone()
    gpu.layer_norm(irreps, x2, W, B, out=x2)
    assert torch.equal(x2, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [4, 7, 130, 1003])
def test_any_element_alignment(gpu, C, dtype):
    # operands one element past an aligned address; what lies around the outputs stays
    irreps = _ir("0e+1o")
    x, dy, w, b = _case(irreps, 19, C, 11 + C, dtype)
    want = gpu.layer_norm(irreps, dev(x, dtype), dev(w), dev(b))
    ref = gpu.layer_norm_backward(irreps, dev(x, dtype), dev(w), dev(dy, dtype))

    def shifted(a, dt=dtype):
        t = dev(a, dt)
        room = torch.full((t.numel() + 2,), 7.0, device="cuda", dtype=t.dtype)
        room[1:-1] = t.view(-1)
        return room, room[1:-1].view(t.shape)

    (_, X), (_, D), (_, W), (_, B) = shifted(x), shifted(dy), shifted(w, "f32"), shifted(b, "f32")
    outs = [shifted(np.zeros_like(x)), shifted(np.zeros_like(x)), shifted(np.zeros_like(w), "f32"),
            shifted(np.zeros_like(b), "f32")]
    gpu.layer_norm(irreps, X, W, B, out=outs[0][1])
    gpu.layer_norm_backward(irreps, X, W, D, dx=outs[1][1], dweight=outs[2][1], dbias=outs[3][1])
    for (room, t), r in zip(outs, (want, *ref)):
        assert torch.equal(t, r)
        assert room[0] == 7.0 and room[-1] == 7.0


def test_rows_apart(gpu):
    # a constant row, a zero row, an infinity and a NaN: only their own rows and blocks change
    irreps = _ir("0e+1o")
    x, dy, w, b = _case(irreps, 12, 64, 12)
    x[2], x[3] = 0.0, 3.0
    y, tol = R.norm_forward(irreps, x, w, b, EPS)
    X = dev(x)
    _within(gpu.layer_norm(irreps, X, dev(w), dev(b)), y, tol, "constant rows")
    bad = x.copy()
    bad[5, 0, 3], bad[7, 2, 1] = np.inf, np.nan
    got = host(gpu.layer_norm(irreps, dev(bad), dev(w), dev(b)))
    dx = host(gpu.layer_norm_backward(irreps, dev(bad), dev(w), dev(dy))[0])
    good = host(gpu.layer_norm_backward(irreps, X, dev(w), dev(dy))[0])
    clean = host(gpu.layer_norm(irreps, X, dev(w), dev(b)))
    hit = np.zeros(x.shape, bool)
    hit[5, :1], hit[7, 1:] = True, True
    assert np.array_equal(got[~hit], clean[~hit]) and np.array_equal(dx[~hit], good[~hit])
    assert np.isnan(got[7, 1:]).all() and np.isnan(dx[5, :1]).all() and np.isnan(dx[7, 1:]).all()
    assert not np.isfinite(got[5, 0, 3])


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("irreps,C", [("0e", 64), ("0e", 1001), ("0e", 2050), ("0e+1o", 3),
                                      ("0e+1o", 9), ("0e+0o", 128), ("0e+1o", 300),
                                      ("0e+1o", 600), ("4e+0e", 64), ("4e+0e", 9)])
def test_a_block_that_is_not_finite(gpu, irreps, C, dtype, flags):
    # an infinity, a NaN or values whose squares leave float32's range, in the last row: NaN all
    # over their block of that row and in its weight's gradient, nothing else changes
    irreps, rows = _ir(irreps), 37
    x, dy, w, b = _case(irreps, rows, C, C + 1, dtype)
    D, W, B = dev(dy, dtype), dev(w), dev(b)

    def both(X):
        return (gpu.layer_norm(irreps, X, W, B, flags=flags),
                *gpu.layer_norm_backward(irreps, X, W, D, flags=flags))

    y, dx, dw, db = both(dev(x, dtype))
    assert all(torch.isfinite(t).all() for t in (y, dx, dw, db))
    for i, (at, nc, _) in enumerate(R.blocks_of(irreps)):
        for value in (np.inf, -np.inf, np.nan, 1e30, -3e38):
            X = dev(x, dtype)
            X[-1, at + nc - 1, C // 2] = value
            got = both(X)
            hit = torch.zeros(x.shape, dtype=torch.bool, device="cuda")
            hit[-1, at:at + nc] = True
            for t, r in zip(got[:2], (y, dx)):
                assert torch.equal(t[~hit], r[~hit]), (i, value)
                assert torch.isnan(t[hit]).all(), (i, value)
            others = [k for k in range(len(irreps)) if k != i]
            assert torch.isnan(got[2][i]).all() and torch.equal(got[2][others], dw[others])
            assert torch.equal(got[3], db)


def test_refused(gpu):
    irreps = _ir("0e+1o")
    x, dy, w, b = (dev(a) for a in _case(irreps, 6, 16, 14))
    for call in (lambda: gpu.layer_norm(_ir("0e+2e"), x), lambda: gpu.layer_norm(irreps, x[0]),
                 lambda: gpu.layer_norm(irreps, x.transpose(0, 2)),
                 lambda: gpu.layer_norm(irreps, x, w[:1]), lambda: gpu.layer_norm(irreps, x, w, w),
                 lambda: gpu.layer_norm(irreps, x, out=x[:5]),
                 lambda: gpu.layer_norm(irreps, x, w.cpu()),
                 lambda: gpu.layer_norm_backward(irreps, x, w, dy[:5]),
                 lambda: gpu.layer_norm_backward(irreps, x, w, None),
                 lambda: gpu.layer_norm_backward(irreps, x, w, dy, dbias=w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gpu.layer_norm(irreps, x.double()), lambda: gpu.layer_norm(irreps, x.half()),
                 lambda: gpu.layer_norm(irreps, x, w.bfloat16()),
                 lambda: gpu.layer_norm_backward(irreps, x, w, dy.bfloat16())):
        with pytest.raises(TypeError):
            call()
    room = torch.zeros(x.numel() + 64, device="cuda")
    room[:x.numel()] = x.view(-1)
    inside, shifted = room[:x.numel()].view(x.shape), room[64:].view(x.shape)
    with pytest.raises(gpu.E3Error, match="overlaps"):
        gpu.layer_norm(irreps, inside, out=shifted)
    with pytest.raises(gpu.E3Error, match="overlaps"):
        gpu.layer_norm_backward(irreps, x, None, inside, dx=shifted)
    with pytest.raises(gpu.E3Error, match="workspace"):
        gpu.layer_norm_backward(irreps, x, w, dy, workspace=torch.empty(16, device="cuda"))
    with pytest.raises(gpu.E3Error, match="eps"):
        gpu.layer_norm(irreps, x, eps=0.0)


def test_empty(gpu):
    irreps = _ir("0e+1o")
    e = torch.empty((0, 4, 16), device="cuda")
    w, b = torch.ones((2, 16), device="cuda"), torch.ones((1, 16), device="cuda")
    assert gpu.layer_norm(irreps, e, w, b).shape == (0, 4, 16)
    dw, db = torch.full_like(w, 5.0), torch.full_like(b, 5.0)
    gpu.layer_norm_backward(irreps, e, w, e, dweight=dw, dbias=db)
    assert torch.all(dw == 0) and torch.all(db == 0)


def test_reproducible_and_streams(gpu):
    irreps = _ir("0e+1o+2e+3o")
    x, dy, w, b = (dev(a) for a in _case(irreps, 3000, 128, 13))
    ref = gpu.layer_norm_backward(irreps, x, w, dy)
    for a, c in zip(gpu.layer_norm_backward(irreps, x, w, dy), ref):
        assert torch.equal(a, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = gpu.layer_norm_backward(irreps, x, w, dy)
    other = gpu.layer_norm_backward(irreps, x, w, dy, stream=side)
    side.synchronize()
    for a, b_, c in zip(got, other, ref):
        assert torch.equal(a, c) and torch.equal(b_, c)


def test_memory_of_another_stream(gpu):
    # what a call on another stream allocates must not be memory that work queued on the current
    # stream still writes
    irreps = _ir("0e+1o")
    x, dy, w, b = (dev(a) for a in _case(irreps, 2000, 64, 17))
    ref = (gpu.layer_norm(irreps, x, w, b), *gpu.layer_norm_backward(irreps, x, w, dy))
    norm = gpu.grad_norm(gpu.Params(grads=[x]))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = gpu.layer_norm_workspace_size(irreps, 2000, 64)
    old = [torch.empty_like(t) for t in (*ref, norm)]
    old += [torch.empty(n, device="cuda", dtype=torch.uint8) for n in (ws, 8 * 512)]
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for t in old:
        t.fill_(7)
    del old, t
    got = (gpu.layer_norm(irreps, x, w, b, stream=side),
           *gpu.layer_norm_backward(irreps, x, w, dy, stream=side))
    got_norm = gpu.grad_norm(gpu.Params(grads=[x]), stream=side)
    torch.cuda.synchronize()
    for a, c in zip((*got, got_norm), (*ref, norm)):
        assert torch.equal(a, c)


def test_beyond_32_bit_offsets(gpu):
    # 2^31 + 2^20 elements: the first, middle and last rows
    irreps, C = _ir("0e+1o"), 128
    rows = (2 ** 31 + 2 ** 20) // (4 * C)
    x = torch.empty((rows, 4, C), device="cuda", dtype=torch.bfloat16)
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    w = torch.ones((2, C), device="cuda")
    b = torch.zeros((1, C), device="cuda")
    y = gpu.layer_norm(irreps, x, w, b)
    dx, dw, db = gpu.layer_norm_backward(irreps, x, w, x)
    at = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1], device="cuda")
    assert torch.equal(gpu.layer_norm(irreps, x[at].contiguous(), w, b), y[at])
    part = gpu.layer_norm_backward(irreps, x[at].contiguous(), w, x[at].contiguous())
    assert torch.equal(part[0], dx[at])
    # dy = x: dw[1] over its channels is the sum over rows of K s / sqrt(s + eps), s the mean of
    # x^2 over the K values of the block; positive terms, of which a lane adds at most 3 rows /
    # (768 workgroups x 8 teams) = 2051 one after another: 2.2e3 x 2^-24 of the sum
    s = x[:, 1:].float().square().mean((1, 2)).double()
    want = float((3 * C * s / (s + EPS).sqrt()).sum())
    assert abs(float(dw[1].double().sum()) - want) <= 2e-4 * want
