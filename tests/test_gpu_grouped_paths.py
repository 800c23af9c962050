"""The channel mixing by group where its work is split another way: one group
with most of the rows, more groups than a wavefront has lanes, wide and ragged
channels, sums over many blocks, and the operators run together, against their
64-bit forms (tests/grouped_reference.py)."""
import numpy as np
import pytest

from clebsch_gordan_tensor_amd import synth as S
from tests import grouped_reference as R
from tests import norm_reference as N
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    from clebsch_gordan_tensor_amd import api
    api.lib()
    return api


def _ir(s):
    return S.parse_irreps(s)[1]


def _case(into, out, group, groups, cin, cout, dtype="f32", seed=0):
    rng = np.random.default_rng(len(group) + 13 * groups + cin + cout + seed)
    x = rng.standard_normal((len(group), S.dim(into), cin)).astype(np.float32)
    W = (rng.standard_normal((groups, len(R.pairs(into, out)), cin, cout)) /
         np.sqrt(cin)).astype(np.float32)
    dy = rng.standard_normal((len(group), S.dim(out), cout)).astype(np.float32)
    return [S.round_bf16(t) if dtype == "bf16" else t for t in (x, W, dy)]


def _skewed(rows, groups, share, seed=0):
    """A share of the rows in one group, the rest evenly; the last group has
    none and a few rows are in no group."""
    rng = np.random.default_rng(rows + groups + seed)
    g = rng.integers(0, max(groups - 1, 1), rows).astype(np.int32)
    g[rng.random(rows) < share] = groups // 2 if groups > 2 else 0
    g[rng.random(rows) < 0.02] = -1
    return g


def _check(gpu, into, out, group, x, W, dy, dtype):
    groups, bf16 = W.shape[0], dtype == "bf16"
    index = gpu.group_rows(dev(group), groups)
    X, Wd, D = dev(x, dtype), dev(W, dtype), dev(dy, dtype)
    y = gpu.linear_grouped(into, out, index, X, Wd)
    R.check(host(y), R.mix(into, out, group, x, W), "y", bf16)
    dx, dW = gpu.linear_grouped_backward(into, out, index, X, Wd, D, dW=torch.full(
        W.shape, np.nan, device="cuda"))
    rx, rW = R.mix_backward(into, out, group, x, W, dy)
    R.check(host(dx), rx, "dx", bf16)
    R.check(host(dW), rW, "dW")


# a group alone in parts; all of them; none; a part's rows and one more or less
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("xs,os_,rows,groups,share,cin,cout", [
    ("0e+1o+2e+3o", "0e+1o", 6000, 41, 0.3, 40, 16), ("0e+1o", "0e+1o", 9000, 3, 0.9, 16, 24),
    ("0e+0e", "0e", 5000, 70, 0.5, 8, 136), ("0e", "0e", 257, 2, 1.0, 16, 16),
    ("0e", "0e", 256, 1, 1.0, 16, 16), ("1o", "1o", 2000, 200, 0.2, 24, 16),
    ("0e", "0e", 4000, 4, 0.8, 264, 392), ("2e+0e", "0e+2e", 1300, 2, 0.6, 128, 128),
    ("0e", "0e", 700, 5, 0.7, 1992, 2040)])
def test_groups_of_other_lengths(gpu, xs, os_, rows, groups, share, cin, cout, dtype):
    into, out = _ir(xs), _ir(os_)
    group = _skewed(rows, groups, share)
    _check(gpu, into, out, group, *_case(into, out, group, groups, cin, cout, dtype), dtype)


# tiled products with more groups than the lanes that look for a tile
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("xs,os_,rows,groups,cin,cout", [
    ("0e", "0e", 3000, 65, 264, 136), ("0e+1o+0e", "1o+0e", 2500, 130, 72, 40),
    ("0e", "0e", 2300, 64, 512, 384), ("0e+0e+0e", "0e", 1500, 20, 328, 520),
    ("0e+1o", "0e+1o", 5000, 200, 128, 128)])
def test_many_groups(gpu, xs, os_, rows, groups, cin, cout, dtype):
    into, out = _ir(xs), _ir(os_)
    group = _skewed(rows, groups, 0.1)
    _check(gpu, into, out, group, *_case(into, out, group, groups, cin, cout, dtype), dtype)


# both sides of the rows at which the tiles of few rows give way to the large
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [127, 128, 129, 143, 144, 145])
def test_around_few_rows(gpu, rows, dtype):
    into = out = _ir("0e")
    for groups in (1, 2):
        group = _skewed(rows, groups, 0.5)
        _check(gpu, into, out, group, *_case(into, out, group, groups, 200, 264, dtype), dtype)


# every row on both sides of the sizes at which tiles of few rows give way to the others: where
# every block has one source of at most 128 channels at (16 groups + 112) / components rows,
# elsewhere by the tiles of 16 x 16 of all blocks (1200 in bf16, 6000 in float32, 1600 and 3000 in
# 8 bits; a row and a column of them for every group besides).  264 columns are 17 tiles.
@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8 f32", "fp8 bf16"])
@pytest.mark.parametrize("xs,os_,groups,cin,cout", [
    ("0e", "0e", 1, 144, 264), ("0e", "0e", 5, 264, 144), ("0e+0e+1o", "0e+1o", 2, 48, 80),
    ("0e+1o", "0e+1o", 3, 64, 48)])
def test_rows_on_both_sides(gpu, xs, os_, groups, cin, cout, dtype):
    into, out, most = _ir(xs), _ir(os_), 9001
    fp8 = dtype.startswith("fp8")
    if fp8:
        cin, cout = (-(-c // 16) * 16 for c in (cin, cout))
    group = _skewed(most, groups, 0.3) if groups > 1 else np.zeros(most, np.int32)
    x, W, dy = _case(into, out, group, groups, cin, cout, dtype)
    if fp8:
        packed = gpu.linear_fp8_pack(into, out, dev(W))
        of = torch.float32 if dtype == "fp8 f32" else None
        runs = [(dev(x), lambda i, t: gpu.linear_fp8(into, out, *gpu.quantize_fp8(t), packed,
                                                     index=i, dtype=of))]
    else:
        Wd = dev(W, dtype)
        # (zeros for dW's operand: only dx is looked at)
        runs = [(dev(x, dtype), lambda i, t: gpu.linear_grouped(into, out, i, t, Wd)),
                (dev(dy, dtype), lambda i, t: gpu.linear_grouped_backward(
                    into, out, i, torch.zeros((t.shape[0], S.dim(into), cin), device="cuda",
                                              dtype=t.dtype), Wd, t)[0])]
    limit = {"f32": 6000, "bf16": 1200, "fp8 f32": 3000, "fp8 bf16": 1600}[dtype]
    for k, (t, run) in enumerate(runs):
        whole = run(gpu.group_rows(dev(group), groups), t)
        blocks = [2 * l + 1 for l, _ in (into if k else out)]
        cols = -(-(cin if k else cout) // 16)
        last = max(n for n in range(1, most) if sum(
            (n * d + 15) // 16 + groups for d in blocks) * cols <= limit)
        few = (16 * groups + 112) // max(blocks)
        for n in {1, 17, few, few + 1, 400, last, last + 1, 6001}:
            got = run(gpu.group_rows(dev(group[:n]), groups), t[:n].contiguous())
            assert torch.equal(got, whole[:n]), n


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("xs,os_,rows,groups,cin,cout", [
    ("0e", "0e", 200, 1, 4096, 144), ("0e", "0e", 300, 3, 2064, 160), ("0e", "0e", 5, 1, 8192, 48),
    ("0e+0e+0e", "0e", 400, 2, 912, 128), ("0e+1o+0e", "1o+0e", 900, 130, 80, 48),
    ("0e", "0e", 2500, 70, 272, 400), ("0e+1o", "0e+1o", 2000, 100, 128, 128)])
def test_mixing_in_8_bits(gpu, xs, os_, rows, groups, cin, cout, out_dtype):
    into, out = _ir(xs), _ir(os_)
    group = _skewed(rows, groups, 0.2) if groups > 1 else np.zeros(rows, np.int32)
    x, W, _ = _case(into, out, group, groups, cin, cout)
    index = gpu.group_rows(dev(group), groups) if groups > 1 else None
    q, scale = gpu.quantize_fp8(dev(x))
    y = gpu.linear_fp8(into, out, q, scale, gpu.linear_fp8_pack(into, out, dev(W)), index=index,
                       dtype=torch.float32 if out_dtype == "f32" else None)
    xv = R.values(host(q.float()).astype(np.float64), host(scale))
    ref = R.mix(into, out, group, xv, R.weight_values(*R.quantize_weights(W)))
    bf16 = out_dtype == "bf16"
    R.check(host(y), ref, "y", bf16, adds=1, drops=R.EIGHTS if bf16 else 0.0)


# no block of the input has a target: nothing of W is there to be read
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", [(5, 48), (700, 48), (5, 208), (9000, 208)])
def test_no_pairs(gpu, rows, C, dtype):
    into, out = _ir("0e+2e"), _ir("1o+0o")
    group = _skewed(rows, 3, 0.3)
    x, W, dy = _case(into, out, group, 3, C, C, dtype)
    assert W.shape[1] == 0
    index, X, Wd = gpu.group_rows(dev(group), 3), dev(x, dtype), torch.empty(
        W.shape, device="cuda", dtype=torch.float32 if dtype == "f32" else torch.bfloat16)
    y = gpu.linear_grouped(into, out, index, X, Wd, out=torch.full_like(dev(dy, dtype), 3.0))
    dx, dW = gpu.linear_grouped_backward(into, out, index, X, Wd, dev(dy, dtype),
                                         dx=torch.full_like(X, 3.0))
    assert not y.any() and not dx.any() and dW.shape == W.shape
    packed = gpu.linear_fp8_pack(into, out, torch.empty(W.shape, device="cuda"))
    y = gpu.linear_fp8(into, out, *gpu.quantize_fp8(X), packed, index=index)
    assert y.shape == dy.shape and not y.any()


# a row alone, among few and among many: the same bits, whichever tiles it is in
@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8 f32", "fp8 bf16"])
@pytest.mark.parametrize("xs,os_,cin,cout", [
    ("0e+0e+1o", "0e+1o", 208, 272), ("0e", "0e", 1040, 560), ("0e+1o", "0e+1o", 96, 144)])
def test_a_row_alone(gpu, xs, os_, cin, cout, dtype):
    into, out = _ir(xs), _ir(os_)
    group = _skewed(4000, 3, 0.4)
    x, W, dy = _case(into, out, group, 3, cin, cout, dtype)
    if dtype.startswith("fp8"):
        packed = gpu.linear_fp8_pack(into, out, dev(W))
        of = torch.float32 if dtype == "fp8 f32" else None
        runs = [(dev(x), lambda i, t: gpu.linear_fp8(into, out, *gpu.quantize_fp8(t), packed,
                                                     index=i, dtype=of))]
    else:
        Wd = dev(W, dtype)
        # (zeros for dW's operand: only dx is looked at)
        runs = [(dev(x, dtype), lambda i, t: gpu.linear_grouped(into, out, i, t, Wd)),
                (dev(dy, dtype), lambda i, t: gpu.linear_grouped_backward(
                    into, out, i, torch.zeros((t.shape[0], S.dim(into), cin), device="cuda",
                                              dtype=t.dtype), Wd, t)[0])]
    for t, run in runs:
        whole = run(gpu.group_rows(dev(group), 3), t)
        for n in (1, 20, 150, 600, 1500):
            assert torch.equal(run(gpu.group_rows(dev(group[:n]), 3), t[:n].contiguous()),
                               whole[:n]), n


def _train(gpu, ir, groups, X, Rd, Wn, B, W, Gd, dY, dH, stream=None):
    """A layer's pass: h = x + r normalised and mixed by element, then back."""
    index = gpu.group_rows(Gd, groups, stream=stream)
    n, h = gpu.layer_norm_residual(ir, X, Rd, Wn, B, stream=stream)
    y = gpu.linear_grouped(ir, ir, index, n, W, stream=stream)
    dn, dW = gpu.linear_grouped_backward(ir, ir, index, n, W, dY, stream=stream)
    dx, dw, db = gpu.layer_norm_residual_backward(ir, h, Wn, dn, dH, stream=stream)
    return y, h, n, dn, dW, dx, dw, db


def _layer(rows, groups, C, seed=0):
    ir = _ir("0e+1o+2e")
    group = _skewed(rows, groups, 0.4, seed)
    x, W, dy = _case(ir, ir, group, groups, C, C, seed=seed)
    rng = np.random.default_rng(seed + 5)
    r, dh = rng.standard_normal((2, *x.shape)).astype(np.float32)
    wn = (1 + 0.2 * rng.standard_normal((3, C))).astype(np.float32)
    b = rng.standard_normal((1, C)).astype(np.float32)
    return ir, group, x, W, dy, r, dh, wn, b


def test_a_layer_and_its_gradients(gpu):
    ir, group, x, W, dy, r, dh, wn, b = _layer(1500, 4, 64)
    got = _train(gpu, ir, 4, *map(dev, (x, r, wn, b, W, group, dy, dh)))
    y, h, n, dn, dW, dx, dw, db = map(host, got)
    # every step against its plain form on what the step before gave
    assert np.array_equal(h, x + r)
    ref, tol = N.norm_forward(ir, h, wn, b, 1e-5)
    assert np.all(np.abs(n - ref) <= tol)
    R.check(y, R.mix(ir, ir, group, n, W), "y")
    rx, rW = R.mix_backward(ir, ir, group, n, W, dy)
    R.check(dn, rx, "dn")
    R.check(dW, rW, "dW")
    (gx, gw, gb), (tx, tw, tb) = N.norm_backward(ir, h, wn, dn, 1e-5)
    assert np.all(np.abs(dx - (gx + dh)) <= tx + R.U * np.abs(gx + dh))
    assert np.all(np.abs(dw - gw) <= tw) and np.all(np.abs(db - gb) <= tb)


def test_layers_on_two_streams(gpu):
    # two passes at once, each with its own memory: what each gives alone
    cases = [_layer(n, 5, 64, seed) for n, seed in ((3000, 1), (4100, 2))]
    args = [(ir, 5, *map(dev, (x, r, wn, b, W, group, dy, dh)))
            for ir, group, x, W, dy, r, dh, wn, b in cases]
    alone = [_train(gpu, *a) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        both = []
        for a, s in zip(args, streams):
            with torch.cuda.stream(s):
                both.append(_train(gpu, *a, stream=s))
        torch.cuda.synchronize()
        for one, two in zip(alone, both):
            for p, q in zip(one, two):
                assert torch.equal(p, q)


def _ends(rows, k, width, dtype, seed, comps=1):
    """Zeros but for k random rows at the end, [rows][comps][width], and these."""
    rng = np.random.default_rng(seed)
    end = S.round_bf16(rng.standard_normal((k, comps, width)).astype(np.float32))
    t = torch.zeros((rows, comps, width), device="cuda", dtype=dtype)
    t[rows - k:] = dev(end).to(dtype)
    return t, end


# as many rows as an index may have: places past the last row are past 2^31 as well
@pytest.mark.parametrize("with_index", [False, True])
def test_most_rows(gpu, with_index):
    rows, k, into = 2 ** 31 - 1, 700, _ir("0e")
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 180e9:
        pytest.skip("needs 180 GB")
    groups, g = (2, 1) if with_index else (1, 0)
    index = None
    if with_index:
        index = gpu.group_rows(torch.ones(rows, device="cuda", dtype=torch.int32), groups)
        assert index.offsets.tolist() == [0, 0, rows]
        assert torch.equal(index.order[-k:].long(), torch.arange(rows - k, rows, device="cuda"))
    x, xe = _ends(rows, k, 8, torch.bfloat16, 1)
    dy, de = _ends(rows, k, 8, torch.bfloat16, 2)
    W = S.round_bf16(np.random.default_rng(3).standard_normal((groups, 1, 8, 8)).astype(np.float32))
    Wd, of = dev(W, "bf16"), np.full(k, g)
    y = gpu.linear_grouped(into, into, index, x, Wd)
    R.check(host(y[-k:]), R.mix(into, into, of, xe, W), "y", True)
    assert not y[:100_000_000].any() and not y[-100_000_000:-k].any()
    del y
    dx, dW = gpu.linear_grouped_backward(into, into, index, x, Wd, dy)
    rx, rW = R.mix_backward(into, into, of, xe, W, de)
    R.check(host(dx[-k:]), rx, "dx", True)
    R.check(host(dW), rW, "dW")
    del x, dx, dy, index
    torch.cuda.empty_cache()


def test_most_rows_in_8_bits(gpu):
    rows, k, into = 2 ** 31 - 1, 700, _ir("0e")
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 180e9:
        pytest.skip("needs 180 GB")
    q, xe = _ends(rows, k, 16, torch.float8_e4m3fn, 4)
    scale = torch.ones((rows, 1, 1), device="cuda")
    W = np.random.default_rng(5).standard_normal((1, 1, 16, 16)).astype(np.float32)
    y = gpu.linear_fp8(into, into, q, scale, gpu.linear_fp8_pack(into, into, dev(W)))
    xv = host(q[-k:].float()).astype(np.float64)
    assert np.array_equal(xv, R.e4m3(xe))
    ref = R.mix(into, into, np.zeros(k, int), xv, R.weight_values(*R.quantize_weights(W)))
    R.check(host(y[-k:]), ref, "y", True, adds=1, drops=R.EIGHTS)
    assert not y[:100_000_000].any() and not y[-100_000_000:-k].any()
    del q, scale, y
    torch.cuda.empty_cache()


# more tiles than one launch holds threads for: 2^24 workgroups and more
@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_more_tiles_than_a_launch(gpu, dtype):
    rows, k, ir = 2 ** 30 + 70_000, 700, _ir("0e+0e")
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 180e9:
        pytest.skip("needs 180 GB")
    C, of = 16 if dtype == "fp8" else 8, np.zeros(k, int)
    T = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}[dtype]
    x, xe = _ends(rows, k, C, T, 1, 2)
    W = S.round_bf16(np.random.default_rng(3).standard_normal((1, 4, C, C)).astype(np.float32))
    y = torch.full((rows, 2, C), 3.0, device="cuda",
                   dtype=torch.float32 if dtype == "f32" else torch.bfloat16)
    if dtype == "fp8":
        scale = torch.ones((rows, 2, 1), device="cuda")
        gpu.linear_fp8(ir, ir, x, scale, gpu.linear_fp8_pack(ir, ir, dev(W)), out=y)
        ref = R.mix(ir, ir, of, R.e4m3(xe), R.weight_values(*R.quantize_weights(W)))
        R.check(host(y[-k:]), ref, "y", True, adds=1, drops=R.EIGHTS)
        del scale
    else:
        Wd, bf16 = dev(W, dtype), dtype == "bf16"
        gpu.linear_grouped(ir, ir, None, x, Wd, out=y)
        R.check(host(y[-k:]), R.mix(ir, ir, of, xe, W), "y", bf16)
    assert not y[:-k].any()
    if dtype == "bf16":
        del y
        dx = torch.full_like(x, 3.0)
        _, dW = gpu.linear_grouped_backward(ir, ir, None, x, Wd, x, dx=dx)
        rx, rW = R.mix_backward(ir, ir, of, xe, W, xe)
        R.check(host(dx[-k:]), rx, "dx", True)
        R.check(host(dW), rW, "dW")
        assert not dx[:-k].any()
        del dx
    del x
    torch.cuda.empty_cache()
