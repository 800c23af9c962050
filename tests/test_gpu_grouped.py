"""The index of rows by group and the channel mixing with weights per group,
with its gradients, on the GPU against their 64-bit forms
(tests/grouped_reference.py)."""
import ctypes

import numpy as np
import pytest

from clebsch_gordan_tensor_amd import synth as S
from tests import grouped_reference as R
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


# -------------------------------------------------------------------- index

@pytest.mark.parametrize("n_groups", [1, 2, 10, 63, 64, 118, 1024])
@pytest.mark.parametrize("rows", [0, 1, 63, 64, 65, 700, 2048, 8191, 8192, 8193, 30011, 600001])
def test_index(gpu, rows, n_groups):
    rng = np.random.default_rng(rows + n_groups)
    ids = (rng.random(rows) ** 2 * n_groups).astype(np.int32)
    ids[rng.random(rows) < 0.05] = -1
    ids[rng.random(rows) < 0.01] = n_groups
    if rows > 2:
        ids[1], ids[2] = np.iinfo(np.int32).min, np.iinfo(np.int32).max
    order, offsets = R.index(ids, n_groups)
    got = gpu.group_rows(dev(ids), n_groups)
    assert np.array_equal(host(got.order), order)
    assert np.array_equal(host(got.offsets), offsets)


def test_index_of_one_group_and_of_none(gpu):
    for ids in (np.full(5000, 7, np.int32), np.full(20000, -3, np.int32),
                np.full(20000, 11, np.int32)):
        order, offsets = R.index(ids, 12)
        got = gpu.group_rows(dev(ids), 12)
        assert np.array_equal(host(got.order), order)
        assert np.array_equal(host(got.offsets), offsets)


# ------------------------------------------------------------------- mixing

def _case(into, out, rows, groups, cin, cout, dtype, stray=0.1, seed=0):
    rng = np.random.default_rng(rows * 31 + groups * 7 + cin + cout + seed)
    group = (rng.random(rows) ** 2 * groups).astype(np.int32)
    group[rng.random(rows) < stray] = -1
    x = rng.standard_normal((rows, S.dim(into), cin)).astype(np.float32)
    W = (rng.standard_normal((groups, len(R.pairs(into, out)), cin, cout)) /
         np.sqrt(cin)).astype(np.float32)
    dy = rng.standard_normal((rows, S.dim(out), cout)).astype(np.float32)
    if dtype == "bf16":
        x, W, dy = S.round_bf16(x), S.round_bf16(W), S.round_bf16(dy)
    return group, x, W, dy


def _check(gpu, into, out, group, x, W, dy, dtype, with_index=True):
    groups, bf16 = W.shape[0], dtype == "bf16"
    index = gpu.group_rows(dev(group), groups) if with_index else None
    X, Wd, D = dev(x, dtype), dev(W, dtype), dev(dy, dtype)
    y = gpu.linear_grouped(into, out, index, X, Wd)
    R.check(host(y), R.mix(into, out, group, x, W), "y", bf16)
    dx, dW = gpu.linear_grouped_backward(into, out, index, X, Wd, D)
    rx, rW = R.mix_backward(into, out, group, x, W, dy)
    R.check(host(dx), rx, "dx", bf16)
    R.check(host(dW), rW, "dW")
    out_of = np.nonzero((group < 0) | (group >= groups))[0]
    assert not host(y)[out_of].any() and not host(dx)[out_of].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("xs,os_,rows,groups,cin,cout", [
    ("0e+1o+2e+3o", "0e+1o+2e+3o", 301, 5, 128, 128),
    ("0e+1o+2e+3o", "0e+1o+2e+3o", 1, 10, 128, 128),
    ("0e+1o", "0e+1o", 64, 3, 8, 8),                   # the smallest widths
    ("0e+1o", "0e+1o+2e+3o", 77, 4, 64, 96),           # output blocks without a source
    ("0e+0e+1o+2e", "1o+0e", 130, 7, 40, 24),          # two sources of a block, one without a target
    ("1o+0e", "0e+1o+1o", 90, 6, 32, 200),             # two targets of a block
    ("0e", "0e", 333, 16, 520, 264),                   # wide, ragged against every tile
    ("0e", "0e", 3, 2, 2048, 136),
    ("0e", "0e", 700, 3, 72, 1000),
    ("8e+0e", "8e", 40, 100, 16, 16),                  # more groups than rows
    ("0e+1o+2e", "0e+1o+2e", 2001, 1000, 16, 32),      # many groups, most of them small
    ("1o", "1o", 4097, 2, 256, 256),                   # several parts of the weight gradient
    ("0e+1o", "0e+1o", 20011, 3, 64, 64),
])
def test_mixing(gpu, xs, os_, rows, groups, cin, cout, dtype):
    into, out = _ir(xs), _ir(os_)
    _check(gpu, into, out, *_case(into, out, rows, groups, cin, cout, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 129, 5000])
def test_one_group_needs_no_index(gpu, rows, dtype):
    into = out = _ir("0e+1o+2e")
    case = _case(into, out, rows, 1, 64, 128, dtype, stray=0.0)
    _check(gpu, into, out, *case, dtype, with_index=False)
    _check(gpu, into, out, *case, dtype)


def test_like_the_ungrouped_mixing(gpu):
    # one set of weights for all groups: e3_linear's results
    into = out = _ir("0e+1o+2e+3o")
    group, x, W, _ = _case(into, out, 500, 4, 128, 128, "f32", stray=0.0)
    W[:] = W[:1]
    y = host(gpu.linear_grouped(into, out, gpu.group_rows(dev(group), 4), dev(x), dev(W)))
    ref = host(gpu.linear(into, out, dev(x), dev(W[0])))
    size = R.mix(into, out, group, x, W)[1]
    assert np.all(np.abs(y - ref) <= 2 * (R.ADDS * 128 + 16) * R.U * size)


def test_no_rows_and_rows_without_a_group(gpu):
    into = out = _ir("0e+1o")
    for rows, ids in ((0, 0), (300, -1), (300, 3)):
        group, x, W, dy = _case(into, out, rows, 3, 16, 24, "f32")
        group[:] = ids
        index = gpu.group_rows(dev(group), 3)
        y = gpu.linear_grouped(into, out, index, dev(x), dev(W), out=torch.full(
            (rows, 4, 24), 5.0, device="cuda"))
        dx, dW = gpu.linear_grouped_backward(into, out, index, dev(x), dev(W), dev(dy),
                                             dW=torch.full(W.shape, 5.0, device="cuda"))
        assert not y.any() and not dx.any() and not dW.any()


def test_values_far_apart(gpu):
    # sizes from 1e-30 to 1e30 in one row, each against weights of the inverse size
    into = out = _ir("0e")
    rng = np.random.default_rng(5)
    scale = 10.0 ** rng.uniform(-30, 30, 96)
    x = (rng.standard_normal((200, 1, 96)) * scale).astype(np.float32)
    W = (rng.standard_normal((2, 1, 96, 64)) / scale[:, None]).astype(np.float32)
    group = rng.integers(0, 2, 200).astype(np.int32)
    y = gpu.linear_grouped(into, out, gpu.group_rows(dev(group), 2), dev(x), dev(W))
    R.check(host(y), R.mix(into, out, group, x, W), "far apart")


def _near(got, ref, extra, what):
    """R.check's bound for every element, and `extra` besides."""
    y, size, terms = ref
    tol = (R.ADDS * terms + 16) * R.U * size + R.U * np.abs(y) + extra
    bad = np.abs(got.astype(np.float64) - y) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside"


# factors down to float32's least: 24 bits to 2^-110, what is below 2^-134 of a smaller one is lost
# (bf16's least value is 2^-133, and a part is the rest rounded to nearest)
@pytest.mark.parametrize("rows,cin,cout", [(3, 96, 64), (400, 96, 64), (300, 520, 136),
                                           (6000, 264, 200)])
def test_values_near_the_least(gpu, rows, cin, cout):
    into = out = _ir("0e")
    rng = np.random.default_rng(rows + cin)
    group = rng.integers(0, 2, rows).astype(np.int32)
    index = gpu.group_rows(dev(group), 2)

    def factors(low, high):
        """Rows and weights, every channel's of inverse sizes."""
        size = 2.0 ** rng.uniform(low, high, cin)
        sign = lambda *n: rng.choice([-1.0, 1.0], n) * rng.uniform(1, 2, n)  # noqa: E731
        return ((sign(rows, 1, cin) * size).astype(np.float32),
                (sign(2, 1, cin, cout) / size[:, None]).astype(np.float32))

    def both(x, W, least):
        """least: the error of every x (of every W, of neither)."""
        y = gpu.linear_grouped(into, out, index, dev(x), dev(W))
        of_x = R.mix(into, out, group, np.ones_like(x), np.abs(W))[1] * (least == "x")
        of_w = R.mix(into, out, group, np.abs(x), np.ones_like(W))[1] * (least == "W")
        _near(host(y), R.mix(into, out, group, x, W), 2.0 ** -134 * (of_x + of_w), "y")

    both(*factors(-110, -100), None)
    both(*factors(-124, -100), "x")
    x, W = factors(100, 124)
    both(x, W, "W")
    # the gradients: dy in the place of x or W
    x, W = factors(-124, -100)
    dy = (rng.standard_normal((rows, 1, cout)) * 2.0 ** rng.uniform(-124, -100, (rows, 1, 1))
          ).astype(np.float32)
    W = (rng.standard_normal(W.shape) * 2.0 ** 100).astype(np.float32)
    x = (rng.standard_normal(x.shape) * 2.0 ** 100).astype(np.float32)
    dx, dW = gpu.linear_grouped_backward(into, out, index, dev(x), dev(W), dev(dy))
    rx, rW = R.mix_backward(into, out, group, x, W, dy)
    one = R.mix_backward(into, out, group, np.abs(x), np.abs(W), np.ones_like(dy))
    _near(host(dx), rx, 2.0 ** -134 * one[0][1], "dx")
    _near(host(dW), rW, 2.0 ** -134 * one[1][1], "dW")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_that_are_not_finite_stay_in_their_rows(gpu, dtype):
    into = out = _ir("0e+1o")
    group, x, W, dy = _case(into, out, 300, 3, 64, 32, dtype, stray=0.2)
    index = gpu.group_rows(dev(group), 3)
    clean = gpu.linear_grouped(into, out, index, dev(x, dtype), dev(W, dtype))
    for row, bad in ((3, np.inf), (150, np.nan), (299, -np.inf)):
        x[row, 2, 5] = bad
    group2 = group.copy()
    got = gpu.linear_grouped(into, out, index, dev(x, dtype), dev(W, dtype))
    keep = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
    for row in (3, 150, 299):
        keep[row, 2] = False
        if group2[row] >= 0:
            assert not torch.isfinite(got[row, 2]).any()
        else:  # a row without a group is not read
            assert not got[row, 2].any()
    assert torch.equal(got[keep], clean[keep])
    # rows without a group add nothing to dW, whatever they hold
    x, dy = np.nan_to_num(x, posinf=1, neginf=1), dy.copy()
    rx, rW = R.mix_backward(into, out, group, x, W, dy)
    stray = group < 0
    assert stray.sum() > 5
    x[stray], dy[stray] = np.nan, np.inf
    dx, dW = gpu.linear_grouped_backward(into, out, index, dev(x, dtype), dev(W, dtype),
                                         dev(dy, dtype))
    R.check(host(dW), rW, "dW")
    R.check(host(dx), rx, "dx", dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_row_does_not_depend_on_the_others(gpu, dtype):
    into = out = _ir("0e+1o+2e")
    group, x, W, _ = _case(into, out, 400, 3, 64, 64, dtype, stray=0.0)
    X, Wd = dev(x, dtype), dev(W, dtype)
    all_ = gpu.linear_grouped(into, out, gpu.group_rows(dev(group), 3), X, Wd)
    for n in (1, 17, 130):
        some = gpu.linear_grouped(into, out, gpu.group_rows(dev(group[:n]), 3),
                                  X[:n].contiguous(), Wd)
        assert torch.equal(some, all_[:n])


def test_gradients_not_wanted(gpu):
    into, out = _ir("0e+1o"), _ir("0e+1o")
    group, x, W, dy = _case(into, out, 5000, 2, 64, 64, "f32")
    index = gpu.group_rows(dev(group), 2)
    X, Wd, D = dev(x), dev(W), dev(dy)
    dx, dW = gpu.linear_grouped_backward(into, out, index, X, Wd, D)
    a, b = gpu._irreps_struct(into, 64), gpu._irreps_struct(out, 64)
    nb = gpu.linear_grouped_workspace_size(into, out, 64, 64, 5000, 2)
    ws = torch.empty(nb, device="cuda", dtype=torch.uint8)
    for want_x, want_w in ((1, 0), (0, 1), (0, 0)):
        gx, gw = torch.full_like(dx, 3.0), torch.full_like(dW, 3.0)
        gpu._check(gpu.lib().e3_linear_grouped_backward(
            ctypes.byref(a), ctypes.byref(b), 5000, 2, index.buffer.data_ptr(),
            index.buffer.numel(), X.data_ptr(), Wd.data_ptr(), D.data_ptr(),
            gx.data_ptr() if want_x else None, gw.data_ptr() if want_w else None, ws.data_ptr(),
            nb, 0, torch.cuda.current_stream().cuda_stream))
        assert torch.equal(gx, dx) if want_x else (gx == 3.0).all()
        assert torch.equal(gw, dW) if want_w else (gw == 3.0).all()


def test_an_index_of_other_sizes_changes_nothing(gpu):
    into = out = _ir("0e+1o")
    group, x, W, dy = _case(into, out, 3000, 2, 16, 16, "f32")
    other = gpu.group_rows(dev(group[:2900]), 2)
    buf = torch.zeros(gpu._index_sizes(3000, 2)[0], device="cuda", dtype=torch.uint8)
    buf[:other.buffer.numel()] = other.buffer
    wrong = gpu.RowGroups(buf, 3000, 2)
    keep = torch.full((3000, 4, 16), 9.0, device="cuda")
    y = gpu.linear_grouped(into, out, wrong, dev(x), dev(W), out=keep.clone())
    dx, dW = gpu.linear_grouped_backward(into, out, wrong, dev(x), dev(W), dev(dy),
                                         dx=keep.clone(), dW=torch.full(W.shape, 9.0, device="cuda"))
    assert torch.equal(y, keep) and torch.equal(dx, keep) and (dW == 9.0).all()


def test_gradients_against_differences(gpu):
    into, out = _ir("0e+1o"), _ir("1o+0e")
    group, x, W, dy = _case(into, out, 50, 3, 16, 24, "f32")
    index = gpu.group_rows(dev(group), 3)
    X, Wd, D = dev(x), dev(W), dev(dy)
    dx, dW = gpu.linear_grouped_backward(into, out, index, X, Wd, D)
    loss = lambda x, w: float((gpu.linear_grouped(into, out, index, x, w).double() *  # noqa: E731
                               D.double()).sum())
    rng = np.random.default_rng(0)
    for t, g, f in ((X, dx, lambda v: loss(v, Wd)), (Wd, dW, lambda v: loss(X, v))):
        d = dev(rng.standard_normal(tuple(t.shape)).astype(np.float32))
        # the loss is linear in each: differences of any step are exact but for rounding
        num = (f(t + d) - f(t - d)) / 2
        ana = float((g.double() * d.double()).sum())
        scale = float((g.double() * d.double()).abs().sum())
        assert abs(num - ana) <= 1e-5 * scale, (num, ana)


def test_far_rows(gpu):
    # x and y past 2^31 elements: rows at both ends and on both sides of the border
    into = out = _ir("0e+1o+2e+3o")
    rows, C = 1_060_000, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((rows, 16, C), device="cuda", generator=gen, dtype=torch.bfloat16)
    W = torch.randn((2, 4, C, C), device="cuda", generator=gen).mul_(0.1).to(torch.bfloat16)
    group = (torch.arange(rows, device="cuda") % 3).int()  # a third has none
    index = gpu.group_rows(group, 2)
    y = gpu.linear_grouped(into, out, index, x, W)
    pick = torch.tensor([0, 1, 2, 2 ** 31 // 2048 - 1, 2 ** 31 // 2048, 2 ** 31 // 2048 + 1,
                         rows - 3, rows - 2, rows - 1], device="cuda")
    ref = R.mix(into, out, host(group[pick]), host(x[pick]), host(W))
    R.check(host(y[pick]), ref, "far rows", True)
    dx, _ = gpu.linear_grouped_backward(into, out, index, x, W, y)
    ref, _ = R.mix_backward(into, out, host(group[pick]), host(x[pick]), host(W), host(y[pick]))
    R.check(host(dx[pick]), ref, "far rows dx", True)


@pytest.mark.parametrize("rows", [40, 20011])
def test_captured_and_on_another_stream(gpu, rows):
    into = out = _ir("0e+1o")
    group, x, W, dy = _case(into, out, rows, 5, 64, 64, "f32")
    X, Wd, D, Gd = dev(x), dev(W), dev(dy), dev(group)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    index = gpu.group_rows(Gd, 5, stream=side)
    y = gpu.linear_grouped(into, out, index, X, Wd, stream=side)
    dx, dW = gpu.linear_grouped_backward(into, out, index, X, Wd, D, stream=side)
    side.synchronize()
    index0 = gpu.group_rows(Gd, 5)
    ref = [gpu.linear_grouped(into, out, index0, X, Wd),
           *gpu.linear_grouped_backward(into, out, index0, X, Wd, D)]
    for a, b in zip((y, dx, dW), ref):
        assert torch.equal(a, b)
    ws = torch.empty(gpu.linear_grouped_workspace_size(into, out, 64, 64, rows, 5), device="cuda",
                     dtype=torch.uint8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu.group_rows(Gd, 5, index=index)
        gpu.linear_grouped(into, out, index, X, Wd, out=y)
        gpu.linear_grouped_backward(into, out, index, X, Wd, D, dx=dx, dW=dW, workspace=ws)
    for seed in range(4):  # other rows, groups and weights every time
        group, x, W, dy = _case(into, out, rows, 5, 64, 64, "f32", seed=seed + 1)
        for t, v in ((X, x), (Wd, W), (D, dy), (Gd, group)):
            t.copy_(torch.from_numpy(v))
        for t in (y, dx, dW):
            t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        fresh = gpu.group_rows(Gd, 5)
        ref = [gpu.linear_grouped(into, out, fresh, X, Wd),
               *gpu.linear_grouped_backward(into, out, fresh, X, Wd, D)]
        for a, b in zip((y, dx, dW), ref):
            assert torch.equal(a, b)
