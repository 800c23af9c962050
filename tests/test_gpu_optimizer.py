"""The gradients' norm and the AdamW step on the GPU against their 64-bit
forms.  Float32 results are held to their own rounding errors
(tests/norm_reference.py); 8-bit codes to the codes of the 64-bit moments,
exactly."""
import numpy as np
import pytest

from clebsch_gordan_tensor_amd import synth as S
from tests import norm_reference as R
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LR, WD = 1e-2, 0.1


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    from clebsch_gordan_tensor_amd import api
    api.lib()
    return api


class Net:
    """Tensors of given sizes with gradients and moments, on the host and the GPU."""

    def __init__(self, gpu, sizes, bits, seed, grad="f32", copies=False, decay=WD, zeros=False,
                 scale=1e-2):
        rng = np.random.default_rng(seed)
        self.bits = [bits] * len(sizes) if isinstance(bits, int) else bits
        f = lambda n: rng.standard_normal(n).astype(np.float32)  # noqa: E731
        self.p = [f(n) for n in sizes]
        self.g = [(scale * f(n) * np.exp(2 * f(n))).astype(np.float32) for n in sizes]
        if grad == "bf16":
            self.g = [S.round_bf16(g) for g in self.g]
        self.m, self.v, self.ms, self.vs = [], [], [], []
        for n, b in zip(sizes, self.bits):
            m, v = 0.3 * scale * f(n) * (not zeros), (scale * f(n)) ** 2 * (not zeros)
            if b == 8:
                ms, vs = R.scales(m, v)
                cm, _ = R.codes(np.abs(m.astype(np.float64)), ms, 127, 1)
                cv, _ = R.codes(v.astype(np.float64), vs, 255, 2)
                m, v = (cm * np.sign(m)).astype(np.int8), np.maximum(cv, v > 0).astype(np.uint8)
                self.ms.append(ms), self.vs.append(vs)
            else:
                self.ms.append(None), self.vs.append(None)
            self.m.append(m), self.v.append(v)
        up = lambda a: [None if t is None else dev(t) for t in a]  # noqa: E731
        self.G = [dev(g, grad) for g in self.g]
        self.P, self.M, self.V, self.MS, self.VS = map(up, (self.p, self.m, self.v, self.ms,
                                                            self.vs))
        self.C = [p.to(torch.bfloat16) for p in self.P] if copies else None
        self.decay = [decay * (i % 2) for i in range(len(sizes))]
        self.list = gpu.Params(self.P, self.G, self.M, self.V, m_scale=self.MS, v_scale=self.VS,
                               copies=self.C, weight_decay=self.decay)

    def values(self, i):
        if self.bits[i] == 8:
            return R.decode(self.m[i], self.v[i], self.ms[i], self.vs[i])
        return self.m[i].astype(np.float64), self.v[i].astype(np.float64)

    def check(self, gpu, t, lr=LR, scale=1.0, **betas):
        for i in range(len(self.p)):
            n = self.p[i].size
            (p, m, v), (tp, tm, tv) = R.adamw(self.p[i], self.g[i], *self.values(i), t, lr,
                                              float(np.float32(self.decay[i])), scale=scale, **betas)
            what = f"tensor {i} ({n} elements, {self.bits[i]} bits)"
            got = host(self.P[i]).astype(np.float64)
            assert np.all(np.abs(got - p) <= tp), (what, np.max(np.abs(got - p) / tp))
            if self.C:
                assert torch.equal(self.C[i], self.P[i].to(torch.bfloat16)), what
            if self.bits[i] == 32:
                for a, r, tol in ((self.M[i], m, tm), (self.V[i], v, tv)):
                    assert np.all(np.abs(host(a) - r) <= tol), what
                continue
            ms, vs = host(self.MS[i]), host(self.VS[i])
            for a, r in zip((ms, vs), R.scales(m, v)):
                assert np.all(np.abs(a - r) <= np.maximum(2.0 ** -23 * r, 2.0 ** -149)), what
            for a, r, s, top, power in ((host(self.M[i]), np.abs(m), ms, 127, 1),
                                        (host(self.V[i]), v, vs, 255, 2)):
                c, near = R.codes(r, s, top, power)
                c = np.maximum(c, r > 0) if power == 2 else c * np.sign(m).astype(np.int64)
                assert np.array_equal(a[~near], c[~near]), what
                assert np.all(np.abs(a[near].astype(int) - c[near]) <= 1), what


SIZES = [1, 2, 3, 255, 256, 257, 1000, 4096, 4097, 70001]


@pytest.mark.parametrize("t", [1, 2, 1000, 10 ** 9])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_step(gpu, bits, grad, t):
    net = Net(gpu, SIZES, bits, t % 97 + bits, grad, copies=grad == "bf16")
    gpu.adamw(net.list, t, LR)
    net.check(gpu, t)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_steps_from_zero(gpu, bits):
    net = Net(gpu, [1000, 5], bits, 3, zeros=True)
    m, v, ms, vs = gpu.adamw_state(net.P, bits)
    assert all(torch.equal(a, b) for a, b in zip(m + v, net.M + net.V))
    assert ms == vs == [None, None] if bits == 32 else torch.all(ms[0] == 0)
    gpu.adamw(net.list, 1, LR)
    net.check(gpu, 1)


@pytest.mark.parametrize("scale", [1e-12, 1e-14, 1e-16, 1e-18, 1e-20, 1e8, 1e17])
def test_gradients_of_any_size(gpu, scale):
    # moments down to float32's smallest values and up to its largest; the scales' own float32
    # rounding (absolute where they are subnormal) is taken from the GPU's
    net = Net(gpu, [5000], 8, 4, scale=scale)
    gpu.adamw(net.list, 3, LR)
    net.check(gpu, 3)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("b1,b2,eps", [(0.0, 0.0, 1e-8), (0.0, 0.99, 1e-3), (0.95, 0.0, 1e-30),
                                       (0.5, 0.9999, 1.0)])
def test_other_constants(gpu, b1, b2, eps, bits):
    net = Net(gpu, [1000, 77], bits, 17)
    gpu.adamw(net.list, 5, LR, beta1=b1, beta2=b2, eps=eps)
    net.check(gpu, 5, b1=b1, b2=b2, eps=eps)


def test_a_count_below_one_is_one(gpu):
    a, b = (Net(gpu, [300], 32, 18) for _ in range(2))
    gpu.adamw(a.list, torch.full((1,), -4, device="cuda", dtype=torch.int64), LR)
    gpu.adamw(b.list, 1, LR)
    assert torch.allclose(a.P[0], b.P[0], rtol=1e-6, atol=1e-7)


def test_mixed_list(gpu):
    # more tensors than one launch takes, empty ones and both forms of the moments among them
    rng = np.random.default_rng(5)
    sizes = [int(n) for n in rng.integers(0, 3000, 130)]
    sizes[3] = sizes[64] = 0
    net = Net(gpu, sizes, [8 if i % 3 else 32 for i in range(130)], 6)
    gpu.adamw(net.list, 7, LR)
    net.check(gpu, 7)


def test_all_alike_and_zero_blocks(gpu):
    # runs of zeros, one value only, and values whose squares leave float32's range
    net = Net(gpu, [1024], 8, 7, zeros=True)
    g = np.zeros(1024, np.float32)
    g[256:512], g[600], g[768:] = 0.25, -3.0, 1e-30
    net.g, _ = [g], net.G[0].copy_(dev(g))
    gpu.adamw(net.list, 1, LR)
    p = host(net.P[0])
    assert np.array_equal(p[:256], net.p[0][:256]) and np.isfinite(p).all()
    m, v = gpu.adamw_moments(net.list)
    m, v = host(m[0]), host(v[0])
    assert not m[:256].any() and not v[:256].any()
    assert np.allclose(m[256:512], 0.025, rtol=1e-6) and np.allclose(v[256:512], 0.0625e-3, rtol=1e-6)
    assert not np.delete(m[512:768], 88).any() and m[600] < 0 and (v[768:] >= 0).all()


def test_values_of_uneven_runs(gpu):
    # every value of a run's moments after a first step: one gradient alone, gradients of one size,
    # and gradients whose squares are below float32's smallest value
    net = Net(gpu, [1024], 8, 7, zeros=True)
    g = np.zeros(1024, np.float32)
    g[256:512], g[600], g[768:] = 0.25, -3.0, 1e-30
    net.G[0].copy_(dev(g))
    gpu.adamw(net.list, 1, LR)
    m, v = (host(t[0]).astype(np.float64) for t in gpu.adamw_moments(net.list))
    g = g.astype(np.float64)
    # the largest value of a run has the largest code: the scale's rounding and that of the value
    # read back, in v's scale twice (it is squared), and of the maximum in float32
    want_m, want_v = 0.1 * g, 0.001 * g * g
    want_v[768:] = 0.0
    assert np.all(np.abs(m - want_m) <= 3 * R.U * np.abs(want_m))
    assert np.all(np.abs(v - want_v) <= 4 * R.U * want_v)


def test_long_read_back(gpu):
    # more than 2048 x 1024 elements: every workgroup reads several pieces; ragged tensors
    rng = np.random.default_rng(25)
    sizes = [2_400_003, 1, 1_000_257]
    f = lambda a: [dev(t) for t in a]  # noqa: E731
    m = [rng.integers(-127, 128, n).astype(np.int8) for n in sizes]
    v = [rng.integers(0, 256, n).astype(np.uint8) for n in sizes]
    ms, vs = ([rng.uniform(1e-9, 1e-3, (n + 255) // 256).astype(np.float32) for n in sizes]
              for _ in range(2))
    p, g = ([torch.zeros(n, device="cuda") for n in sizes] for _ in range(2))
    net = gpu.Params(p, g, f(m), f(v), m_scale=f(ms), v_scale=f(vs))
    for i, got in enumerate(zip(*gpu.adamw_moments(net))):
        for a, r in zip(got, R.decode(m[i], v[i], ms[i], vs[i])):
            assert np.array_equal(host(a), r.astype(np.float32)), i


def test_moments_read_back(gpu):
    net = Net(gpu, [1, 300, 70001], 8, 8)
    for i, (m, v) in enumerate(zip(*gpu.adamw_moments(net.list))):
        rm, rv = net.values(i)
        assert np.array_equal(host(m), rm.astype(np.float32))
        assert np.array_equal(host(v), rv.astype(np.float32))


def test_moments_read_back_with_empty_tensors(gpu):
    # a list as adamw_state makes it, first, middle and last tensor empty
    net = Net(gpu, [0, 300, 0, 257, 0], 8, 22)
    gpu.adamw(net.list, 3, LR)
    net.m, net.v, net.ms, net.vs = ([host(x) for x in c] for c in (net.M, net.V, net.MS, net.VS))
    for i, (m, v) in enumerate(zip(*gpu.adamw_moments(net.list))):
        rm, rv = net.values(i)
        assert np.array_equal(host(m), rm.astype(np.float32))
        assert np.array_equal(host(v), rv.astype(np.float32))
    state = gpu.adamw_state(net.P, 8)
    fresh = gpu.Params(net.P, net.G, state[0], state[1], m_scale=state[2], v_scale=state[3])
    assert [m.numel() for m in gpu.adamw_moments(fresh)[0]] == [0, 300, 0, 257, 0]
    assert not any(t.any() for c in gpu.adamw_moments(fresh) for t in c)


@pytest.mark.parametrize("bits", [32, 8])
def test_any_element_alignment(gpu, bits):
    # tensors packed end to end in one buffer each, behind one element
    sizes = [5, 1000, 3, 257, 4099]
    ref = Net(gpu, sizes, bits, 9, grad="bf16", copies=True)
    total = sum(sizes) + 2

    def packed(ts):
        room = torch.full((total,), 7, device="cuda", dtype=ts[0].dtype)
        at, out = 1, []
        for t in ts:
            room[at:at + t.numel()] = t
            out.append(room[at:at + t.numel()])
            at += t.numel()
        return room, out

    rooms, cols = zip(*(packed(c) for c in (ref.P, ref.G, ref.M, ref.V, ref.C)))
    ms, vs = ([t.clone() if t is not None else None for t in c] for c in (ref.MS, ref.VS))
    got = gpu.Params(cols[0], cols[1], cols[2], cols[3], m_scale=ms, v_scale=vs, copies=cols[4],
                     weight_decay=ref.decay)
    gpu.adamw(got, 3, LR)
    gpu.adamw(ref.list, 3, LR)
    for mine, theirs in zip(cols, (ref.P, ref.G, ref.M, ref.V, ref.C)):
        assert all(torch.equal(a, b) for a, b in zip(mine, theirs))
    assert all(room[0] == 7 and room[-1] == 7 for room in rooms)


def test_not_finite(gpu):
    # 32 bits: the element alone; 8 bits: its run reads back as NaN, the others stay
    for bits in (32, 8):
        net, ref = (Net(gpu, [1024], bits, 10) for _ in range(2))
        net.G[0][300], net.G[0][301] = float("inf"), float("nan")
        gpu.adamw(net.list, 2, LR)
        gpu.adamw(ref.list, 2, LR)
        p, q = host(net.P[0]), host(ref.P[0])
        rest = np.delete(np.arange(1024), [300, 301])
        assert np.array_equal(p[rest], q[rest]) and not np.isfinite(p[301])
        if bits == 8:
            m, _ = gpu.adamw_moments(net.list)
            m = host(m[0])
            assert np.isnan(m[256:512]).all()
            assert np.isfinite(np.delete(m, np.arange(256, 512))).all()


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[1], [255, 3], [16384, 16385, 1], [3_000_001, 70000] + [17] * 60,
                                   [n % 977 for n in range(1, 4000, 9)]])
def test_grad_norm(gpu, sizes, grad):
    rng = np.random.default_rng(len(sizes))
    g = [(rng.standard_normal(n) * 0.1).astype(np.float32) for n in sizes]
    if grad == "bf16":
        g = [S.round_bf16(a) for a in g]
    norm = np.sqrt(sum(float((a.astype(np.float64) ** 2).sum()) for a in g))
    for top in (0.5 * norm, 2 * norm, float("inf")):
        out = host(gpu.grad_norm(gpu.Params(grads=[dev(a, grad) for a in g]), max_norm=top))
        f = min(1.0, top / (norm + 1e-6))
        # one rounding each, and 64-bit sums
        assert abs(out[0] - norm) <= 1.001 * R.U * norm and abs(out[1] - f) <= 1.001 * R.U * f


def test_grad_norm_range_and_empty(gpu):
    big = torch.full((1000,), 1e30, device="cuda")
    out = host(gpu.grad_norm(gpu.Params(grads=[big]), max_norm=1.0))
    assert abs(out[0] - np.sqrt(1000) * 1e30) <= 1e24 and 0 < out[1] < 1e-30
    for bad in (float("inf"), float("nan")):
        big[7] = bad
        out = host(gpu.grad_norm(gpu.Params(grads=[big]), max_norm=1.0))
        assert not np.isfinite(out[0]) and np.isnan(out[1])
    assert host(gpu.grad_norm(gpu.Params(grads=[]), max_norm=1.0)).tolist() == [0.0, 1.0]
    e = torch.empty(0, device="cuda")
    assert host(gpu.grad_norm(gpu.Params(grads=[e, e]), max_norm=1.0)).tolist() == [0.0, 1.0]


@pytest.mark.parametrize("bits", [32, 8])
def test_scale_and_skip(gpu, bits):
    net = Net(gpu, [5000, 70], bits, 11)
    norm = gpu.grad_norm(net.list, max_norm=0.5)
    f = float(host(norm)[1])
    assert f < 1.0
    gpu.adamw(net.list, 4, LR, grad_scale=norm[1:], flags=gpu.E3_ADAMW_SKIP_NONFINITE)
    net.check(gpu, 4, scale=f)
    kept = [t.clone() for t in net.P + net.M + net.V]
    bad = torch.full((1,), float("nan"), device="cuda")
    gpu.adamw(net.list, 5, LR, grad_scale=bad, flags=gpu.E3_ADAMW_SKIP_NONFINITE)
    assert all(torch.equal(a, b) for a, b in zip(kept, net.P + net.M + net.V))


def test_skip_leaves_the_scales(gpu):
    # larger gradients than before: a step would change the scales of every run, a skipped one none
    net = Net(gpu, [5000, 70, 0], 8, 24)
    for g in net.G:
        g.mul_(1e3)
    every = [t for c in (net.P, net.M, net.V, net.MS, net.VS) for t in c]
    kept = [t.clone() for t in every]
    for bad in (float("nan"), float("inf"), float("-inf")):
        scale = torch.full((1,), bad, device="cuda")
        gpu.adamw(net.list, 5, LR, grad_scale=scale, flags=gpu.E3_ADAMW_SKIP_NONFINITE)
        assert all(torch.equal(a, b) for a, b in zip(kept, every))
    gpu.adamw(net.list, 5, LR, grad_scale=torch.ones(1, device="cuda"),
              flags=gpu.E3_ADAMW_SKIP_NONFINITE)
    for scales, before in ((net.MS, kept[9:12]), (net.VS, kept[12:15])):
        assert all((a != b).all() for a, b in zip(scales, before))


@pytest.mark.parametrize("bits", [32, 8])
def test_step_and_lr_on_the_device(gpu, bits):
    a, b = (Net(gpu, [3000, 12], bits, 12) for _ in range(2))
    t = torch.zeros(1, device="cuda", dtype=torch.int64)
    lr = torch.full((1,), LR, device="cuda")
    for k in (1, 2, 3):
        t.add_(1)
        gpu.adamw(a.list, t, lr)
        gpu.adamw(b.list, k, float(np.float32(LR)))
        for x, y in zip(a.P + a.M + a.V, b.P + b.M + b.V):
            # the powers of the betas are formed by other products: the factors differ by a step
            assert torch.allclose(x.float(), y.float(), rtol=1e-6, atol=1e-9)


def test_lists_refused(gpu):
    net = Net(gpu, [300, 20], 8, 13)
    good = dict(params=net.P, grads=net.G, m=net.M, v=net.V, m_scale=net.MS, v_scale=net.VS)
    half = lambda ts: [t.to(torch.float16) for t in ts]  # noqa: E731
    wide = torch.zeros((300, 2), device="cuda")[:, 0]
    for over, error, text in (
            (dict(grads=net.G[:1]), ValueError, "params has 2"),
            (dict(grads=half(net.G)), TypeError, "dtype"),
            (dict(params=half(net.P)), TypeError, r"params\[0\]"),
            (dict(params=[net.P[0][:299], net.P[1]]), ValueError, r"params\[0\]"),
            (dict(grads=[wide, net.G[1]]), ValueError, "contiguous"),
            (dict(m=[net.M[0], net.M[1].float()]), TypeError, r"m\[1\]"),
            (dict(v=[net.V[0][:299], net.V[1]]), ValueError, r"v\[0\]"),
            (dict(m_scale=[net.MS[0], None]), ValueError, r"m_scale\[1\]"),
            (dict(v_scale=[net.VS[0][:1], net.VS[1]]), ValueError, r"v_scale\[0\]"),
            (dict(copies=[net.P[0], None]), TypeError, r"copies\[0\]"),
            (dict(weight_decay=[0.1]), ValueError, "weight_decay"),
            (dict(v=[net.M[0].view(torch.uint8), net.V[1]]), gpu.E3Error, "overlaps"),
            (dict(params=[net.P[0], net.P[0][:20]]), gpu.E3Error, "overlaps")):
        with pytest.raises(error, match=text):
            gpu.Params(**{**good, **over})
    # new gradients that overlap a parameter are refused, and the list works on with the old ones
    with pytest.raises(gpu.E3Error, match="overlaps"):
        net.list.set_grads([net.P[0], net.G[1]])
    with pytest.raises(ValueError):
        net.list.set_grads(net.G[:1])
    gpu.adamw(net.list, 1, LR)
    net.check(gpu, 1)
    only = gpu.Params(grads=net.G)
    for call in (lambda: gpu.adamw(only, 1, LR), lambda: gpu.adamw_moments(only),
                 lambda: gpu.adamw_moments(net.list, [net.P[0]], [net.P[1]]),
                 lambda: gpu.adamw_moments(net.list, net.P, [net.P[0], net.P[0]]),
                 lambda: gpu.adamw(net.list, 1, LR, grad_scale=torch.ones(2, device="cuda")),
                 lambda: gpu.adamw(net.list, 1, torch.ones(1)),
                 lambda: gpu.grad_norm(only, out=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gpu.adamw(net.list, torch.ones(1, device="cuda"), LR),
                 lambda: gpu.grad_norm(only, out=torch.zeros(2, device="cuda", dtype=torch.float64))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(gpu.E3Error, match="codes"):
        gpu.adamw_moments(Net(gpu, [5], 32, 1).list)


def test_new_gradients_each_step(gpu):
    # gradients that autograd allocates anew, a bf16 one among float32 ones
    net = Net(gpu, [300, 20], [8, 32], 14)
    for t in (1, 2):
        net.G = [torch.randn(300, device="cuda"), torch.randn(20, device="cuda").bfloat16()]
        net.g = [host(g) for g in net.G]
        net.p, net.m, net.v = ([host(x) for x in c] for c in (net.P, net.M, net.V))
        net.ms, net.vs = ([None if x is None else host(x) for x in c] for c in (net.MS, net.VS))
        net.list.set_grads(net.G)
        gpu.adamw(net.list, t, LR)
        net.check(gpu, t)


def test_new_gradients_without_one_are_refused(gpu):
    # the list works on with the gradients it had
    net = Net(gpu, [300, 20], [8, 32], 23)
    with pytest.raises(ValueError, match=r"grads\[1\] is required"):
        net.list.set_grads([torch.ones(300, device="cuda"), None])
    gpu.adamw(net.list, 2, LR)
    net.check(gpu, 2)
    only = gpu.Params(grads=net.G)
    with pytest.raises(ValueError, match=r"grads\[0\] is required"):
        only.set_grads([None, net.G[1]])


def test_long_tensor(gpu):
    # past 2^31 elements: the ends against the same values in a short list
    n, k = 2 ** 31 + 515, 1027
    G = torch.empty(n, device="cuda", dtype=torch.bfloat16)
    G.normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    P = torch.zeros(n, device="cuda")
    m, v, ms, vs = gpu.adamw_state([P], 8)
    gpu.adamw(gpu.Params([P], [G], m, v, m_scale=ms, v_scale=vs), 1, LR)
    tail = n - n % 256 - 1024
    for lo, hi in ((0, k), (tail, n)):
        p, g = torch.zeros(hi - lo, device="cuda"), G[lo:hi].clone()
        sm, sv, sms, svs = gpu.adamw_state([p], 8)
        gpu.adamw(gpu.Params([p], [g], sm, sv, m_scale=sms, v_scale=svs), 1, LR)
        whole = (hi - lo) // 256 * 256 if hi != n else hi - lo
        assert torch.equal(p, P[lo:hi])
        assert torch.equal(sm[0][:whole], m[0][lo:lo + whole])
        assert torch.equal(sv[0][:whole], v[0][lo:lo + whole])
    out = host(gpu.grad_norm(gpu.Params(grads=[G])))
    assert abs(out[0] - np.sqrt(n)) <= 1e-3 * np.sqrt(n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_a_long_tensor(gpu, dtype):
    # past 2^31 elements: 64-bit sums of slices of the same values; a lost slice of 65536 would be
    # 3e-5 / 2 of the norm, the bound is float32's rounding of it
    n = 2 ** 31 + 515 if dtype == "bf16" else 2 ** 28 + 515
    G = torch.empty(n, device="cuda", dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    G.normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    total = sum(float(G[i:i + 2 ** 27].double().square().sum()) for i in range(0, n, 2 ** 27))
    out = host(gpu.grad_norm(gpu.Params(grads=[G])))
    assert abs(out[0] - np.sqrt(total)) <= 1.001 * R.U * np.sqrt(total)


def _training(gpu, seed):
    """A network's last layer as it would be trained: mixing, normalisation,
    their gradients, the clipped update with mixed moments."""
    rng = np.random.default_rng(seed)
    irreps = S.parse_irreps("0e+1o+2e")[1]
    rows, C = 500, 64
    f = lambda *s: dev(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    s = {"x": f(rows, 9, C), "dy": f(rows, 9, C), "W": f(3, C, C) / 8, "w": 1 + f(3, C) / 10,
         "b": f(1, C) / 10, "t": torch.zeros(1, device="cuda", dtype=torch.int64)}
    dW, dw, db = (torch.zeros_like(s[k]) for k in ("W", "w", "b"))
    m, v, ms, vs = gpu.adamw_state([s["W"], s["w"], s["b"]], [8, 32, 32])
    params = gpu.Params([s["W"], s["w"], s["b"]], [dW, dw, db], m, v, m_scale=ms, v_scale=vs,
                        weight_decay=[0.01, 0.0, 0.0])
    keep = {"h": torch.empty_like(s["x"]), "y": torch.empty_like(s["x"]),
            "dh": torch.empty_like(s["x"]), "dx": torch.empty_like(s["x"]),
            "norm": torch.empty(2, device="cuda"),
            "nws": torch.empty(params.workspace_bytes, device="cuda", dtype=torch.uint8),
            "ws": torch.empty(gpu.layer_norm_workspace_size(irreps, rows, C), device="cuda",
                              dtype=torch.uint8)}

    def step():
        gpu.linear(irreps, irreps, s["x"], s["W"], out=keep["h"])
        gpu.layer_norm(irreps, keep["h"], s["w"], s["b"], out=keep["y"])
        d = s["dy"] + keep["y"]  # the cotangent of a loss <dy, y> + |y|^2 / 2
        gpu.layer_norm_backward(irreps, keep["h"], s["w"], d, dx=keep["dh"], dweight=dw, dbias=db,
                                workspace=keep["ws"])
        gpu.linear_backward(irreps, irreps, s["x"], s["W"], keep["dh"], dx=keep["dx"], dW=dW)
        gpu.grad_norm(params, max_norm=1.0, out=keep["norm"], workspace=keep["nws"])
        s["t"].add_(1)
        gpu.adamw(params, s["t"], 1e-2, grad_scale=keep["norm"][1:])

    return step, [s["W"], s["w"], s["b"], *m, *v, keep["y"], keep["dx"], keep["norm"]]


def test_training_steps_captured_and_eager(gpu):
    # two captured runs of the same operators, each with its own buffers, replayed in turn with
    # eager steps of a third between them: all three stay equal, bit for bit
    runs = [_training(gpu, 20) for _ in range(3)]
    graphs = []
    for step, _ in runs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    first = [t.clone() for t in runs[2][1]]
    for k in range(5):
        graphs[0].replay()
        runs[2][0]()
        graphs[1].replay()
        torch.cuda.synchronize()
        for a, b, c in zip(*(r[1] for r in runs)):
            assert torch.equal(a, b) and torch.equal(a, c), k
    assert not torch.equal(first[0], runs[2][1][0])
    assert all(torch.isfinite(t.float()).all() for t in runs[0][1])


def test_training_gradients_against_differences(gpu):
    # d loss / d W and d weight through normalisation and mixing, against central differences of
    # the 64-bit network
    from oracle import oracle as O
    rng = np.random.default_rng(21)
    irreps, rows, C = S.parse_irreps("0e+1o")[1], 40, 32
    x = rng.standard_normal((rows, 4, C)).astype(np.float32)
    dy = rng.standard_normal((rows, 4, C)).astype(np.float32)
    W = (rng.standard_normal((2, C, C)) / 6).astype(np.float32)
    w, b = (np.ones((k, C), np.float32) for k in (2, 1))
    h = gpu.linear(irreps, irreps, dev(x), dev(W))
    dh, dw, _ = gpu.layer_norm_backward(irreps, h, dev(w), dev(dy))
    _, dW = gpu.linear_backward(irreps, irreps, dev(x), dev(W), dh)

    def loss(W, w):
        h = np.concatenate([x[:, :1].astype(np.float64) @ W[0], x[:, 1:].astype(np.float64) @ W[1]], 1)
        return float((R.norm_forward(irreps, h, w, b, 1e-5)[0] * dy).sum())

    assert O.linear_num_weights(irreps, irreps) == 2
    args, e = [W.astype(np.float64), w.astype(np.float64)], 1e-5
    for at, grad in ((0, dW), (1, dw)):
        d = rng.standard_normal(args[at].shape)
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + e * d, args[at] - e * d
        g = host(grad).astype(np.float64) * d
        assert abs((loss(*up) - loss(*down)) / (2 * e) - g.sum()) <= 1e-5 * np.abs(g).sum()
