"""CPU checks of the normalisation's and the optimizer's entry points: what
they refuse, with which status, before any GPU work; workspace sizes; the
64-bit forms the GPU tests compare with, against differences."""
import ctypes as C

import numpy as np
import pytest

from clebsch_gordan_tensor_amd import api
from clebsch_gordan_tensor_amd import synth as S
from tests import norm_reference as R

INVALID, IRREPS, UNSUPPORTED, ALIGNMENT, WORKSPACE = -1, -2, -3, -4, -6
AT = 1 << 20  # a fake, aligned device address: never read


@pytest.fixture(scope="module")
def lib():
    return api.lib()


def _irreps(s, mul):
    return api._irreps_struct(S.parse_irreps(s)[1], mul)


def _forward(lib, ir="0e+1o", mul=8, rows=4, x=AT, w=AT, b=AT, eps=1e-5, flags=0, y=AT * 2,
             dtype=0):
    st = _irreps(ir, mul) if isinstance(ir, str) else ir
    return lib.e3_layer_norm(C.byref(st) if st is not None else None, rows, x, w, b, eps, flags, y,
                             dtype, None)


def _backward(lib, ir="0e+1o", mul=8, rows=4, x=AT, w=AT, dy=AT * 2, eps=1e-5, flags=0, dx=AT * 3,
              dw=AT * 4, db=AT * 5, ws=AT * 6, nb=1 << 20, dtype=0):
    st = _irreps(ir, mul)
    return lib.e3_layer_norm_backward(C.byref(st), rows, x, w, dy, eps, flags, dx, dw, db, ws, nb,
                                      dtype, None)


def test_layer_norm_refusals(lib):
    mixed = api._Irreps(2, (api._Irrep * 2)(api._Irrep(4, 0, 1), api._Irrep(8, 1, -1)))
    for call, status in ((dict(ir=None), INVALID), (dict(rows=-1), INVALID), (dict(x=None), INVALID),
                         (dict(y=None), INVALID), (dict(eps=0.0), INVALID),
                         (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(eps=1e-40), INVALID),
                         (dict(flags=2), INVALID), (dict(dtype=7), INVALID), (dict(ir=mixed), IRREPS),
                         (dict(ir=api._Irreps(0, None)), IRREPS), (dict(ir="9e"), UNSUPPORTED),
                         (dict(mul=4097), UNSUPPORTED), (dict(ir="4e", mul=1025), UNSUPPORTED),
                         (dict(ir=api._Irreps(1025, None)), UNSUPPORTED),
                         (dict(rows=1 << 60), UNSUPPORTED), (dict(x=AT + 2), ALIGNMENT),
                         (dict(y=AT + 1, dtype=1), ALIGNMENT), (dict(w=AT + 1), ALIGNMENT),
                         (dict(b=AT + 2), ALIGNMENT), (dict(y=AT + 4), INVALID),
                         (dict(y=AT - 4), INVALID), (dict(rows=0, x=None, y=None), 0)):
        assert _forward(lib, **call) == status, call
        assert (status == 0) == (lib.e3_last_error() == b""), call


def test_layer_norm_backward_refusals(lib):
    for call, status in ((dict(rows=-1), INVALID), (dict(x=None), INVALID), (dict(dy=None), INVALID),
                         (dict(dx=None), INVALID), (dict(eps=-1.0), INVALID),
                         (dict(flags=8), INVALID), (dict(dtype=2), INVALID),
                         (dict(mul=5000), UNSUPPORTED), (dict(ws=None), WORKSPACE),
                         (dict(nb=8), WORKSPACE), (dict(ws=AT + 8), ALIGNMENT),
                         (dict(dy=AT * 2 + 2), ALIGNMENT), (dict(dx=AT * 3 + 1), ALIGNMENT),
                         (dict(dw=AT + 2), ALIGNMENT), (dict(db=AT + 2), ALIGNMENT),
                         (dict(dx=AT + 4), INVALID), (dict(dx=AT * 2 - 4), INVALID)):
        assert _backward(lib, **call) == status, call


def test_layer_norm_workspace(lib):
    nb = C.c_size_t()
    assert lib.e3_layer_norm_workspace_size(C.byref(_irreps("0e", 8)), 5, None) == INVALID
    assert lib.e3_layer_norm_workspace_size(C.byref(_irreps("0e", 5000)), 5, C.byref(nb)) == UNSUPPORTED
    last = 0
    for rows in (0, 1, 100, 10 ** 4, 10 ** 6, 10 ** 9):
        size = api.layer_norm_workspace_size([(0, 1), (1, -1)], rows, 128)
        assert last <= size <= 32 * 1024 * 128
        last = size


def _param(n=300, **over):
    d = dict(n=n, p=AT, grad=AT * 2, m=AT * 3, v=AT * 4, m_scale=None, v_scale=None, p_bf16=None,
             weight_decay=0.0, grad_dtype=0)
    d.update(over)
    return api._Param(**d)


def _list(*ps):
    return len(ps), (api._Param * max(1, len(ps)))(*ps)


@pytest.mark.parametrize("over,status", [
    (dict(), 0), (dict(n=0, p=None, grad=None, m=None, v=None), 0), (dict(n=-1), INVALID),
    (dict(n=(1 << 33) + 1), INVALID), (dict(grad_dtype=3), INVALID), (dict(p=None), INVALID),
    (dict(grad=None), INVALID), (dict(m=None), INVALID), (dict(v=None), INVALID),
    (dict(m_scale=AT * 5), INVALID), (dict(v_scale=AT * 5), INVALID),
    (dict(weight_decay=float("nan")), INVALID), (dict(p=AT + 2), ALIGNMENT),
    (dict(grad=AT * 2 + 2), ALIGNMENT), (dict(grad=AT * 2 + 2, grad_dtype=1), 0),
    (dict(grad=AT * 2 + 1, grad_dtype=1), ALIGNMENT), (dict(m=AT * 3 + 2), ALIGNMENT),
    (dict(m=AT * 3 + 1, v=AT * 4 + 3, m_scale=AT * 5, v_scale=AT * 6), 0),
    (dict(m_scale=AT * 5 + 2, v_scale=AT * 6), ALIGNMENT), (dict(p_bf16=AT * 7 + 1), ALIGNMENT),
    (dict(v=AT * 3), INVALID), (dict(grad=AT + 1196), INVALID), (dict(grad=AT + 1200), 0),
    (dict(p_bf16=AT * 2 - 4), INVALID), (dict(m_scale=AT * 5, v_scale=AT * 5 + 4), INVALID),
    (dict(m_scale=AT * 5, v_scale=AT * 5 + 8), 0),
])
def test_tensor_checks(lib, over, status):
    n, arr = _list(_param(**over))
    assert lib.e3_param_check(n, arr) == status, lib.e3_last_error()


def test_overlap_between_tensors(lib):
    far = dict(p=1 << 40, grad=1 << 41, m=1 << 42, v=1 << 43)
    assert lib.e3_param_check(*_list(_param(), _param(**far))) == 0
    assert lib.e3_param_check(*_list(_param(), _param(**{**far, "grad": AT * 2}))) == 0  # both read
    for over in (dict(p=AT), dict(m=AT * 4), dict(grad=AT + 400), dict(v=AT * 2)):
        assert lib.e3_param_check(*_list(_param(), _param(**{**far, **over}))) == INVALID, over
        assert b"tensor" in lib.e3_last_error()
    assert lib.e3_param_check(-1, None) == INVALID and lib.e3_param_check(1, None) == INVALID
    assert lib.e3_param_check(0, None) == 0 and lib.e3_param_check(70000, arr_of(1)) == UNSUPPORTED


def arr_of(n):
    return (api._Param * n)(*[_param() for _ in range(n)])


def test_grad_norm_refusals(lib):
    nb = C.c_size_t()
    n, arr = _list(_param(n=5000))
    assert lib.e3_grad_norm_workspace_size(n, arr, C.byref(nb)) == 0 and nb.value == 5 * 8
    assert lib.e3_grad_norm_workspace_size(n, arr, None) == INVALID
    assert lib.e3_grad_norm_workspace_size(0, None, C.byref(nb)) == 0 and nb.value == 8
    f = lambda top=1.0, out=AT, ws=AT * 2, b=40: lib.e3_grad_norm(n, arr, top, out, ws, b, None)  # noqa: E731
    for call, status in ((dict(top=0.0), INVALID), (dict(top=float("nan")), INVALID),
                         (dict(out=None), INVALID), (dict(ws=None), WORKSPACE), (dict(b=39), WORKSPACE),
                         (dict(ws=AT + 4), ALIGNMENT), (dict(out=AT + 2), ALIGNMENT)):
        assert f(**call) == status, call
    bad = _list(_param(grad=None))
    assert lib.e3_grad_norm(*bad, 1.0, AT, AT, 1 << 20, None) == INVALID


@pytest.mark.parametrize("over", [
    dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.5), dict(beta2=float("nan")), dict(eps=0.0),
    dict(eps=1e-60), dict(eps=1e-40), dict(eps=float("inf")), dict(lr=float("nan")), dict(step=0), dict(flags=2),
    dict(flags=1),
])
def test_adamw_refusals(lib, over):
    n, arr = _list(_param())
    a = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, step_dev=None, lr_dev=None,
             grad_scale=None, flags=0)
    assert lib.e3_adamw(n, arr, C.byref(api._AdamwArgs(**{**a, **over})), None) == INVALID
    assert lib.e3_adamw(n, arr, None, None) == INVALID
    for name, at in (("step_dev", AT + 4), ("lr_dev", AT + 2), ("grad_scale", AT + 2)):
        assert lib.e3_adamw(n, arr, C.byref(api._AdamwArgs(**{**a, name: at})), None) == ALIGNMENT
    assert lib.e3_adamw(0, None, C.byref(api._AdamwArgs(**a)), None) == 0


def test_adamw_moments_refusals(lib):
    out = (C.c_void_p * 1)(AT * 8)
    odd, none = (C.c_void_p * 1)(AT * 8 + 2), (C.c_void_p * 1)(None)
    n, arr = _list(_param(m_scale=AT * 5, v_scale=AT * 6))
    assert lib.e3_adamw_moments(n, arr, None, out, None) == INVALID
    assert lib.e3_adamw_moments(n, arr, out, none, None) == INVALID
    assert lib.e3_adamw_moments(n, arr, odd, out, None) == ALIGNMENT
    assert lib.e3_adamw_moments(*_list(_param()), out, out, None) == INVALID
    assert lib.e3_adamw_moments(0, None, None, None, None) == 0


def test_empty_tensors_have_no_moments_to_read(lib):
    # zero-length scales have no address: an empty tensor is left out, whatever its moments were
    empty = dict(n=0, p=None, grad=None, m=None, v=None)
    none = (C.c_void_p * 2)(None, None)
    assert lib.e3_adamw_moments(*_list(_param(**empty), _param(**empty)), none, none, None) == 0
    out = (C.c_void_p * 2)(None, AT * 8)
    assert lib.e3_adamw_moments(*_list(_param(**empty), _param()), out, out, None) == INVALID
    assert b"tensor 1" in lib.e3_last_error()


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((3, 4, 8))
    with pytest.raises(ValueError, match="GPU"):
        api.layer_norm([(0, 1), (1, -1)], x)
    with pytest.raises(ValueError, match="GPU"):
        api.layer_norm_backward([(0, 1), (1, -1)], x, None, x)
    with pytest.raises(ValueError, match="GPU"):
        api.Params(grads=[torch.zeros(3)])
    with pytest.raises(ValueError, match="required"):
        api.Params(params=[x], grads=[x])
    with pytest.raises(ValueError, match="grads"):
        api.Params(params=[x], grads=[], m=[x], v=[x])
    with pytest.raises(ValueError, match="bits"):
        api.adamw_state([x], 16)


def test_a_parameter_without_a_gradient_is_named():
    torch = pytest.importorskip("torch")
    g = torch.zeros(3)
    for grads, error, text in (([None], ValueError, r"grads\[0\] is required"),
                               ([g, None], ValueError, r"grads\[1\] is required"),
                               ([g, 2.0], TypeError, r"grads\[1\] must be a tensor")):
        with pytest.raises(error, match=text):
            api.Params(grads=grads)
        with pytest.raises(error, match=text):
            api.Params(params=[g] * len(grads), grads=grads, m=[g] * len(grads), v=[g] * len(grads))


# --------------------------------------------------- the 64-bit forms themselves

def test_norm_gradients_against_differences():
    rng = np.random.default_rng(0)
    irreps = S.parse_irreps("0e+1o+0o+2e")[1]
    x, dy = rng.standard_normal((2, 7, 10, 6))
    w, b = rng.standard_normal((4, 6)), rng.standard_normal((1, 6))
    for centered in (True, False):
        f = lambda x, w, b: float((R.norm_forward(irreps, x, w, b, 1e-3, centered)[0] * dy).sum())  # noqa: E731
        grads, _ = R.norm_backward(irreps, x, w, dy, 1e-3, centered)
        for at, g in enumerate(grads):
            d = rng.standard_normal(g.shape)
            up, down = [x, w, b], [x, w, b]
            up[at], down[at] = up[at] + 1e-5 * d, down[at] - 1e-5 * d
            assert abs((f(*up) - f(*down)) / 2e-5 - (g * d).sum()) <= 1e-7 * np.abs(g * d).sum()


@pytest.mark.parametrize("case", R.LONG_SUMS, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}")
def test_bounds_of_long_sums_see_a_lost_row(case):
    # a sum over rows that misses one row, or all of them, is outside the bound it is held to
    ir, C, dtype, rows, lane, depth = case
    irreps = S.parse_irreps(ir)[1]
    dw, db = R.long_sums(irreps, *R.long_case(irreps, C, dtype, rows), 1e-5, lane, depth)
    for sums in (dw, db):
        total, tol = (np.concatenate([s[k] for s in sums]) for k in (1, 2))
        assert np.mean(np.abs(total) > tol) >= 0.9
        for row in (0, rows // 2, rows - 1):
            lost = np.concatenate([s[0][row] for s in sums])
            seen = np.mean(np.abs(lost) > tol)
            print(f"{ir} C {C}: row {row} seen in {seen:.2f} of {lost.size} sums")
            assert seen > 0


def test_norm_is_equivariant():
    # rotating the components of every block rotates the result; so does the inversion
    from tests.test_oracle_cg import _rand_rot, wigner_d  # fitted from scipy's harmonics
    rng = np.random.default_rng(1)
    irreps = S.parse_irreps("0e+1o+2e")[1]
    x = rng.standard_normal((5, 9, 4))
    w, b = rng.standard_normal((3, 4)), rng.standard_normal((1, 4))
    y = R.norm_forward(irreps, x, w, b, 1e-5)[0]
    rot = _rand_rot(rng)
    D = [wigner_d(l, rot, rng) for l, _ in irreps]
    for mats in (D, [p * np.eye(2 * l + 1) for l, p in irreps]):  # a rotation, the inversion
        turn = lambda t: np.concatenate([np.einsum("ij,rjk->rik", M, t[:, a:a + n]) for M, (a, n, _)  # noqa: E731
                                         in zip(mats, R.blocks_of(irreps))], 1)
        assert np.allclose(R.norm_forward(irreps, turn(x), w, b, 1e-5)[0], turn(y), atol=1e-9)


def test_codes_of_moments():
    # a code is the nearest in the square (fourth) root: at most half a step from the value there
    rng = np.random.default_rng(2)
    m = rng.standard_normal(1000) * np.exp(2 * rng.standard_normal(1000))
    v = m ** 2
    ms, vs = R.scales(m, v)
    cm, _ = R.codes(np.abs(m), ms, 127, 1)
    cv, _ = R.codes(v, vs, 255, 2)
    s1, s2 = (np.repeat(s.astype(np.float64), 256)[:1000] for s in (ms, vs))
    assert np.all(np.abs(np.sqrt(np.abs(m) / s1) - cm) <= 0.5 + 1e-5)
    assert np.all(np.abs(np.sqrt(np.sqrt(v) / s2) - cv) <= 0.5 + 1e-5)
    assert cm.max() == 127 and cv.max() == 255
