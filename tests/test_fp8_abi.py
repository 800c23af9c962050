"""CPU checks of the residual normalisation's and the 8-bit operators' entry
points: what they refuse, with which status, before any GPU work; the 8-bit
forms that the GPU tests compare with, against torch's conversion."""
import ctypes as C

import numpy as np
import pytest

from clebsch_gordan_tensor_amd import api
from clebsch_gordan_tensor_amd import synth as S
from tests import grouped_reference as R

INVALID, IRREPS, UNSUPPORTED, ALIGNMENT, WORKSPACE = -1, -2, -3, -4, -6
AT = 1 << 24  # a fake, aligned device address: never read


@pytest.fixture(scope="module")
def lib():
    return api.lib()


def _irreps(s, mul):
    return api._irreps_struct(S.parse_irreps(s)[1], mul) if isinstance(s, str) else s


def _refuses(lib, call, cases):
    for args, status in cases:
        assert call(lib, **args) == status, args
        assert (status == 0) == (lib.e3_last_error() == b""), args


def _residual(lib, ir="0e+1o", mul=8, rows=4, x=AT, r=AT * 2, w=AT * 3, b=AT * 4, eps=1e-5, flags=0,
              h=AT * 5, y=AT * 6, dtype=0):
    st = _irreps(ir, mul)
    return lib.e3_layer_norm_residual(C.byref(st) if st is not None else None, rows, x, r, w, b, eps,
                                      flags, h, y, dtype, None)


def test_residual_refusals(lib):
    _refuses(lib, _residual, [
        (dict(ir=None), INVALID), (dict(rows=-1), INVALID), (dict(x=None), INVALID),
        (dict(r=None), INVALID), (dict(h=None), INVALID), (dict(y=None), INVALID),
        (dict(eps=0.0), INVALID), (dict(flags=2), INVALID), (dict(dtype=7), INVALID),
        (dict(ir=api._Irreps(0, None)), IRREPS), (dict(ir="9e"), UNSUPPORTED),
        (dict(mul=4097), UNSUPPORTED), (dict(x=AT + 2), ALIGNMENT), (dict(r=AT * 2 + 1), ALIGNMENT),
        (dict(h=AT * 5 + 2), ALIGNMENT), (dict(y=AT * 6 + 3), ALIGNMENT), (dict(w=AT + 2), ALIGNMENT),
        (dict(h=AT + 4), INVALID), (dict(y=AT * 2 - 4), INVALID), (dict(h=AT * 6), INVALID),
        (dict(h=AT * 6 + 8), INVALID), (dict(rows=0, x=None, r=None, h=None, y=None), 0)])


def _residual_backward(lib, ir="0e+1o", mul=8, rows=4, h=AT, w=AT * 2, dy=AT * 3, dh=AT * 4,
                       eps=1e-5, flags=0, dx=AT * 5, dw=AT * 6, db=AT * 7, ws=AT * 8, nb=1 << 20,
                       dtype=0):
    return lib.e3_layer_norm_residual_backward(C.byref(_irreps(ir, mul)), rows, h, w, dy, dh, eps,
                                               flags, dx, dw, db, ws, nb, dtype, None)


def test_residual_backward_refusals(lib):
    _refuses(lib, _residual_backward, [
        (dict(rows=-1), INVALID), (dict(h=None), INVALID), (dict(dy=None), INVALID),
        (dict(dh=None), INVALID), (dict(dx=None), INVALID), (dict(eps=-1.0), INVALID),
        (dict(flags=8), INVALID), (dict(dtype=2), INVALID), (dict(mul=5000), UNSUPPORTED),
        (dict(ws=None), WORKSPACE), (dict(nb=8), WORKSPACE), (dict(ws=AT * 8 + 8), ALIGNMENT),
        (dict(dh=AT * 4 + 2), ALIGNMENT), (dict(dx=AT * 5 + 1), ALIGNMENT),
        (dict(dw=AT * 6 + 2), ALIGNMENT), (dict(dx=AT + 4), INVALID),
        (dict(dx=AT * 3 - 4), INVALID), (dict(dx=AT * 4 + 8), INVALID)])


def _norm_fp8(lib, ir="0e+1o", mul=16, rows=4, x=AT, r=AT * 2, w=AT * 3, b=AT * 4, eps=1e-5, flags=0,
              h=AT * 5, q=AT * 6, scale=AT * 7, dtype=0):
    return lib.e3_layer_norm_fp8(C.byref(_irreps(ir, mul)), rows, x, r, w, b, eps, flags, h, q,
                                 scale, dtype, None)


def test_norm_in_8_bits_refusals(lib):
    _refuses(lib, _norm_fp8, [
        (dict(mul=8), UNSUPPORTED), (dict(mul=24), UNSUPPORTED), (dict(mul=4112), UNSUPPORTED),
        (dict(rows=-1), INVALID), (dict(x=None), INVALID), (dict(q=None), INVALID),
        (dict(scale=None), INVALID), (dict(h=None), INVALID), (dict(r=None), INVALID),
        (dict(eps=0.0), INVALID), (dict(flags=4), INVALID), (dict(dtype=3), INVALID),
        (dict(x=AT + 1), ALIGNMENT), (dict(q=AT * 6 + 8), ALIGNMENT),
        (dict(scale=AT * 7 + 2), ALIGNMENT), (dict(h=AT + 4), INVALID), (dict(q=AT), INVALID),
        (dict(scale=AT * 2 + 64), INVALID), (dict(q=AT * 5 + 16), INVALID),
        (dict(scale=AT * 6 + 16), INVALID), (dict(rows=0, x=None, r=None, h=None, q=None), 0)])


def _quantize(lib, rows=4, ch=64, x=AT, q=AT * 2, scale=AT * 3, dtype=0):
    return lib.e3_quantize_fp8(rows, ch, x, q, scale, dtype, None)


def test_quantize_refusals(lib):
    _refuses(lib, _quantize, [
        (dict(rows=-1), INVALID), (dict(ch=0), INVALID), (dict(ch=-16), INVALID),
        (dict(ch=40), UNSUPPORTED), (dict(ch=8208), UNSUPPORTED), (dict(rows=1 << 60), UNSUPPORTED),
        (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID),
        (dict(dtype=4), INVALID), (dict(x=AT + 4), ALIGNMENT), (dict(q=AT + 4), ALIGNMENT),
        (dict(scale=AT * 3 + 1), ALIGNMENT), (dict(q=AT + 16), INVALID), (dict(scale=AT), INVALID),
        (dict(scale=AT * 2 + 16), INVALID), (dict(rows=0, x=None, q=None, scale=None), 0)])


def _pack(lib, into="0e+1o", out="1o+0e", cin=32, cout=48, groups=3, W=AT, packed=AT * 2, nb=1 << 20):
    return lib.e3_linear_fp8_pack(C.byref(_irreps(into, cin)), C.byref(_irreps(out, cout)), groups, W,
                                  packed, nb, None)


def test_pack_refusals(lib):
    _refuses(lib, _pack, [
        (dict(cin=8), UNSUPPORTED), (dict(cout=40), UNSUPPORTED), (dict(cin=8208), UNSUPPORTED),
        (dict(groups=0), INVALID), (dict(groups=1025), UNSUPPORTED), (dict(W=None), INVALID),
        (dict(packed=None), WORKSPACE), (dict(nb=100), WORKSPACE), (dict(W=AT + 4), ALIGNMENT),
        (dict(packed=AT * 2 + 4), ALIGNMENT), (dict(packed=AT + 64), INVALID),
        (dict(out="2e", W=None), 0)])
    nb = C.c_size_t()
    a, b = _irreps("0e+1o", 144), _irreps("0e+1o", 80)
    assert lib.e3_linear_fp8_pack_size(C.byref(a), C.byref(b), 3, C.byref(nb)) == 0
    assert nb.value == 64 + 64 + 3 * 2 * 80 * 256  # 12 scales in 64 bytes, codes to 256 of 144
    assert lib.e3_linear_fp8_pack_size(C.byref(a), C.byref(b), 3, None) == INVALID
    assert lib.e3_linear_fp8_pack_size(C.byref(a), C.byref(b), 0, C.byref(nb)) == INVALID


def _mix(lib, into="0e+1o", out="1o+0e", cin=32, cout=48, rows=10, groups=3, index=AT, ib=1 << 20,
         q=AT * 2, scale=AT * 3, packed=AT * 4, pb=1 << 20, y=AT * 5, dtype=1):
    return lib.e3_linear_fp8(C.byref(_irreps(into, cin)), C.byref(_irreps(out, cout)), rows, groups,
                             index, ib, q, scale, packed, pb, y, dtype, None)


def test_mixing_refusals(lib):
    _refuses(lib, _mix, [
        (dict(cin=24), UNSUPPORTED), (dict(cout=8), UNSUPPORTED), (dict(rows=-1), INVALID),
        (dict(rows=1 << 31), UNSUPPORTED), (dict(index=None), INVALID), (dict(ib=8), WORKSPACE),
        (dict(index=AT + 4), ALIGNMENT), (dict(q=None), INVALID), (dict(scale=None), INVALID),
        (dict(packed=None), WORKSPACE), (dict(pb=64), WORKSPACE), (dict(y=None), INVALID),
        (dict(q=AT * 2 + 4), ALIGNMENT), (dict(scale=AT * 3 + 2), ALIGNMENT),
        (dict(packed=AT * 4 + 8), ALIGNMENT), (dict(y=AT * 5 + 8), ALIGNMENT),
        (dict(dtype=2), INVALID), (dict(y=AT * 2), INVALID), (dict(y=AT * 3 - 16), INVALID),
        (dict(y=AT * 4 + 64), INVALID), (dict(y=AT), INVALID), (dict(groups=0), INVALID),
        (dict(rows=0, q=None, scale=None, y=None), 0)])


def test_e4m3_against_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.uniform(-4, 2, 20000),
                        np.linspace(-448, 448, 10001), np.exp2(np.arange(-14, 9)),
                        1.0625 * np.exp2(np.arange(-10.0, 8)), [0.0, 448.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    v = v[np.abs(v) <= 448].astype(np.float32)
    got = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(R.e4m3(v), got)


def test_quantised_values_are_near():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((50, 300)) * 10.0 ** rng.uniform(-3, 3, (50, 1))).astype(np.float32)
    q, s = R.quantize(x)
    step = np.maximum(2.0 ** -4 * np.abs(x), np.repeat(s, 128, -1)[:, :300] * 2.0 ** -10)
    assert np.all(np.abs(R.values(q, s) - x) <= step * (1 + 1e-6))
    W = rng.standard_normal((2, 3, 200, 130)).astype(np.float32)
    q, s = R.quantize_weights(W)
    assert s.shape == (2, 3, 2, 2)
    err = np.abs(R.weight_values(q, s) - W)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(W), s.max() * 2.0 ** -10) * (1 + 1e-6))


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 1, 16)  # on the CPU
    with pytest.raises(ValueError):
        api.quantize_fp8(x)
    with pytest.raises(ValueError):
        api.layer_norm_residual([(0, 1)], x, x)
    with pytest.raises(ValueError):
        api.layer_norm_fp8([(0, 1)], x)
    with pytest.raises(ValueError):
        api.linear_fp8_pack([(0, 1)], [(0, 1)], torch.zeros(1, 1, 16, 16))
    with pytest.raises(ValueError):
        api.linear_fp8([(0, 1)], [(0, 1)], x.to(torch.float8_e4m3fn), x, None)
