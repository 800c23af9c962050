"""CPU checks of the entry points on grouped rows: what they refuse, with which
status, before any GPU work, and the sizes of their memory."""
import ctypes as C

import numpy as np
import pytest

from clebsch_gordan_tensor_amd import api
from clebsch_gordan_tensor_amd import synth as S

INVALID, IRREPS, UNSUPPORTED, ALIGNMENT, WORKSPACE = -1, -2, -3, -4, -6
AT = 1 << 24  # a fake, aligned device address: never read
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return api.lib()


def _irreps(s, mul):
    return api._irreps_struct(S.parse_irreps(s)[1], mul)


def test_index_sizes(lib):
    b, off, order = C.c_size_t(), C.c_size_t(), C.c_size_t()
    last = 0
    for rows in (0, 1, 8192, 8193, 10 ** 6, 2 ** 31 - 1):
        for groups in (1, 7, 1024):
            assert lib.e3_group_index_size(rows, groups, C.byref(b)) == 0
            assert lib.e3_group_index_at(rows, groups, C.byref(off), C.byref(order)) == 0
            assert off.value >= 12 and order.value >= off.value + 4 * (groups + 1)
            assert order.value % 64 == 0 and b.value >= order.value + 4 * rows
        assert b.value >= last
        last = b.value
    for rows, groups, status in ((-1, 4, INVALID), (4, 0, INVALID), (4, -2, INVALID),
                                 (4, 1025, UNSUPPORTED), (2 ** 31, 4, UNSUPPORTED)):
        assert lib.e3_group_index_size(rows, groups, C.byref(b)) == status
        assert lib.e3_group_index_at(rows, groups, C.byref(off), C.byref(order)) == status
    assert lib.e3_group_index_size(4, 4, None) == INVALID
    assert lib.e3_group_index_at(4, 4, None, C.byref(order)) == INVALID


def _index(lib, rows=100, groups=4, group=AT, index=AT * 2, nb=1 << 20):
    return lib.e3_group_index(rows, groups, group, index, nb, None)


def test_index_refusals(lib):
    for call, status in ((dict(rows=-1), INVALID), (dict(groups=0), INVALID),
                         (dict(groups=1025), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
                         (dict(group=None), INVALID), (dict(index=None), INVALID),
                         (dict(index=None, groups=1), INVALID), (dict(nb=400), WORKSPACE),
                         (dict(group=AT + 2), ALIGNMENT), (dict(index=AT * 2 + 8), ALIGNMENT),
                         (dict(group=AT * 2 + 64), INVALID)):
        assert _index(lib, **call) == status, call
        assert lib.e3_last_error() != b""


def _forward(lib, into="0e+1o", out="1o+0e", cin=16, cout=24, rows=10, groups=3, index=AT,
             nb=1 << 20, x=AT * 2, W=AT * 3, y=AT * 4, dtype=0):
    a = _irreps(into, cin) if isinstance(into, str) else into
    b = _irreps(out, cout) if isinstance(out, str) else out
    return lib.e3_linear_grouped(C.byref(a) if a is not None else None,
                                 C.byref(b) if b is not None else None, rows, groups, index, nb, x,
                                 W, y, dtype, None)


def test_mixing_refusals(lib):
    mixed = api._Irreps(2, (api._Irrep * 2)(api._Irrep(8, 0, 1), api._Irrep(16, 1, -1)))
    for call, status in (
            (dict(into=None), INVALID), (dict(out=None), INVALID), (dict(into=mixed), IRREPS),
            (dict(out=api._Irreps(0, None)), IRREPS), (dict(cin=12), UNSUPPORTED),
            (dict(cout=4), UNSUPPORTED), (dict(cin=8200), UNSUPPORTED),
            (dict(into="9e", out="9e"), UNSUPPORTED), (dict(into="+".join(["0e"] * 33)), UNSUPPORTED),
            (dict(into="+".join(["0e"] * 20), out="+".join(["0e"] * 20)), UNSUPPORTED),
            (dict(rows=-1), INVALID), (dict(rows=1 << 31), UNSUPPORTED), (dict(groups=0), INVALID),
            (dict(groups=2000), UNSUPPORTED), (dict(index=None), INVALID), (dict(nb=64), WORKSPACE),
            (dict(index=AT + 4), ALIGNMENT), (dict(x=None), INVALID), (dict(W=None), INVALID),
            (dict(y=None), INVALID), (dict(x=AT * 2 + 4), ALIGNMENT), (dict(W=AT * 3 + 8), ALIGNMENT),
            (dict(y=AT * 4 + 2), ALIGNMENT), (dict(dtype=5), INVALID), (dict(y=AT * 2), INVALID),
            (dict(y=AT * 2 - 64), INVALID), (dict(y=AT * 3 + 16), INVALID), (dict(y=AT + 64), INVALID),
            (dict(rows=2 ** 31 - 1, nb=BIG, into="8e+8e+8e", out="8e"), UNSUPPORTED),
            (dict(rows=0, x=None, y=None, W=None), 0)):
        assert _forward(lib, **call) == status, call
        assert (status == 0) == (lib.e3_last_error() == b""), call


def _backward(lib, into="0e+1o", out="1o+0e", cin=64, cout=64, rows=20000, groups=3, index=AT,
              nb=BIG, x=BIG, W=BIG * 2, dy=BIG * 3, dx=BIG * 4, dW=BIG * 5, ws=BIG * 6, wb=BIG // 2,
              dtype=0):
    a, b = _irreps(into, cin), _irreps(out, cout)
    return lib.e3_linear_grouped_backward(C.byref(a), C.byref(b), rows, groups, index, nb, x, W, dy,
                                          dx, dW, ws, wb, dtype, None)


def test_mixing_backward_refusals(lib):
    for call, status in (
            (dict(cin=4), UNSUPPORTED), (dict(rows=-5), INVALID), (dict(groups=-1), INVALID),
            (dict(index=None), INVALID), (dict(nb=16), WORKSPACE), (dict(x=None), INVALID),
            (dict(dy=None), INVALID), (dict(W=None), INVALID), (dict(ws=None), WORKSPACE),
            (dict(wb=100), WORKSPACE), (dict(ws=BIG * 6 + 4), ALIGNMENT),
            (dict(x=BIG + 8), ALIGNMENT), (dict(dW=BIG * 5 + 4), ALIGNMENT),
            (dict(dx=BIG * 4 + 8), ALIGNMENT), (dict(dtype=9), INVALID), (dict(dx=BIG), INVALID),
            (dict(dx=BIG * 3 + 16), INVALID), (dict(dW=BIG * 2), INVALID), (dict(dW=BIG * 4), INVALID),
            (dict(ws=BIG * 5), INVALID), (dict(ws=BIG + 16), INVALID)):
        assert _backward(lib, nb=call.pop("nb", 1 << 20), **call) == status, call
        assert lib.e3_last_error() != b""


def test_workspace(lib):
    ir = [(0, 1), (1, -1), (2, 1), (3, -1)]
    last = 0
    for rows in (0, 10, 1000, 64000, 10 ** 6, 10 ** 8):
        n = api.linear_grouped_workspace_size(ir, ir, 128, 128, rows, 10)
        assert last <= n <= 256 << 20  # at most a few partials for each workgroup
        last = n
    assert api.linear_grouped_workspace_size([(0, 1)], [(0, 1)], 2048, 2048, 10 ** 6, 16) == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    # tensors on the CPU are refused before the library is called
    x, W = torch.zeros(4, 1, 8), torch.zeros(2, 1, 8, 8)
    with pytest.raises(ValueError):
        api.linear_grouped([(0, 1)], [(0, 1)], None, x, W)
    with pytest.raises(ValueError):
        api.group_rows(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(TypeError):
        api._index_args(torch.device("cuda", 0), torch.zeros(3), 4, 2)
    with pytest.raises(ValueError):
        api._index_args(torch.device("cuda", 0), api.RowGroups(torch.zeros(8), 4, 2), 5, 2)
    with pytest.raises(api.E3Error):
        api._index_sizes(4, 0)
    assert np.all(np.array(api._index_sizes(1, 1)) > 0)
