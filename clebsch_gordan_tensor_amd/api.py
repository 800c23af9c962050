"""Thin Python binding of libe3hip.so (include/e3hip.h), via ctypes.

Argument marshalling only: every step of the convolution runs in the HIP
kernels of the library.  Tensors are torch tensors on the GPU (torch is used
for device memory and streams); the calls are asynchronous on the current
torch stream.  The library must have been built (``__graft_entry__.build()``
or ``python -m clebsch_gordan_tensor_amd.build``); a missing library raises.
"""
from __future__ import annotations

import ctypes as C
import functools
import operator
import os
from dataclasses import dataclass

from . import synth

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libe3hip.so")
_lib = None

E3_F32, E3_BF16 = 0, 1
E3_Y_GIVEN = 1
E3_OUT_PER_PATH = 2
E3_CHECK = 4
E3_ERR_GRAPH = -5


class E3Error(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"e3hip status {status}: {msg}")
        self.status = status


class _Irrep(C.Structure):
    _fields_ = [("mul", C.c_int32), ("l", C.c_int32), ("parity", C.c_int32)]


class _Irreps(C.Structure):
    _fields_ = [("n", C.c_int32), ("v", C.POINTER(_Irrep))]


class _Desc(C.Structure):
    _fields_ = [("x", _Irreps), ("y", _Irreps), ("out", _Irreps), ("flags", C.c_int32)]


EXPORTS = ["e3_num_paths", "e3_path_info", "e3_supported", "e3_cg_block",
           "e3_spherical_harmonics", "e3_spherical_harmonics_backward", "e3_tp_forward",
           "e3_tp_backward", "e3_conv_forward", "e3_conv_workspace_size",
           "e3_conv_prepare_transpose", "e3_conv_backward", "e3_edge_grad_to_nodes",
           "e3_linear_num_weights", "e3_linear", "e3_linear_workspace_size",
           "e3_linear_backward", "e3_conv_double_backward_scratch_size",
           "e3_conv_double_backward", "e3_radial_mlp", "e3_conv_forward_radial",
           "e3_radial_mlp_backward_workspace_size", "e3_radial_mlp_backward",
           "e3_generic_plan_size", "e3_generic_plan_build", "e3_tp_forward_generic",
           "e3_tp_forward_gemm", "e3_conv_forward_gemm",
           "e3_tp_backward_generic", "e3_conv_forward_generic", "e3_conv_backward_generic",
           "e3_conv_double_backward_generic", "e3_check_graph", "e3_check_graph_host", "e3_conv_backward_noalloc",
           "e3_tp_backward_gemm", "e3_conv_backward_gemm",
           "e3_radial_hidden_size", "e3_radial_hidden", "e3_conv_forward_radial_hidden",
           "e3_radial_mlp_hidden", "e3_conv_backward_radial_scratch_size",
           "e3_conv_backward_radial_hidden",
           "e3_layer_norm", "e3_layer_norm_workspace_size", "e3_layer_norm_backward",
           "e3_param_check", "e3_grad_norm_workspace_size", "e3_grad_norm", "e3_adamw",
           "e3_adamw_moments",
           "e3_release_all",
           "e3_last_error"]
E3_GEN_FORWARD, E3_GEN_DX, E3_GEN_DW, E3_GEN_DY, E3_GEN_GEMM = 0, 1, 2, 3, 4
E3_GEN_GEMM_DX, E3_GEN_GEMM_DW, E3_GEN_GEMM_DY = 5, 6, 7
E3_NORM_UNCENTERED = 1
E3_ADAMW_SKIP_NONFINITE = 1


class _CRadial(C.Structure):
    _fields_ = [("cutoff", C.c_float), ("n_basis", C.c_int32), ("hidden", C.c_int32),
                ("W1", C.c_void_p), ("W2", C.c_void_p)]


class _Param(C.Structure):
    _fields_ = [("n", C.c_int64), ("p", C.c_void_p), ("grad", C.c_void_p), ("m", C.c_void_p),
                ("v", C.c_void_p), ("m_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("p_bf16", C.c_void_p), ("weight_decay", C.c_float), ("grad_dtype", C.c_int)]


class _AdamwArgs(C.Structure):
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double),
                ("eps", C.c_double), ("step", C.c_int64), ("step_dev", C.c_void_p),
                ("lr_dev", C.c_void_p), ("grad_scale", C.c_void_p), ("flags", C.c_int32)]


def lib():
    """Open libe3hip.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with __graft_entry__.build()")
    L = C.CDLL(_LIB_PATH)
    vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    dp = C.POINTER(_Desc)
    L.e3_num_paths.argtypes = [dp, C.POINTER(i32)]
    L.e3_path_info.argtypes = [dp, i32, C.POINTER(i32), C.POINTER(i32), C.POINTER(i32)]
    L.e3_supported.argtypes = [dp, C.c_int]
    L.e3_supported.restype = i32
    L.e3_cg_block.argtypes = [i32, i32, i32, C.POINTER(C.c_double)]
    L.e3_spherical_harmonics.argtypes = [i32, i64, vp, vp, vp]
    L.e3_spherical_harmonics_backward.argtypes = [i32, i64, vp, vp, vp, vp]
    L.e3_tp_forward.argtypes = [dp, i64, vp, vp, vp, vp, C.c_int, vp]
    L.e3_tp_backward.argtypes = [dp, i64, vp, vp, vp, vp, vp, vp, vp, C.c_int, vp]
    L.e3_edge_grad_to_nodes.argtypes = [i32, i32, vp, vp, vp, sz, vp, vp, vp]
    ip = C.POINTER(_Irreps)
    L.e3_linear_num_weights.argtypes = [ip, ip, C.POINTER(i32)]
    L.e3_linear.argtypes = [ip, ip, i64, vp, vp, vp, C.c_int, vp]
    L.e3_linear_workspace_size.argtypes = [ip, ip, C.POINTER(sz)]
    L.e3_radial_mlp.argtypes = [C.POINTER(_CRadial), i32, i32, vp, vp, vp]
    L.e3_conv_forward_radial.argtypes = [dp, i32, i32, vp, vp, vp, sz, vp, vp,
                                         C.POINTER(_CRadial), vp, vp]
    L.e3_radial_hidden_size.argtypes = [i32, C.POINTER(sz)]
    L.e3_radial_hidden.argtypes = [C.POINTER(_CRadial), i32, vp, vp, sz, vp]
    L.e3_radial_mlp_hidden.argtypes = [C.POINTER(_CRadial), i32, i32, vp, sz, vp, vp]
    L.e3_conv_forward_radial_hidden.argtypes = [dp, i32, i32, vp, vp, vp, sz, vp, vp,
                                                C.POINTER(_CRadial), vp, sz, vp, vp]
    L.e3_conv_backward_radial_scratch_size.argtypes = [dp, i32, C.POINTER(sz)]
    L.e3_conv_backward_radial_hidden.argtypes = [dp, i32, i32, vp, vp, vp, sz, vp, vp,
                                                 C.POINTER(_CRadial), vp, sz, vp, vp, vp, vp, vp,
                                                 sz, vp]
    L.e3_generic_plan_size.argtypes = [dp, i32, C.POINTER(sz)]
    L.e3_generic_plan_build.argtypes = [dp, i32, vp, sz]
    L.e3_tp_backward_generic.argtypes = [dp, i64, vp, sz, vp, sz, vp, sz, vp, vp, vp, vp, vp, vp,
                                         vp, C.c_int, vp]
    L.e3_tp_forward_generic.argtypes = [dp, i64, vp, sz, vp, vp, vp, vp, C.c_int, vp]
    L.e3_tp_forward_gemm.argtypes = [dp, i64, vp, sz, vp, vp, vp, vp, vp]
    L.e3_conv_forward_gemm.argtypes = [dp, i32, i32, vp, vp, vp, sz, vp, vp, vp, vp, vp]
    L.e3_conv_forward_generic.argtypes = [dp, i32, i32, vp, vp, vp, sz, vp, sz, vp, vp, vp, vp,
                                          C.c_int, vp]
    L.e3_conv_backward_generic.argtypes = [dp, i32, i32, vp, vp, vp, sz, vp, sz, vp, sz, vp, sz,
                                           vp, vp, vp, vp, vp, vp, vp, C.c_int, vp]
    L.e3_conv_double_backward_generic.argtypes = [dp, i32, i32, vp, vp, vp, sz, vp, sz, vp, sz,
                                                  vp, sz, vp, sz, vp, vp, vp, vp, vp, vp, vp, vp,
                                                  vp, vp, vp, vp, sz, C.c_int, vp]
    L.e3_radial_mlp_backward_workspace_size.argtypes = [C.POINTER(_CRadial), i32, i32,
                                                        C.POINTER(sz)]
    L.e3_radial_mlp_backward.argtypes = [C.POINTER(_CRadial), i32, i32, vp, vp, vp, vp, vp, vp,
                                         sz, vp]
    L.e3_conv_double_backward_scratch_size.argtypes = [dp, i32, i32, C.c_int, C.POINTER(sz)]
    L.e3_conv_double_backward.argtypes = [dp, i32, i32, vp, vp, vp, sz, vp, vp, vp, vp, vp, vp,
                                          vp, vp, vp, vp, vp, vp, sz, C.c_int, vp]
    L.e3_linear_backward.argtypes = [ip, ip, i64, vp, vp, vp, vp, vp, vp, sz, C.c_int, vp]
    L.e3_conv_forward.argtypes = [dp, i32, i32, vp, vp, vp, sz, vp, vp, vp, vp, C.c_int, vp]
    L.e3_conv_workspace_size.argtypes = [i32, i32, C.POINTER(sz)]
    L.e3_conv_prepare_transpose.argtypes = [i32, i32, vp, vp, vp, vp, sz, vp]
    L.e3_conv_backward.argtypes = [dp, i32, i32, vp, vp, vp, sz, vp, vp, vp, vp, vp, vp, vp,
                                   C.c_int, vp]
    L.e3_check_graph.argtypes = [i32, i32, vp, vp, vp]
    L.e3_tp_backward_gemm.argtypes = [dp, i64, vp, sz, vp, sz, vp, sz, vp, vp, vp, vp, vp, vp, vp,
                                      vp]
    L.e3_conv_backward_gemm.argtypes = [dp, i32, i32, vp, vp, vp, sz, vp, sz, vp, sz, vp, sz, vp,
                                        vp, vp, vp, vp, vp, vp, vp]
    L.e3_conv_backward_noalloc.argtypes = [dp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                           C.c_int, vp]
    L.e3_check_graph_host.argtypes = [i32, i32, vp, vp]
    L.e3_layer_norm.argtypes = [ip, i64, vp, vp, vp, C.c_float, i32, vp, C.c_int, vp]
    L.e3_layer_norm_workspace_size.argtypes = [ip, i64, C.POINTER(sz)]
    L.e3_layer_norm_backward.argtypes = [ip, i64, vp, vp, vp, C.c_float, i32, vp, vp, vp, vp, sz,
                                         C.c_int, vp]
    pp = C.POINTER(_Param)
    L.e3_param_check.argtypes = [i32, pp]
    L.e3_grad_norm_workspace_size.argtypes = [i32, pp, C.POINTER(sz)]
    L.e3_grad_norm.argtypes = [i32, pp, C.c_double, vp, vp, sz, vp]
    L.e3_adamw.argtypes = [i32, pp, C.POINTER(_AdamwArgs), vp]
    L.e3_adamw_moments.argtypes = [i32, pp, C.POINTER(vp), C.POINTER(vp), vp]
    L.e3_release_all.argtypes = []
    L.e3_last_error.restype = C.c_char_p
    for name in EXPORTS:
        if name not in ("e3_last_error", "e3_supported", "e3_release_all"):
            getattr(L, name).restype = C.c_int
    L.e3_release_all.restype = None
    _lib = L
    return L


def _check(status):
    if status != 0:
        raise E3Error(status, lib().e3_last_error().decode())


@dataclass
class Desc:
    """Irreps of x, y (multiplicity 1) and the output, as lists of (l, parity),
    with C channels on x and the output."""
    x: list
    y: list
    out: list
    channels: int
    flags: int = 0

    @classmethod
    def from_strings(cls, x: str, y: str, out: str, flags: int = 0):
        C_, xi = synth.parse_irreps(x)
        _, yi = synth.parse_irreps(y)
        C2, oi = synth.parse_irreps(out)
        if C2 != C_:
            raise ValueError("x and out need the same multiplicity")
        return cls(xi, yi, oi, C_, flags)

    def with_flags(self, flags):
        return Desc(self.x, self.y, self.out, self.channels, flags)

    @property
    def dx(self):
        return synth.dim(self.x)

    @property
    def dy(self):
        return synth.dim(self.y)

    @property
    def dout(self):
        if self.flags & E3_OUT_PER_PATH:  # one output block per path, as the library lists them
            return sum(2 * self.out[path_info(self, i)[2]][0] + 1
                       for i in range(num_paths(self)))
        return synth.dim(self.out)

    def c(self):
        """ctypes struct (kept alive together with its arrays)."""
        def arr(ir, mul):
            a = (_Irrep * max(1, len(ir)))()
            for i, (l, p) in enumerate(ir):
                a[i] = _Irrep(mul, l, p)
            return a
        ax, ay, ao = arr(self.x, self.channels), arr(self.y, 1), arr(self.out, self.channels)
        d = _Desc(_Irreps(len(self.x), ax), _Irreps(len(self.y), ay),
                  _Irreps(len(self.out), ao), self.flags)
        d._keep = (ax, ay, ao)
        return d


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return E3_F32
    if t.dtype == torch.bfloat16:
        return E3_BF16
    raise TypeError(f"unsupported storage dtype {t.dtype}")


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _need(t, name, shape=None, dtype=None):
    import torch
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def check_graph(rowptr, sender, stream=None):
    """Host-side check of a CSR graph on the GPU (e3_check_graph): raises
    E3Error (status E3_ERR_GRAPH) naming the first violation.  Synchronises
    the stream."""
    import torch
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    _check(lib().e3_check_graph(rowptr.shape[0] - 1, sender.shape[0], _ptr(rowptr), _ptr(sender),
                                _stream(stream)))


def check_graph_host(rowptr, sender):
    """e3_check_graph on host (numpy int32) arrays: raises E3Error
    (status E3_ERR_GRAPH) naming the first violation."""
    import numpy as np
    rp = np.ascontiguousarray(rowptr, dtype=np.int32)
    sn = np.ascontiguousarray(sender, dtype=np.int32)
    _check(lib().e3_check_graph_host(rp.shape[0] - 1, sn.shape[0], rp.ctypes.data_as(C.c_void_p),
                                     sn.ctypes.data_as(C.c_void_p)))


def release_all():
    """Frees the library's host-side plan cache (e3_release_all)."""
    lib().e3_release_all()


def num_paths(desc: Desc) -> int:
    n = C.c_int32()
    _check(lib().e3_num_paths(C.byref(desc.c()), C.byref(n)))
    return n.value


def path_info(desc: Desc, i: int):
    a, b, c = C.c_int32(), C.c_int32(), C.c_int32()
    _check(lib().e3_path_info(C.byref(desc.c()), i, C.byref(a), C.byref(b), C.byref(c)))
    return a.value, b.value, c.value


def supported(desc: Desc, dtype_code: int = E3_F32) -> bool:
    return bool(lib().e3_supported(C.byref(desc.c()), dtype_code))


def cg_block(l1: int, l2: int, L: int):
    import numpy as np
    out = np.zeros((2 * L + 1) * (2 * l1 + 1) * (2 * l2 + 1))
    _check(lib().e3_cg_block(l1, l2, L, out.ctypes.data_as(C.POINTER(C.c_double))))
    return out.reshape(2 * L + 1, 2 * l1 + 1, 2 * l2 + 1)


def spherical_harmonics(lmax: int, vec, out=None, stream=None):
    import torch
    _need(vec, "vec", dtype=torch.float32)
    n = vec.shape[0]
    if out is None:
        out = torch.empty((n, (lmax + 1) ** 2), device=vec.device, dtype=torch.float32)
    _need(out, "out", shape=(n, (lmax + 1) ** 2), dtype=torch.float32)
    _check(lib().e3_spherical_harmonics(lmax, n, _ptr(vec), _ptr(out), _stream(stream)))
    return out


def spherical_harmonics_backward(lmax: int, vec, dY, out=None, stream=None):
    """dvec [n][3] = J^T dY, J the Jacobian of the harmonics of vec [n][3]."""
    import torch
    _need(vec, "vec", dtype=torch.float32)
    n = vec.shape[0]
    _need(vec, "vec", shape=(n, 3))
    _need(dY, "dY", shape=(n, (lmax + 1) ** 2), dtype=torch.float32)
    if out is None:
        out = torch.empty((n, 3), device=vec.device, dtype=torch.float32)
    _need(out, "out", shape=(n, 3), dtype=torch.float32)
    _check(lib().e3_spherical_harmonics_backward(lmax, n, _ptr(vec), _ptr(dY), _ptr(out),
                                                 _stream(stream)))
    return out


def tp_backward(desc: Desc, x, y, w, dz, dx=None, dw=None, dy=None, stream=None):
    """(dx, dw, dy) of z = tp_forward(x, y, w) for the cotangent dz."""
    import torch
    B = x.shape[0]
    P = num_paths(desc)
    _need(x, "x", shape=(B, desc.dx, desc.channels))
    _need(y, "y", shape=(B, desc.dy), dtype=torch.float32)
    _need(w, "w", shape=(B, P, desc.channels), dtype=x.dtype)
    _need(dz, "dz", shape=(B, desc.dout, desc.channels), dtype=x.dtype)
    dev, dt = x.device, x.dtype
    if dx is None:
        dx = torch.empty((B, desc.dx, desc.channels), device=dev, dtype=dt)
    if dw is None:
        dw = torch.empty((B, P, desc.channels), device=dev, dtype=dt)
    if dy is None:
        dy = torch.empty((B, desc.dy), device=dev, dtype=torch.float32)
    _need(dx, "dx", shape=(B, desc.dx, desc.channels), dtype=dt)
    _need(dw, "dw", shape=(B, P, desc.channels), dtype=dt)
    _need(dy, "dy", shape=(B, desc.dy), dtype=torch.float32)
    _check(lib().e3_tp_backward(C.byref(desc.c()), B, _ptr(x), _ptr(y), _ptr(w), _ptr(dz),
                                _ptr(dx), _ptr(dw), _ptr(dy), _dtype_code(x), _stream(stream)))
    return dx, dw, dy


def tp_forward(desc: Desc, x, y, w, out=None, stream=None):
    import torch
    B = x.shape[0]
    P = num_paths(desc)
    _need(x, "x", shape=(B, desc.dx, desc.channels))
    _need(y, "y", shape=(B, desc.dy), dtype=torch.float32)
    _need(w, "w", shape=(B, P, desc.channels), dtype=x.dtype)
    if out is None:
        out = torch.empty((B, desc.dout, desc.channels), device=x.device, dtype=x.dtype)
    _need(out, "out", shape=(B, desc.dout, desc.channels), dtype=x.dtype)
    _check(lib().e3_tp_forward(C.byref(desc.c()), B, _ptr(x), _ptr(y), _ptr(w), _ptr(out),
                               _dtype_code(x), _stream(stream)))
    return out


def conv_forward(desc: Desc, rowptr, sender, edge_vec_or_Y, x, w, out=None, workspace=None,
                 stream=None):
    """m = conv(x, Y(edge_vec), w).  workspace (optional) is the prepared
    per-graph index; with it receivers are visited in its locality order."""
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    P = num_paths(desc)
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    ycols = desc.dy if desc.flags & E3_Y_GIVEN else 3
    _need(edge_vec_or_Y, "edge_vec_or_Y", shape=(E, ycols), dtype=torch.float32)
    _need(x, "x", shape=(N, desc.dx, desc.channels))
    _need(w, "w", shape=(E, P, desc.channels), dtype=x.dtype)
    if out is None:
        out = torch.empty((N, desc.dout, desc.channels), device=x.device, dtype=x.dtype)
    _need(out, "out", shape=(N, desc.dout, desc.channels), dtype=x.dtype)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().e3_conv_forward(C.byref(desc.c()), N, E, _ptr(rowptr), _ptr(sender),
                                 _ptr(workspace), wsb, _ptr(edge_vec_or_Y), _ptr(x), _ptr(w),
                                 _ptr(out), _dtype_code(x), _stream(stream)))
    return out


def workspace_size(n_nodes: int, n_edges: int) -> int:
    b = C.c_size_t()
    _check(lib().e3_conv_workspace_size(n_nodes, n_edges, C.byref(b)))
    return b.value


def conv_prepare_transpose(rowptr, sender, workspace=None, edge_vec=None, stream=None):
    """Build the per-graph index (sender-ordered edge list and node locality
    order); returns the workspace (uint8 tensor).  edge_vec (optional, [E][3]
    float32) lets the order follow rebuilt positions."""
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    nb = workspace_size(N, E)
    if workspace is None:
        workspace = torch.empty(nb, device=rowptr.device, dtype=torch.uint8)
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    if edge_vec is not None:
        _need(edge_vec, "edge_vec", shape=(E, 3), dtype=torch.float32)
    _check(lib().e3_conv_prepare_transpose(N, E, _ptr(rowptr), _ptr(sender), _ptr(edge_vec),
                                           _ptr(workspace),
                                           workspace.numel() * workspace.element_size(),
                                           _stream(stream)))
    return workspace


def conv_backward(desc: Desc, rowptr, sender, workspace, edge_vec_or_Y, x, w, dm,
                  dx=None, dw=None, dY=None, stream=None):
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    P = num_paths(desc)
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    ycols = desc.dy if desc.flags & E3_Y_GIVEN else 3
    _need(edge_vec_or_Y, "edge_vec_or_Y", shape=(E, ycols), dtype=torch.float32)
    _need(x, "x", shape=(N, desc.dx, desc.channels))
    _need(w, "w", shape=(E, P, desc.channels), dtype=x.dtype)
    _need(dm, "dm", shape=(N, desc.dout, desc.channels), dtype=x.dtype)
    dev, dt = x.device, x.dtype
    if dx is None:
        dx = torch.empty((N, desc.dx, desc.channels), device=dev, dtype=dt)
    if dw is None:
        dw = torch.empty((E, P, desc.channels), device=dev, dtype=dt)
    if dY is None:
        dY = torch.empty((E, desc.dy), device=dev, dtype=torch.float32)
    _need(dx, "dx", shape=(N, desc.dx, desc.channels), dtype=dt)
    _need(dw, "dw", shape=(E, P, desc.channels), dtype=dt)
    _need(dY, "dY", shape=(E, desc.dy), dtype=torch.float32)
    _check(lib().e3_conv_backward(C.byref(desc.c()), N, E, _ptr(rowptr), _ptr(sender),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _ptr(edge_vec_or_Y), _ptr(x), _ptr(w), _ptr(dm), _ptr(dx),
                                  _ptr(dw), _ptr(dY), _dtype_code(x), _stream(stream)))
    return dx, dw, dY


def conv_backward_noalloc(desc: Desc, rowptr, sender, edge_vec_or_Y, x, w, dm, dx=None, dw=None,
                          dY=None, stream=None):
    """The backward with its per-graph index built inside the call in the
    library's fixed device scratch (e3_conv_backward_noalloc); the library
    allocates nothing (this wrapper allocates the outputs it is not given)."""
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    P = num_paths(desc)
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    ycols = desc.dy if desc.flags & E3_Y_GIVEN else 3
    _need(edge_vec_or_Y, "edge_vec_or_Y", shape=(E, ycols), dtype=torch.float32)
    _need(x, "x", shape=(N, desc.dx, desc.channels))
    _need(w, "w", shape=(E, P, desc.channels), dtype=x.dtype)
    _need(dm, "dm", shape=(N, desc.dout, desc.channels), dtype=x.dtype)
    dev, dt = x.device, x.dtype
    if dx is None:
        dx = torch.empty((N, desc.dx, desc.channels), device=dev, dtype=dt)
    if dw is None:
        dw = torch.empty((E, P, desc.channels), device=dev, dtype=dt)
    if dY is None:
        dY = torch.empty((E, desc.dy), device=dev, dtype=torch.float32)
    _need(dx, "dx", shape=(N, desc.dx, desc.channels), dtype=dt)
    _need(dw, "dw", shape=(E, P, desc.channels), dtype=dt)
    _need(dY, "dY", shape=(E, desc.dy), dtype=torch.float32)
    _check(lib().e3_conv_backward_noalloc(C.byref(desc.c()), N, E, _ptr(rowptr), _ptr(sender),
                                          _ptr(edge_vec_or_Y), _ptr(x), _ptr(w), _ptr(dm),
                                          _ptr(dx), _ptr(dw), _ptr(dY), _dtype_code(x),
                                          _stream(stream)))
    return dx, dw, dY


def edge_grad_to_nodes(rowptr, sender, workspace, edge_grad, out=None, stream=None):
    """node_grad [N][3]: sum of edge_grad over each node's in-edges minus the
    sum over its out-edges (r_e = pos[recv] - pos[sender]); forces are its
    negative.  workspace: from conv_prepare_transpose on the same graph."""
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    _need(edge_grad, "edge_grad", shape=(E, 3), dtype=torch.float32)
    if out is None:
        out = torch.empty((N, 3), device=rowptr.device, dtype=torch.float32)
    _need(out, "out", shape=(N, 3), dtype=torch.float32)
    _check(lib().e3_edge_grad_to_nodes(N, E, _ptr(rowptr), _ptr(sender), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       _ptr(edge_grad), _ptr(out), _stream(stream)))
    return out


def _irreps_struct(irreps, mul):
    a = (_Irrep * max(1, len(irreps)))()
    for i, (l, p) in enumerate(irreps):
        a[i] = _Irrep(mul, l, p)
    st = _Irreps(len(irreps), a)
    st._keep = a
    return st


def linear_num_weights(in_irreps, out_irreps) -> int:
    """Number of [Cin][Cout] weight matrices of the per-irrep channel mixing."""
    n = C.c_int32()
    a, b = _irreps_struct(in_irreps, 8), _irreps_struct(out_irreps, 32)
    _check(lib().e3_linear_num_weights(C.byref(a), C.byref(b), C.byref(n)))
    return n.value


def linear(in_irreps, out_irreps, x, W, out=None, stream=None):
    """y [rows][dout][Cout] = per-irrep channel mixing of x [rows][din][Cin]
    with W [n_pairs][Cin][Cout] (float32); in/out irreps as lists of (l, parity)."""
    import torch
    rows, din, cin = x.shape
    n_pairs, cin_w, cout = W.shape
    if cin_w != cin:
        raise ValueError("W and x disagree on Cin")
    if din != synth.dim(in_irreps):
        raise ValueError("x does not match the input irreps")
    _need(x, "x")
    _need(W, "W", dtype=torch.float32)
    dout = synth.dim(out_irreps)
    if out is None:
        out = torch.empty((rows, dout, cout), device=x.device, dtype=x.dtype)
    _need(out, "out", shape=(rows, dout, cout), dtype=x.dtype)
    a, b = _irreps_struct(in_irreps, cin), _irreps_struct(out_irreps, cout)
    if n_pairs != linear_num_weights(in_irreps, out_irreps):
        raise ValueError("W has the wrong number of matrices")
    _check(lib().e3_linear(C.byref(a), C.byref(b), rows, _ptr(x), _ptr(W), _ptr(out),
                           _dtype_code(x), _stream(stream)))
    return out


def linear_backward(in_irreps, out_irreps, x, W, dy, dx=None, dW=None, workspace=None,
                    stream=None):
    """(dx, dW) of linear() for the cotangent dy."""
    import torch
    rows, din, cin = x.shape
    n_pairs, _, cout = W.shape
    _need(x, "x")
    _need(W, "W", dtype=torch.float32)
    _need(dy, "dy", shape=(rows, synth.dim(out_irreps), cout), dtype=x.dtype)
    a, b = _irreps_struct(in_irreps, cin), _irreps_struct(out_irreps, cout)
    nb = C.c_size_t()
    _check(lib().e3_linear_workspace_size(C.byref(a), C.byref(b), C.byref(nb)))
    if workspace is None:
        workspace = torch.empty(nb.value, device=x.device, dtype=torch.uint8)
    if dx is None:
        dx = torch.empty_like(x)
    if dW is None:
        dW = torch.empty_like(W)
    _need(dx, "dx", shape=tuple(x.shape), dtype=x.dtype)
    _need(dW, "dW", shape=tuple(W.shape), dtype=torch.float32)
    _check(lib().e3_linear_backward(C.byref(a), C.byref(b), rows, _ptr(x), _ptr(W), _ptr(dy),
                                    _ptr(dx), _ptr(dW), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _dtype_code(x), _stream(stream)))
    return dx, dW


def conv_double_backward(desc: Desc, rowptr, sender, workspace, Y, x, w, dm, ddx, ddY, ddw,
                         scratch=None, stream=None):
    """(dx2, dY2, dw2, ddm): the double backward of the convolution for the
    variations (ddx, ddY, ddw) of the backward's outputs; desc needs
    E3_Y_GIVEN and Y the given harmonics."""
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    P = num_paths(desc)
    dt = x.dtype
    _need(Y, "Y", shape=(E, desc.dy), dtype=torch.float32)
    _need(ddY, "ddY", shape=(E, desc.dy), dtype=torch.float32)
    for t, n, shp in ((x, "x", (N, desc.dx, desc.channels)), (ddx, "ddx", (N, desc.dx, desc.channels)),
                      (w, "w", (E, P, desc.channels)), (ddw, "ddw", (E, P, desc.channels)),
                      (dm, "dm", (N, desc.dout, desc.channels))):
        _need(t, n, shape=shp, dtype=dt)
    nb = C.c_size_t()
    _check(lib().e3_conv_double_backward_scratch_size(C.byref(desc.c()), N, E, _dtype_code(x),
                                                      C.byref(nb)))
    if scratch is None:
        scratch = torch.empty(nb.value, device=x.device, dtype=torch.uint8)
    dx2, dw2 = torch.empty_like(x), torch.empty_like(w)
    dY2 = torch.empty_like(Y)
    ddm = torch.empty_like(dm)
    _check(lib().e3_conv_double_backward(
        C.byref(desc.c()), N, E, _ptr(rowptr), _ptr(sender), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(Y), _ptr(x), _ptr(w), _ptr(dm),
        _ptr(ddx), _ptr(ddY), _ptr(ddw), _ptr(dx2), _ptr(dY2), _ptr(dw2), _ptr(ddm),
        _ptr(scratch), scratch.numel() * scratch.element_size(), _dtype_code(x), _stream(stream)))
    return dx2, dY2, dw2, ddm


def _radial(cutoff, W1, W2):
    import torch
    _need(W1, "W1", dtype=torch.float32)
    _need(W2, "W2", dtype=torch.float32)
    if W1.dim() != 2 or W2.dim() != 2 or W1.shape[1] != W2.shape[0]:
        raise ValueError("W1 [n_basis][hidden] and W2 [hidden][n_cols] expected")
    return _CRadial(float(cutoff), W1.shape[0], W1.shape[1], W1.data_ptr(), W2.data_ptr())


def radial_mlp(edge_vec, cutoff, W1, W2, out=None, stream=None):
    """w[E][n_cols] = silu(B(|r|) W1) W2 with the 8-function Bessel basis."""
    import torch
    E = edge_vec.shape[0]
    _need(edge_vec, "edge_vec", shape=(E, 3), dtype=torch.float32)
    r = _radial(cutoff, W1, W2)
    n_cols = W2.shape[1]
    if out is None:
        out = torch.empty((E, n_cols), device=edge_vec.device, dtype=torch.float32)
    _need(out, "out", shape=(E, n_cols), dtype=torch.float32)
    _check(lib().e3_radial_mlp(C.byref(r), E, n_cols, _ptr(edge_vec), _ptr(out), _stream(stream)))
    return out


def conv_forward_radial(desc: Desc, rowptr, sender, edge_vec, x, cutoff, W1, W2, out=None,
                        workspace=None, stream=None):
    """m = conv(x, Y(edge_vec), w) with w = radial_mlp(edge_vec) computed inside
    the kernel (never stored); W2 is [64][P*C]."""
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    _need(edge_vec, "edge_vec", shape=(E, 3), dtype=torch.float32)
    _need(x, "x", shape=(N, desc.dx, desc.channels), dtype=torch.float32)
    r = _radial(cutoff, W1, W2)
    if W2.shape[1] != num_paths(desc) * desc.channels:
        raise ValueError("W2 must have P*C columns")
    if out is None:
        out = torch.empty((N, desc.dout, desc.channels), device=x.device, dtype=torch.float32)
    _need(out, "out", shape=(N, desc.dout, desc.channels), dtype=torch.float32)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().e3_conv_forward_radial(C.byref(desc.c()), N, E, _ptr(rowptr), _ptr(sender),
                                        _ptr(workspace), wsb, _ptr(edge_vec), _ptr(x), C.byref(r),
                                        _ptr(out), _stream(stream)))
    return out


def radial_hidden(edge_vec, cutoff, W1, W2, out=None, stream=None):
    """The radial MLP's hidden layer of every edge in the packed operand form
    conv_forward_radial_hidden reads (uint8 [E * 256])."""
    import torch
    E = edge_vec.shape[0]
    _need(edge_vec, "edge_vec", shape=(E, 3), dtype=torch.float32)
    r = _radial(cutoff, W1, W2)
    n = C.c_size_t()
    _check(lib().e3_radial_hidden_size(E, C.byref(n)))
    if out is None:
        out = torch.empty(n.value, device=edge_vec.device, dtype=torch.uint8)
    nb = out.numel() * out.element_size()
    _check(lib().e3_radial_hidden(C.byref(r), E, _ptr(edge_vec), _ptr(out), nb, _stream(stream)))
    return out


def radial_mlp_hidden(hidden, n_edges, cutoff, W1, W2, out=None, stream=None):
    """radial_mlp with the hidden layer from radial_hidden."""
    import torch
    r = _radial(cutoff, W1, W2)
    n_cols = W2.shape[1]
    if out is None:
        out = torch.empty((n_edges, n_cols), device=hidden.device, dtype=torch.float32)
    _need(out, "out", shape=(n_edges, n_cols), dtype=torch.float32)
    hb = hidden.numel() * hidden.element_size()
    _check(lib().e3_radial_mlp_hidden(C.byref(r), n_edges, n_cols, _ptr(hidden), hb, _ptr(out),
                                      _stream(stream)))
    return out


def conv_forward_radial_hidden(desc: Desc, rowptr, sender, edge_vec, x, cutoff, W1, W2, hidden,
                               out=None, workspace=None, stream=None):
    """conv_forward_radial with the hidden layer from radial_hidden."""
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    _need(edge_vec, "edge_vec", shape=(E, 3), dtype=torch.float32)
    _need(x, "x", shape=(N, desc.dx, desc.channels), dtype=torch.float32)
    r = _radial(cutoff, W1, W2)
    if W2.shape[1] != num_paths(desc) * desc.channels:
        raise ValueError("W2 must have P*C columns")
    if out is None:
        out = torch.empty((N, desc.dout, desc.channels), device=x.device, dtype=torch.float32)
    _need(out, "out", shape=(N, desc.dout, desc.channels), dtype=torch.float32)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    hb = hidden.numel() * hidden.element_size()
    _check(lib().e3_conv_forward_radial_hidden(C.byref(desc.c()), N, E, _ptr(rowptr),
                                               _ptr(sender), _ptr(workspace), wsb, _ptr(edge_vec),
                                               _ptr(x), C.byref(r), _ptr(hidden), hb, _ptr(out),
                                               _stream(stream)))
    return out


def conv_backward_radial_scratch_bytes(desc: Desc, n_edges):
    """Device scratch bytes conv_backward_radial_hidden needs."""
    nb = C.c_size_t()
    _check(lib().e3_conv_backward_radial_scratch_size(C.byref(desc.c()), n_edges, C.byref(nb)))
    return max(nb.value, 16)


def conv_backward_radial_hidden(desc: Desc, rowptr, sender, workspace, edge_vec, x, cutoff, W1,
                                W2, hidden, dm, dx=None, dw=None, dY=None, scratch=None,
                                stream=None):
    """(dx, dw, dY) of the fused radial forward: conv_backward with w formed
    from the hidden layer (radial_hidden of the same edge vectors)."""
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    P = num_paths(desc)
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    _need(edge_vec, "edge_vec", shape=(E, 3), dtype=torch.float32)
    _need(x, "x", shape=(N, desc.dx, desc.channels), dtype=torch.float32)
    _need(dm, "dm", shape=(N, desc.dout, desc.channels), dtype=torch.float32)
    r = _radial(cutoff, W1, W2)
    if W2.shape[1] != P * desc.channels:
        raise ValueError("W2 must have P*C columns")
    dev = x.device
    if dx is None:
        dx = torch.empty((N, desc.dx, desc.channels), device=dev, dtype=torch.float32)
    if dw is None:
        dw = torch.empty((E, P, desc.channels), device=dev, dtype=torch.float32)
    if dY is None:
        dY = torch.empty((E, desc.dy), device=dev, dtype=torch.float32)
    _need(dx, "dx", shape=(N, desc.dx, desc.channels), dtype=torch.float32)
    _need(dw, "dw", shape=(E, P, desc.channels), dtype=torch.float32)
    _need(dY, "dY", shape=(E, desc.dy), dtype=torch.float32)
    if scratch is None:
        scratch = torch.empty(conv_backward_radial_scratch_bytes(desc, E), device=dev,
                              dtype=torch.uint8)
    _check(lib().e3_conv_backward_radial_hidden(
        C.byref(desc.c()), N, E, _ptr(rowptr), _ptr(sender), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(edge_vec), _ptr(x), C.byref(r),
        _ptr(hidden), hidden.numel() * hidden.element_size(), _ptr(dm), _ptr(dx), _ptr(dw),
        _ptr(dY), _ptr(scratch), scratch.numel() * scratch.element_size(), _stream(stream)))
    return dx, dw, dY


def radial_mlp_backward_workspace_bytes(W1, W2, n_edges, n_cols):
    """Device workspace bytes radial_mlp_backward needs for n_edges x n_cols."""
    r = _radial(5.0, W1, W2)
    nb = C.c_size_t()
    _check(lib().e3_radial_mlp_backward_workspace_size(C.byref(r), n_edges, n_cols, C.byref(nb)))
    return nb.value


def radial_mlp_backward(edge_vec, cutoff, W1, W2, dw, workspace=None, stream=None):
    """(dW1, dW2, dvec) for the cotangent dw [E][n_cols] of radial_mlp; dvec is
    the edge-vector gradient through |r| only."""
    import torch
    E, n_cols = dw.shape
    _need(edge_vec, "edge_vec", shape=(E, 3), dtype=torch.float32)
    _need(dw, "dw", shape=(E, n_cols), dtype=torch.float32)
    r = _radial(cutoff, W1, W2)
    nb = C.c_size_t()
    _check(lib().e3_radial_mlp_backward_workspace_size(C.byref(r), E, n_cols, C.byref(nb)))
    if workspace is None:
        workspace = torch.empty(nb.value, device=dw.device, dtype=torch.uint8)
    dW1, dW2 = torch.empty_like(W1), torch.empty_like(W2)
    dvec = torch.empty_like(edge_vec)
    _check(lib().e3_radial_mlp_backward(
        C.byref(r), E, n_cols, _ptr(edge_vec), _ptr(dw), _ptr(dW1), _ptr(dW2), _ptr(dvec),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return dW1, dW2, dvec


_GENERIC_PLANS = {}


def generic_plan(desc: Desc, device, table=0):
    """Coefficient table `table` (E3_GEN_FORWARD, E3_GEN_DX, E3_GEN_DW,
    E3_GEN_DY) of the generic tensor product for desc: built on the host by the library, copied
    to device memory once per descriptor."""
    import numpy as np
    import torch
    key = (repr(desc.x), repr(desc.y), repr(desc.out), desc.channels, desc.flags, str(device),
           table)
    if key not in _GENERIC_PLANS:
        nb = C.c_size_t()
        _check(lib().e3_generic_plan_size(C.byref(desc.c()), table, C.byref(nb)))
        host = np.zeros(nb.value // 4, dtype=np.int32)
        _check(lib().e3_generic_plan_build(C.byref(desc.c()), table, host.ctypes.data, nb.value))
        _GENERIC_PLANS[key] = torch.from_numpy(host).to(device)
    return _GENERIC_PLANS[key]


def tp_forward_generic(desc: Desc, x, y, w, out=None, stream=None):
    """z = tensor product of x and y weighted by w (as tp_forward) through the
    coefficient-table kernel: any signature with degrees up to 7 (at most 63
    components per operand)."""
    import torch
    B = x.shape[0]
    P = num_paths(desc)
    _need(x, "x", shape=(B, desc.dx, desc.channels))
    _need(y, "y", shape=(B, desc.dy), dtype=torch.float32)
    _need(w, "w", shape=(B, P, desc.channels), dtype=x.dtype)
    if out is None:
        out = torch.empty((B, desc.dout, desc.channels), device=x.device, dtype=x.dtype)
    _need(out, "out", shape=(B, desc.dout, desc.channels), dtype=x.dtype)
    plan = generic_plan(desc, x.device)
    _check(lib().e3_tp_forward_generic(C.byref(desc.c()), B, _ptr(plan), plan.numel() * 4, _ptr(x),
                                       _ptr(y), _ptr(w), _ptr(out), _dtype_code(x),
                                       _stream(stream)))
    return out


def tp_forward_gemm(desc: Desc, x, y, w, out=None, stream=None):
    """z = tensor product of x and y weighted by w (as tp_forward_generic) as
    one dense product per output block on the fp32 matrix cores (float32,
    C % 16 == 0, degrees up to 7)."""
    import torch
    B = x.shape[0]
    P = num_paths(desc)
    _need(x, "x", shape=(B, desc.dx, desc.channels), dtype=torch.float32)
    _need(y, "y", shape=(B, desc.dy), dtype=torch.float32)
    _need(w, "w", shape=(B, P, desc.channels), dtype=torch.float32)
    if out is None:
        out = torch.empty((B, desc.dout, desc.channels), device=x.device, dtype=torch.float32)
    _need(out, "out", shape=(B, desc.dout, desc.channels), dtype=torch.float32)
    plan = generic_plan(desc, x.device, E3_GEN_GEMM)
    _check(lib().e3_tp_forward_gemm(C.byref(desc.c()), B, _ptr(plan), plan.numel() * 4, _ptr(x),
                                    _ptr(y), _ptr(w), _ptr(out), _stream(stream)))
    return out


def conv_forward_gemm(desc: Desc, rowptr, sender, edge_vec_or_Y, x, w, out=None, stream=None):
    """m = the convolution (as conv_forward_generic) as dense products per
    receiver and output block on the fp32 matrix cores; edge_vec_or_Y is the
    edge vectors [E][3] or, with E3_Y_GIVEN, the harmonics [E][dy]."""
    import torch
    N, E = rowptr.numel() - 1, sender.numel()
    P = num_paths(desc)
    Y = edge_vec_or_Y
    _need(x, "x", shape=(N, desc.dx, desc.channels), dtype=torch.float32)
    _need(Y, "edge_vec_or_Y", shape=(E, desc.dy if desc.flags & E3_Y_GIVEN else 3),
          dtype=torch.float32)
    _need(w, "w", shape=(E, P, desc.channels), dtype=torch.float32)
    if out is None:
        out = torch.empty((N, desc.dout, desc.channels), device=x.device, dtype=torch.float32)
    _need(out, "out", shape=(N, desc.dout, desc.channels), dtype=torch.float32)
    plan = generic_plan(desc, x.device, E3_GEN_GEMM)
    _check(lib().e3_conv_forward_gemm(C.byref(desc.c()), N, E, _ptr(rowptr), _ptr(sender),
                                      _ptr(plan), plan.numel() * 4, _ptr(Y), _ptr(x), _ptr(w),
                                      _ptr(out), _stream(stream)))
    return out


def tp_backward_gemm(desc: Desc, x, y, w, dz, dx=None, dw=None, dy=None, stream=None):
    """(dx, dw, dy) of tp_forward_gemm for the cotangent dz, as dense products
    on the fp32 matrix cores (tables E3_GEN_GEMM_DX, _DW, _DY)."""
    import torch
    B = x.shape[0]
    P = num_paths(desc)
    f32 = torch.float32
    _need(x, "x", shape=(B, desc.dx, desc.channels), dtype=f32)
    _need(y, "y", shape=(B, desc.dy), dtype=f32)
    _need(w, "w", shape=(B, P, desc.channels), dtype=f32)
    _need(dz, "dz", shape=(B, desc.dout, desc.channels), dtype=f32)
    dx = torch.empty_like(x) if dx is None else dx
    dw = torch.empty_like(w) if dw is None else dw
    dy = torch.empty_like(y) if dy is None else dy
    for t, n, ref in ((dx, "dx", x), (dw, "dw", w), (dy, "dy", y)):
        _need(t, n, shape=tuple(ref.shape), dtype=f32)
    px, pw, py = (generic_plan(desc, x.device, t)
                  for t in (E3_GEN_GEMM_DX, E3_GEN_GEMM_DW, E3_GEN_GEMM_DY))
    _check(lib().e3_tp_backward_gemm(C.byref(desc.c()), B, _ptr(px), px.numel() * 4, _ptr(pw),
                                     pw.numel() * 4, _ptr(py), py.numel() * 4, _ptr(x), _ptr(y),
                                     _ptr(w), _ptr(dz), _ptr(dx), _ptr(dw), _ptr(dy),
                                     _stream(stream)))
    return dx, dw, dy


def conv_backward_gemm(desc: Desc, rowptr, sender, workspace, Y, x, w, dm, dx=None, dw=None,
                       dY=None, stream=None):
    """(dx, dw, dY) of conv_forward_gemm with given harmonics (desc needs
    E3_Y_GIVEN), as dense products on the fp32 matrix cores; workspace from
    conv_prepare_transpose on the same graph."""
    import torch
    N, E = rowptr.numel() - 1, sender.numel()
    P = num_paths(desc)
    f32 = torch.float32
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    _need(Y, "Y", shape=(E, desc.dy), dtype=f32)
    _need(x, "x", shape=(N, desc.dx, desc.channels), dtype=f32)
    _need(w, "w", shape=(E, P, desc.channels), dtype=f32)
    _need(dm, "dm", shape=(N, desc.dout, desc.channels), dtype=f32)
    dx = torch.empty_like(x) if dx is None else dx
    dw = torch.empty_like(w) if dw is None else dw
    dY = torch.empty_like(Y) if dY is None else dY
    px, pw, py = (generic_plan(desc, x.device, t)
                  for t in (E3_GEN_GEMM_DX, E3_GEN_GEMM_DW, E3_GEN_GEMM_DY))
    _check(lib().e3_conv_backward_gemm(C.byref(desc.c()), N, E, _ptr(rowptr), _ptr(sender),
                                       _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _ptr(px), px.numel() * 4, _ptr(pw), pw.numel() * 4,
                                       _ptr(py), py.numel() * 4, _ptr(Y), _ptr(x), _ptr(w),
                                       _ptr(dm), _ptr(dx), _ptr(dw), _ptr(dY), _stream(stream)))
    return dx, dw, dY


def tp_backward_generic(desc: Desc, x, y, w, dz, stream=None):
    """(dx, dw, dy) of tp_forward_generic for the cotangent dz."""
    import torch
    B = x.shape[0]
    P = num_paths(desc)
    _need(x, "x", shape=(B, desc.dx, desc.channels))
    _need(y, "y", shape=(B, desc.dy), dtype=torch.float32)
    _need(w, "w", shape=(B, P, desc.channels), dtype=x.dtype)
    _need(dz, "dz", shape=(B, desc.dout, desc.channels), dtype=x.dtype)
    px, pw, py = (generic_plan(desc, x.device, t) for t in (E3_GEN_DX, E3_GEN_DW, E3_GEN_DY))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    dy = torch.empty((B, desc.dy), device=x.device, dtype=torch.float32)
    _check(lib().e3_tp_backward_generic(
        C.byref(desc.c()), B, _ptr(px), px.numel() * 4, _ptr(pw), pw.numel() * 4, _ptr(py),
        py.numel() * 4, _ptr(x), _ptr(y), _ptr(w), _ptr(dz), _ptr(dx), _ptr(dw), _ptr(dy),
        _dtype_code(x), _stream(stream)))
    return dx, dw, dy


def conv_forward_generic(desc: Desc, rowptr, sender, edge_vec_or_Y, x, w, out=None,
                         workspace=None, stream=None):
    """m = conv(x, Y(edge_vec), w) (as conv_forward) through the
    coefficient-table kernels: any signature with degrees up to 7 (at most 63
    components per operand; harmonics from edge vectors to degree 6)."""
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    P = num_paths(desc)
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    ycols = desc.dy if desc.flags & E3_Y_GIVEN else 3
    _need(edge_vec_or_Y, "edge_vec_or_Y", shape=(E, ycols), dtype=torch.float32)
    _need(x, "x", shape=(N, desc.dx, desc.channels))
    _need(w, "w", shape=(E, P, desc.channels), dtype=x.dtype)
    if out is None:
        out = torch.empty((N, desc.dout, desc.channels), device=x.device, dtype=x.dtype)
    _need(out, "out", shape=(N, desc.dout, desc.channels), dtype=x.dtype)
    plan = generic_plan(desc, x.device, E3_GEN_FORWARD)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().e3_conv_forward_generic(
        C.byref(desc.c()), N, E, _ptr(rowptr), _ptr(sender), _ptr(workspace), wsb, _ptr(plan),
        plan.numel() * 4, _ptr(edge_vec_or_Y), _ptr(x), _ptr(w), _ptr(out), _dtype_code(x),
        _stream(stream)))
    return out


def conv_backward_generic(desc: Desc, rowptr, sender, workspace, edge_vec_or_Y, x, w, dm,
                          dx=None, dw=None, dY=None, stream=None):
    """(dx, dw, dY) of conv_forward_generic for the cotangent dm; workspace
    from conv_prepare_transpose on the same graph."""
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    P = num_paths(desc)
    _need(rowptr, "rowptr", dtype=torch.int32)
    _need(sender, "sender", dtype=torch.int32)
    ycols = desc.dy if desc.flags & E3_Y_GIVEN else 3
    _need(edge_vec_or_Y, "edge_vec_or_Y", shape=(E, ycols), dtype=torch.float32)
    _need(x, "x", shape=(N, desc.dx, desc.channels))
    _need(w, "w", shape=(E, P, desc.channels), dtype=x.dtype)
    _need(dm, "dm", shape=(N, desc.dout, desc.channels), dtype=x.dtype)
    dev, dt = x.device, x.dtype
    if dx is None:
        dx = torch.empty((N, desc.dx, desc.channels), device=dev, dtype=dt)
    if dw is None:
        dw = torch.empty((E, P, desc.channels), device=dev, dtype=dt)
    if dY is None:
        dY = torch.empty((E, desc.dy), device=dev, dtype=torch.float32)
    _need(dx, "dx", shape=(N, desc.dx, desc.channels), dtype=dt)
    _need(dw, "dw", shape=(E, P, desc.channels), dtype=dt)
    _need(dY, "dY", shape=(E, desc.dy), dtype=torch.float32)
    px, pw, py = (generic_plan(desc, x.device, t) for t in (E3_GEN_DX, E3_GEN_DW, E3_GEN_DY))
    _check(lib().e3_conv_backward_generic(
        C.byref(desc.c()), N, E, _ptr(rowptr), _ptr(sender), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(px), px.numel() * 4, _ptr(pw),
        pw.numel() * 4, _ptr(py), py.numel() * 4, _ptr(edge_vec_or_Y), _ptr(x), _ptr(w), _ptr(dm),
        _ptr(dx), _ptr(dw), _ptr(dY), _dtype_code(x), _stream(stream)))
    return dx, dw, dY


def conv_double_backward_generic(desc: Desc, rowptr, sender, workspace, Y, x, w, dm, ddx, ddY,
                                 ddw, scratch=None, stream=None):
    """(dx2, dY2, dw2, ddm) as conv_double_backward through the coefficient
    tables (degrees up to 7); desc needs E3_Y_GIVEN."""
    import torch
    N, E = rowptr.shape[0] - 1, sender.shape[0]
    P = num_paths(desc)
    dt = x.dtype
    _need(Y, "Y", shape=(E, desc.dy), dtype=torch.float32)
    _need(ddY, "ddY", shape=(E, desc.dy), dtype=torch.float32)
    for t, n, shp in ((x, "x", (N, desc.dx, desc.channels)), (ddx, "ddx", (N, desc.dx, desc.channels)),
                      (w, "w", (E, P, desc.channels)), (ddw, "ddw", (E, P, desc.channels)),
                      (dm, "dm", (N, desc.dout, desc.channels))):
        _need(t, n, shape=shp, dtype=dt)
    nb = C.c_size_t()
    _check(lib().e3_conv_double_backward_scratch_size(C.byref(desc.c()), N, E, _dtype_code(x),
                                                      C.byref(nb)))
    if scratch is None:
        scratch = torch.empty(nb.value, device=x.device, dtype=torch.uint8)
    pf, px, pw, py = (generic_plan(desc, x.device, t)
                      for t in (E3_GEN_FORWARD, E3_GEN_DX, E3_GEN_DW, E3_GEN_DY))
    dx2, dw2 = torch.empty_like(x), torch.empty_like(w)
    dY2 = torch.empty_like(Y)
    ddm = torch.empty_like(dm)
    _check(lib().e3_conv_double_backward_generic(
        C.byref(desc.c()), N, E, _ptr(rowptr), _ptr(sender), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(pf), pf.numel() * 4, _ptr(px),
        px.numel() * 4, _ptr(pw), pw.numel() * 4, _ptr(py), py.numel() * 4, _ptr(Y), _ptr(x),
        _ptr(w), _ptr(dm), _ptr(ddx), _ptr(ddY), _ptr(ddw), _ptr(dx2), _ptr(dY2), _ptr(dw2),
        _ptr(ddm), _ptr(scratch), scratch.numel() * scratch.element_size(), _dtype_code(x),
        _stream(stream)))
    return dx2, dY2, dw2, ddm


# ------------------------------------------------------------ normalisation

def _raw_stream(device, stream):
    """The given stream's handle, or that of the device's current stream."""
    import torch
    return (torch._C._cuda_getCurrentRawStream(device.index) if stream is None
            else stream.cuda_stream)


def _on(device, fn, *args, stream=None):
    """Calls fn(*args, stream) with `device` current, whichever device is now."""
    import torch
    s = _raw_stream(device, stream)
    if torch.cuda.current_device() == device.index:
        status = fn(*args, s)
    else:
        with torch.cuda.device(device):
            status = fn(*args, s)
    if status != 0:
        _check(status)


_dtype_of = operator.attrgetter("dtype")


def _new(stream, shape, device, dtype):
    """Memory for a call on `stream`: of that stream's own, since work still
    queued on the current one may use what it frees."""
    import torch
    if stream is None:
        return torch.empty(shape, device=device, dtype=dtype)
    with torch.cuda.stream(stream):
        return torch.empty(shape, device=device, dtype=dtype)


def _addr(t):
    return None if t is None else t.data_ptr()


def _need_on(device, t, name, shape, dtype):
    """_need, on `device`; None passes."""
    if t is not None:
        _need(t, name, shape, dtype)
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


@functools.lru_cache(maxsize=256)
def _norm_spec(irreps, channels):
    """(struct, components, blocks, 0e blocks) of an irreps tuple."""
    return (_irreps_struct(irreps, channels), synth.dim(irreps), len(irreps),
            sum(1 for l, p in irreps if l == 0 and p == 1))


@functools.lru_cache(maxsize=256)
def _norm_workspace_size(irreps, rows, channels):
    nb = C.c_size_t()
    _check(lib().e3_layer_norm_workspace_size(C.byref(_norm_spec(irreps, channels)[0]), rows,
                                              C.byref(nb)))
    return nb.value


def _norm_x(irreps, x):
    """(irreps tuple, its spec) after the checks of x."""
    _need(x, "x")
    irreps = tuple(map(tuple, irreps))
    if x.dim() != 3:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [rows][components][channels]")
    spec = _norm_spec(irreps, x.shape[2])
    if x.shape[1] != spec[1]:
        raise ValueError(f"x has {x.shape[1]} components, the irreps {spec[1]}")
    return irreps, spec


def layer_norm(irreps, x, weight=None, bias=None, eps=1e-5, flags=0, out=None, stream=None):
    """Normalised features y [rows][dim][C] of x over `irreps` ([(l, parity)]),
    block by block: 0e blocks centred over their channels (unless
    E3_NORM_UNCENTERED), every block divided by its root mean square over
    components and channels, times weight [blocks][C], plus bias [0e blocks][C]
    for 0e blocks.  [(0, 1)] is the ordinary layer norm over C channels.  out
    may be x."""
    import torch
    irreps, (st, _, n_blocks, scalars) = _norm_x(irreps, x)
    dev, shape = x.device, x.shape
    _need_on(dev, weight, "weight", (n_blocks, shape[2]), torch.float32)
    _need_on(dev, bias, "bias", (scalars, shape[2]), torch.float32)
    if out is None:
        out = _new(stream, shape, dev, x.dtype)
    else:
        _need_on(dev, out, "out", shape, x.dtype)
    _on(dev, lib().e3_layer_norm, C.byref(st), shape[0], x.data_ptr(), _addr(weight), _addr(bias),
        eps, flags, out.data_ptr(), _dtype_code(x), stream=stream)
    return out


def layer_norm_workspace_size(irreps, rows: int, channels: int) -> int:
    """Bytes of layer_norm_backward's workspace."""
    return _norm_workspace_size(tuple(map(tuple, irreps)), rows, channels)


def layer_norm_backward(irreps, x, weight, dy, eps=1e-5, flags=0, dx=None, dweight=None,
                        dbias=None, workspace=None, stream=None):
    """(dx, dweight [blocks][C], dbias [0e blocks][C]) of layer_norm for the
    cotangent dy; weight may be None (ones).  dx may be x or dy."""
    import torch
    irreps, (st, _, n_blocks, scalars) = _norm_x(irreps, x)
    dev, shape, f32 = x.device, x.shape, torch.float32
    ch = shape[2]
    _need_on(dev, weight, "weight", (n_blocks, ch), f32)
    _need(dy, "dy")
    _need_on(dev, dy, "dy", shape, x.dtype)
    _need_on(dev, dx, "dx", shape, x.dtype)
    _need_on(dev, dweight, "dweight", (n_blocks, ch), f32)
    _need_on(dev, dbias, "dbias", (scalars, ch), f32)
    _need_on(dev, workspace, "workspace", None, None)
    if dx is None:
        dx = _new(stream, shape, dev, x.dtype)
    if dweight is None:
        dweight = _new(stream, (n_blocks, ch), dev, f32)
    if dbias is None:
        dbias = _new(stream, (scalars, ch), dev, f32)
    if workspace is None:
        workspace = _new(stream, _norm_workspace_size(irreps, shape[0], ch), dev, torch.uint8)
    _on(dev, lib().e3_layer_norm_backward, C.byref(st), shape[0], x.data_ptr(), _addr(weight),
        dy.data_ptr(), eps, flags, dx.data_ptr(), dweight.data_ptr(), dbias.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _dtype_code(x),
        stream=stream)
    return dx, dweight, dbias


# ---------------------------------------------------------------- optimizer

def _column(device, tensors, dtypes):
    """Whether every one is a contiguous tensor of its dtype on `device` (a
    list may hold hundreds: the whole column is looked at once)."""
    import torch
    T = torch.Tensor
    try:
        return (all(map(T.is_contiguous, tensors))
                and set(map(T.get_device, tensors)) <= {device.index}
                and list(map(_dtype_of, tensors)) == dtypes)
    except TypeError:  # something else than a tensor
        return False


def _tensors(column, name):
    """Refuses what is no tensor, such as the None of a parameter without a gradient."""
    import torch
    if all(issubclass(c, torch.Tensor) for c in set(map(type, column))):
        return
    i, t = next((i, t) for i, t in enumerate(column) if not isinstance(t, torch.Tensor))
    if t is None:
        raise ValueError(f"{name}[{i}] is required")
    raise TypeError(f"{name}[{i}] must be a tensor, got {type(t).__name__}")


class Params:
    """The tensors of a network's weights with what their update reads and
    writes (lists of equal length; every tensor contiguous, on one GPU):

      params        float32, any shape; None for a list that only serves
                    grad_norm
      grads         float32 or bfloat16, the shape of the parameter
      m, v          moments: float32 of as many elements, or 8-bit codes
                    (int8 and uint8), for which m_scale and v_scale (float32
                    [ceil(n/256)], None for the other tensors) are needed;
                    adamw_state makes them
      copies        bfloat16 copies of the parameters to be kept up to date,
                    or None
      weight_decay  one number, or one a tensor

    Keeps references to the tensors and their addresses: a tensor whose
    storage is replaced needs a new list (set_grads for new gradients)."""

    def __init__(self, params=None, grads=None, m=None, v=None, m_scale=None, v_scale=None,
                 copies=None, weight_decay=0.0):
        import torch
        if grads is None:
            raise ValueError("grads is required")
        n = len(grads)
        self.updates = params is not None
        cols = {"params": params, "m": m, "v": v, "m_scale": m_scale, "v_scale": v_scale,
                "copies": copies}
        if not self.updates and any(c is not None for c in cols.values()):
            raise ValueError("params is required with moments, scales or copies")
        if self.updates and (m is None or v is None):
            raise ValueError("m and v are required with params")
        for name, c in cols.items():
            if c is not None and len(c) != n:
                raise ValueError(f"{name} has {len(c)} tensors, grads {n}")
        _tensors(grads, "grads")
        decay = [weight_decay] * n if isinstance(weight_decay, (int, float)) else list(weight_decay)
        if len(decay) != n:
            raise ValueError(f"weight_decay has {len(decay)} values, expected {n}")
        self._arr = (_Param * max(1, n))()
        self._n = n
        self._keep = {k: list(c) if c is not None else [None] * n for k, c in cols.items()}
        self.device = grads[0].device if n else torch.device("cuda", torch.cuda.current_device())
        self.sizes = [g.numel() for g in grads]
        if self.updates:
            codes = [a is not None or b is not None
                     for a, b in zip(self._keep["m_scale"], self._keep["v_scale"])]
            runs = [((k + 255) // 256,) if c else None for k, c in zip(self.sizes, codes)]
            self._fill("p", "params", torch.float32, [g.shape for g in grads])
            self._fill("m", "m", [torch.int8 if c else torch.float32 for c in codes])
            self._fill("v", "v", [torch.uint8 if c else torch.float32 for c in codes])
            self._fill("m_scale", "m_scale", torch.float32, runs, codes)
            self._fill("v_scale", "v_scale", torch.float32, runs, codes)
            self._fill("p_bf16", "copies", torch.bfloat16, [g.shape for g in grads],
                       [c is not None for c in self._keep["copies"]])
        for e, k, d in zip(self._arr, self.sizes, decay):
            e.n, e.weight_decay = k, d
        self.set_grads(grads)
        nb = C.c_size_t()
        _check(lib().e3_grad_norm_workspace_size(n, self._arr, C.byref(nb)))
        self.workspace_bytes = nb.value  # of grad_norm

    def _fill(self, field, name, dtypes, shapes=None, given=None):
        """One pointer of every tensor, after its checks."""
        at = range(self._n) if given is None else [i for i in range(self._n) if given[i]]
        ts = [self._keep[name][i] for i in at]
        want = [dtypes[i] for i in at] if isinstance(dtypes, list) else [dtypes] * len(ts)
        if not (_column(self.device, ts, want) and
                ([t.shape for t in ts] == [shapes[i] for i in at] if shapes else
                 [t.numel() for t in ts] == [self.sizes[i] for i in at])):
            for i, t, dt in zip(at, ts, want):  # which one it is
                _need(t, f"{name}[{i}]")
                _need_on(self.device, t, f"{name}[{i}]", shapes[i] if shapes else None, dt)
                if t.numel() != (self.sizes[i] if shapes is None else t.numel()):
                    raise ValueError(f"{name}[{i}] has {t.numel()} elements, "
                                     f"expected {self.sizes[i]}")
        for i, t in zip(at, ts):
            setattr(self._arr[i], field, t.data_ptr())

    def set_grads(self, grads):
        """Other gradient tensors for the same parameters."""
        import torch
        if len(grads) != self._n:
            raise ValueError(f"grads has {len(grads)} tensors, expected {self._n}")
        _tensors(grads, "grads")
        types = {torch.float32: E3_F32, torch.bfloat16: E3_BF16}
        shapes = [g.shape if p is None else p.shape for g, p in zip(grads, self._keep["params"])]
        if not (_column(self.device, grads, [g.dtype for g in grads])
                and all(g.dtype in types for g in grads)
                and [g.shape for g in grads] == shapes
                and [g.numel() for g in grads] == self.sizes):
            for i, g in enumerate(grads):  # which one it is
                _need(g, f"grads[{i}]")
                _need_on(self.device, g, f"grads[{i}]", shapes[i], None)
                _dtype_code(g)
                if g.numel() != self.sizes[i]:
                    raise ValueError(f"grads[{i}] has {g.numel()} elements, "
                                     f"expected {self.sizes[i]}")
        before = [(e.grad, e.grad_dtype) for e in self._arr]
        for e, g in zip(self._arr, grads):
            e.grad, e.grad_dtype = g.data_ptr(), types[g.dtype]
        try:
            if self.updates:
                _check(lib().e3_param_check(self._n, self._arr))
        except E3Error:  # the list stays as it was
            for e, (at, code) in zip(self._arr, before):
                e.grad, e.grad_dtype = at, code
            raise
        self._grads = list(grads)

    def __len__(self):
        return self._n


def adamw_state(params, bits=32):
    """Zero moments for a list of parameters: (m, v, m_scale, v_scale), lists
    as Params takes them; bits 32, or 8 (a list gives each tensor its own)."""
    import torch
    bits = [bits] * len(params) if isinstance(bits, int) else list(bits)
    if len(bits) != len(params) or any(b not in (8, 32) for b in bits):
        raise ValueError("bits is 8 or 32, or one of them for every parameter")
    m, v, ms, vs = [], [], [], []
    for p, b in zip(params, bits):
        n, dev = p.numel(), p.device
        z = lambda size, dt: torch.zeros(size, device=dev, dtype=dt)  # noqa: E731
        m.append(z(n, torch.int8 if b == 8 else torch.float32))
        v.append(z(n, torch.uint8 if b == 8 else torch.float32))
        ms.append(z((n + 255) // 256, torch.float32) if b == 8 else None)
        vs.append(z((n + 255) // 256, torch.float32) if b == 8 else None)
    return m, v, ms, vs


def grad_norm(params: Params, max_norm=float("inf"), out=None, workspace=None, stream=None):
    """float32 [2] on the GPU: the 2-norm of all gradients together and the
    factor min(1, max_norm / (norm + 1e-6)) that clips it (NaN for a norm that
    is not finite); out[1:] is adamw's grad_scale."""
    import torch
    dev = params.device
    _need_on(dev, out, "out", (2,), torch.float32)
    _need_on(dev, workspace, "workspace", None, None)
    if out is None:
        out = _new(stream, 2, dev, torch.float32)
    if workspace is None:
        workspace = _new(stream, params.workspace_bytes, dev, torch.uint8)
    _on(dev, lib().e3_grad_norm, len(params), params._arr, max_norm, out.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), stream=stream)
    return out


def adamw(params: Params, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=None, flags=0,
          stream=None):
    """One AdamW step over every tensor of the list.  step (1 for the first
    update) is an int, or an int64 GPU tensor of one element; lr a number, or
    a float32 GPU tensor of one element (both are read when the step runs, so
    a captured step can be replayed); grad_scale a float32 GPU tensor of one
    element that multiplies the gradients."""
    import torch
    if not params.updates:
        raise ValueError("the list holds gradients only")
    dev = params.device
    a = _AdamwArgs(0.0, beta1, beta2, eps, 1, None, None, None, flags)
    if isinstance(step, torch.Tensor):
        a.step_dev = _one_value(dev, step, "step", torch.int64)
    else:
        a.step = step
    if isinstance(lr, torch.Tensor):
        a.lr_dev = _one_value(dev, lr, "lr", torch.float32)
    else:
        a.lr = lr
    if grad_scale is not None:
        a.grad_scale = _one_value(dev, grad_scale, "grad_scale", torch.float32)
    _on(dev, lib().e3_adamw, len(params), params._arr, C.byref(a), stream=stream)


def _one_value(device, t, name, dtype):
    _need_on(device, t, name, None, dtype)
    if t.numel() != 1:
        raise ValueError(f"{name} must hold one element")
    return t.data_ptr()


def adamw_moments(params: Params, m_out=None, v_out=None, stream=None):
    """(m, v): lists of the 8-bit moments of every tensor as float32 [n]."""
    import torch
    if not params.updates:
        raise ValueError("the list holds gradients only")
    n, dev = len(params), params.device
    outs = []
    for given, name in ((m_out, "m_out"), (v_out, "v_out")):
        if given is None:
            given = [_new(stream, k, dev, torch.float32) for k in params.sizes]
        if len(given) != n:
            raise ValueError(f"{name} has {len(given)} tensors, expected {n}")
        if not (_column(dev, given, [torch.float32] * n)
                and list(map(torch.Tensor.numel, given)) == params.sizes):
            for i, (t, k) in enumerate(zip(given, params.sizes)):
                _need_on(dev, _need(t, f"{name}[{i}]"), f"{name}[{i}]", None, torch.float32)
                if t.numel() != k:
                    raise ValueError(f"{name}[{i}] has {t.numel()} elements, expected {k}")
        outs.append((given, (C.c_void_p * max(1, n))(*map(torch.Tensor.data_ptr, given))))
    _on(dev, lib().e3_adamw_moments, n, params._arr, outs[0][1], outs[1][1], stream=stream)
    return outs[0][0], outs[1][0]
