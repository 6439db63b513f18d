"""The network operators of libgs: layer norm, the linear layer with bias,
activation and residual in its epilogue, and the linear layer whose weights
go by ragged group, each forward and backward.

They carry the names of the C entry points (``include/gs.h``).  Matrices are
torch tensors [rows][width] of bfloat16, float16 or float32 whose last
stride is 1 (any leading stride of at least the width); bias, gamma, beta,
statistics and db are float32.  Outputs and workspaces that are not passed
in are taken from torch's allocator on the stream of the call.  Argument
errors raise ``ValueError`` (what only the tensors show: types, shapes,
devices) or ``GSError`` (what the library refuses); both before any work is
enqueued.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import GS_ACT_NONE, GS_OP_LAYER_NORM_BWD, _check, gs_workspace_size, lib

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_byref, _size_t = C.byref, C.c_size_t


def _type(x, name="x"):
    t = _TYPES.get(x.dtype)
    if t is None:
        raise ValueError(f"{name} is {x.dtype}: bfloat16, float16 or float32 expected")
    if x.dim() != 2:
        raise ValueError(f"{name} has {x.dim()} dimensions: [rows][width] expected")
    return t


def _ld(t, rows, width):
    """The leading dimension (a tensor of one row may hold any stride)."""
    return t.stride(0) if rows > 1 else max(t.stride(0), width)


def _matrix(t, rows, width, like, name):
    if t.dtype != like.dtype or t.shape != (rows, width):
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}: {like.dtype} ({rows}, {width}) expected")
    _placed(t, like, name)
    return _ld(t, rows, width)


def _placed(t, like, name):
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, x on {like.device}")
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name}: last stride {t.stride(-1)}, 1 expected")


def _vector(t, shape, like, name):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.shape != shape:
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}: torch.float32 {tuple(shape)} expected")
    if t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} has to be contiguous and on {like.device}")
    return t.data_ptr()


def _weights(w, groups, like, inner):
    """(leading dimension, out) of w [out][in] or [groups][out][in]."""
    if w.dtype != like.dtype or w.dim() != (3 if groups else 2) or w.shape[-1] != inner:
        want = "(groups, out, in)" if groups else "(out, in)"
        raise ValueError(f"w is {w.dtype} {tuple(w.shape)}: {like.dtype} {want} with in = {inner} expected")
    _placed(w, like, "w")
    out = w.shape[-2]
    ld = _ld(w, out if not groups else out * groups, inner) if not groups else max(w.stride(1), inner)
    if groups:
        if w.shape[0] != groups:
            raise ValueError(f"w holds {w.shape[0]} groups, offsets {groups}")
        if out == 1:
            ld = max(w.stride(0), inner) if groups > 1 else inner
        elif groups > 1 and w.stride(0) != out * ld:
            raise ValueError("w: the groups have to follow each other without a gap")
    return ld, out


def _groups(offsets, like):
    if offsets.dtype != torch.int64 or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"offsets is {offsets.dtype} {tuple(offsets.shape)}: torch.int64 (groups + 1,) expected")
    if offsets.device != like.device or not offsets.is_contiguous():
        raise ValueError(f"offsets has to be contiguous and on {like.device}")
    return offsets.shape[0] - 1


def _optional(t):
    return None if t is None else t.data_ptr()


_raw_stream = torch._C._cuda_getCurrentRawStream


def _launch(x, stream, call):
    """call(stream handle) with the tensors it makes, workspaces among them,
    belonging to the stream and the device of x."""
    if not x.is_cuda:
        raise ValueError(f"x is on {x.device}: the kernels need a GPU tensor")
    device = x.device.index
    if stream is not None:
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            return call(_raw_stream(device))
    return call(_raw_stream(device))


def _workspace(ws, need, like):
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device), need
    return ws, ws.numel() * ws.element_size()


def gs_layer_norm_fwd(x, gamma=None, beta=None, eps=1e-5, y=None, mean=None, rstd=None, stream=None):
    """y, mean and rstd of the rows of ``x`` (``mean``, ``rstd``: [rows]
    float32, what the backward pass reads)."""
    t = _type(x)
    rows, width = x.shape
    _placed(x, x, "x")
    g, b = _vector(gamma, (width,), x, "gamma"), _vector(beta, (width,), x, "beta")

    def call(s):
        nonlocal y, mean, rstd
        if y is None:
            y = torch.empty(rows, width, dtype=x.dtype, device=x.device)
        if mean is None:
            mean = torch.empty(rows, dtype=torch.float32, device=x.device)
        if rstd is None:
            rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
        _check(lib().gs_layer_norm_fwd(x.data_ptr(), _ld(x, rows, width), g, b, rows, width, eps, t, y.data_ptr(),
                                       _matrix(y, rows, width, x, "y"), _vector(mean, (rows,), x, "mean"),
                                       _vector(rstd, (rows,), x, "rstd"), s), "gs_layer_norm_fwd")
    _launch(x, stream, call)
    return y, mean, rstd


def gs_layer_norm_bwd(x, dy, gamma, mean, rstd, dres=None, dx=None, dgamma=None, dbeta=None, workspace=None,
                      stream=None):
    """(dx, dgamma, dbeta); ``dres`` is added into dx (the gradient that
    reaches x past the norm)."""
    t = _type(x)
    rows, width = x.shape
    _placed(x, x, "x")
    lddy = _matrix(dy, rows, width, x, "dy")
    ldr = 0 if dres is None else _matrix(dres, rows, width, x, "dres")
    g = _vector(gamma, (width,), x, "gamma")
    m, r = _vector(mean, (rows,), x, "mean"), _vector(rstd, (rows,), x, "rstd")

    def call(s):
        nonlocal dx, dgamma, dbeta
        if dx is None:
            dx = torch.empty(rows, width, dtype=x.dtype, device=x.device)
        if dgamma is None:
            dgamma = torch.empty(width, dtype=torch.float32, device=x.device)
        if dbeta is None:
            dbeta = torch.empty(width, dtype=torch.float32, device=x.device)
        ws, nbytes = _workspace(workspace, gs_workspace_size(GS_OP_LAYER_NORM_BWD, rows, width), x)
        _check(lib().gs_layer_norm_bwd(x.data_ptr(), _ld(x, rows, width), dy.data_ptr(), lddy, g, m, r,
                                       _optional(dres), ldr, rows, width, t, dx.data_ptr(),
                                       _matrix(dx, rows, width, x, "dx"), _vector(dgamma, (width,), x, "dgamma"),
                                       _vector(dbeta, (width,), x, "dbeta"), ws.data_ptr(), nbytes, s),
               "gs_layer_norm_bwd")
    _launch(x, stream, call)
    return dx, dgamma, dbeta


def _fwd(x, w, offsets, bias, act, residual, y, z, save_z, stream, where):
    t = _type(x)
    rows, inner = x.shape
    _placed(x, x, "x")
    groups = 0 if offsets is None else _groups(offsets, x)
    ldw, out = _weights(w, groups, x, inner)
    b = _vector(bias, (groups, out) if groups else (out,), x, "bias")
    ldr = 0 if residual is None else _matrix(residual, rows, out, x, "residual")

    def call(s):
        nonlocal y, z
        if y is None:
            y = torch.empty(rows, out, dtype=x.dtype, device=x.device)
        if z is None and save_z:
            z = torch.empty(rows, out, dtype=x.dtype, device=x.device)
        ldz = 0 if z is None else _matrix(z, rows, out, x, "z")
        head = (x.data_ptr(), _ld(x, rows, inner), w.data_ptr(), ldw, b)
        tail = (_optional(residual), ldr, rows, inner, out, t, act, y.data_ptr(), _matrix(y, rows, out, x, "y"),
                _optional(z), ldz, s)
        if groups:
            _check(lib().gs_grouped_linear_fwd(*head, offsets.data_ptr(), groups, *tail), where)
        else:
            _check(lib().gs_linear_fwd(*head, *tail), where)
    _launch(x, stream, call)
    return y if z is None else (y, z)


def gs_linear_fwd(x, w, bias=None, act=GS_ACT_NONE, residual=None, y=None, z=None, save_z=False, stream=None):
    """y = act(x w^T + bias) + residual; with ``save_z`` (or a ``z`` to
    write) also the value before the activation: (y, z)."""
    return _fwd(x, w, None, bias, act, residual, y, z, save_z, stream, "gs_linear_fwd")


def gs_grouped_linear_fwd(x, w, offsets, bias=None, act=GS_ACT_NONE, residual=None, y=None, z=None, save_z=False,
                          stream=None):
    """gs_linear_fwd with w[e], bias[e] for the rows offsets[e] ..
    offsets[e + 1] - 1 (``offsets``: int64 on the device, read there).
    Rows in no group are not written."""
    return _fwd(x, w, offsets, bias, act, residual, y, z, save_z, stream, "gs_grouped_linear_fwd")


def gs_linear_workspace_size(rows, inner, out, num_groups, type, act) -> int:
    b = _size_t(0)
    _check(lib().gs_linear_workspace_size(rows, inner, out, num_groups, type, act, _byref(b)),
           "gs_linear_workspace_size")
    return b.value


def _bwd(x, w, offsets, dy, z, act, dx, dw, db, want_dx, workspace, stream, where):
    t = _type(x)
    rows, inner = x.shape
    _placed(x, x, "x")
    groups = 0 if offsets is None else _groups(offsets, x)
    ldw, out = _weights(w, groups, x, inner)
    lddy = _matrix(dy, rows, out, x, "dy")
    if z is None and act != GS_ACT_NONE:
        raise ValueError("the activation's slope needs z, the value before it")
    ldz = 0 if z is None else _matrix(z, rows, out, x, "z")
    bshape = (groups, out) if groups else (out,)

    def call(s):
        nonlocal dx, dw, db
        if dx is None and want_dx:
            dx = torch.empty(rows, inner, dtype=x.dtype, device=x.device)
        if dw is None:
            dw = torch.empty(w.shape, dtype=w.dtype, device=x.device)
        elif dw.shape != w.shape or dw.dtype not in (w.dtype, torch.float32) or not dw.is_contiguous():
            raise ValueError(f"dw is {dw.dtype} {tuple(dw.shape)}: contiguous {w.dtype} or torch.float32 "
                             f"{tuple(w.shape)} expected")
        _placed(dw, x, "dw")
        if db is None:
            db = torch.empty(bshape, dtype=torch.float32, device=x.device)
        ws, nbytes = _workspace(workspace, gs_linear_workspace_size(rows, inner, out, groups, t, act), x)
        head = (x.data_ptr(), _ld(x, rows, inner), w.data_ptr(), ldw)
        tail = (_optional(z), ldz, dy.data_ptr(), lddy, rows, inner, out, t, act, _optional(dx),
                0 if dx is None else _matrix(dx, rows, inner, x, "dx"), dw.data_ptr(), _TYPES[dw.dtype],
                _vector(db, bshape, x, "db"), ws.data_ptr(), nbytes, s)
        if groups:
            _check(lib().gs_grouped_linear_bwd(*head, offsets.data_ptr(), groups, *tail), where)
        else:
            _check(lib().gs_linear_bwd(*head, *tail), where)
    _launch(x, stream, call)
    return dx, dw, db


def gs_linear_bwd(x, w, dy, z=None, act=GS_ACT_NONE, dx=None, dw=None, db=None, want_dx=True, workspace=None,
                  stream=None):
    """(dx, dw, db) of gs_linear_fwd for the gradient ``dy`` of y (the
    residual's gradient is dy itself).  ``dw`` is of w's type, or float32
    where such a tensor is passed in; ``want_dx`` false leaves dx out."""
    return _bwd(x, w, None, dy, z, act, dx, dw, db, want_dx, workspace, stream, "gs_linear_bwd")


def gs_grouped_linear_bwd(x, w, offsets, dy, z=None, act=GS_ACT_NONE, dx=None, dw=None, db=None, want_dx=True,
                          workspace=None, stream=None):
    """(dx, dw, db) of gs_grouped_linear_fwd; dw[e] and db[e] are 0 for an
    empty group, rows in no group have no dx."""
    return _bwd(x, w, offsets, dy, z, act, dx, dw, db, want_dx, workspace, stream, "gs_grouped_linear_bwd")
