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
_F32, _I64, _U8 = torch.float32, torch.int64, torch.uint8
_empty = torch.empty
_byref, _size_t = C.byref, C.c_size_t
# the stream's handle without a Stream object, where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = torch.cuda.current_device


def _type(x, name="x"):
    t = _TYPES.get(x.dtype)
    if t is None:
        raise ValueError(f"{name} is {x.dtype}: bfloat16, float16 or float32 expected")
    if x.dim() != 2:
        raise ValueError(f"{name} has {x.dim()} dimensions: [rows][width] expected")
    return t


def _matrix(t, rows, width, like, name):
    """The leading dimension of t [rows][width] (one row may hold any stride)."""
    if t.dtype != like.dtype or t.shape != (rows, width):
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}: {like.dtype} ({rows}, {width}) expected")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, x on {like.device}")
    ld, last = t.stride()
    if last != 1 and width != 1:
        raise ValueError(f"{name}: last stride {last}, 1 expected")
    return ld if rows > 1 or ld >= width else width


def _vector(t, shape, like, name):
    if t is None:
        return None
    if t.dtype != _F32 or t.shape != shape:
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}: torch.float32 {tuple(shape)} expected")
    if t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} has to be contiguous and on {like.device}")
    return t.data_ptr()


def _weights(w, groups, like, inner):
    """(leading dimension, out) of w [out][inner], or of [groups][out][inner]
    whose groups follow each other without a gap."""
    if w.dtype != like.dtype or w.dim() != (3 if groups else 2) or w.shape[-1] != inner:
        want = "(groups, out, in)" if groups else "(out, in)"
        raise ValueError(f"w is {w.dtype} {tuple(w.shape)}: {like.dtype} {want} with in = {inner} expected")
    out = w.shape[-2]
    if not groups:
        return _matrix(w, out, inner, like, "w"), out
    if w.device != like.device:
        raise ValueError(f"w is on {w.device}, x on {like.device}")
    if w.shape[0] != groups:
        raise ValueError(f"w holds {w.shape[0]} groups, offsets {groups}")
    apart, ld, last = w.stride()
    if last != 1 and inner != 1:
        raise ValueError(f"w: last stride {last}, 1 expected")
    if out == 1:
        ld = apart      # a group's one row may hold any stride
    if groups > 1 and apart != out * ld:
        raise ValueError("w: the groups have to follow each other without a gap")
    return (ld if groups > 1 or out > 1 else max(ld, inner)), out


def _groups(offsets, like):
    if offsets.dtype != _I64 or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"offsets is {offsets.dtype} {tuple(offsets.shape)}: torch.int64 (groups + 1,) expected")
    if offsets.device != like.device or not offsets.is_contiguous():
        raise ValueError(f"offsets has to be contiguous and on {like.device}")
    return offsets.shape[0] - 1


def _optional(t):
    return None if t is None else t.data_ptr()


def _on_gpu(x):
    if not x.is_cuda:
        raise ValueError(f"x is on {x.device}: the kernels need a GPU tensor")


def _launch(call, x, stream, *args):
    """call(stream handle, x, *args) with the tensors it makes, workspaces
    among them, belonging to the stream and the device of x."""
    device = x.get_device()
    if device < 0:
        return call(0, x, *args)      # the checks of the other arguments, then _on_gpu's refusal
    if stream is not None:
        if stream.device != x.device:
            raise ValueError(f"stream is on {stream.device}, x on {x.device}")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream, x, *args)
    if device != _current_device():
        with torch.cuda.device(device):
            return call(_raw_stream(device), x, *args)
    return call(_raw_stream(device), x, *args)


def _scratch(ws, like):
    """Checks a caller's workspace: the library sees its address and size alone."""
    if ws is not None and (ws.device != like.device or not ws.is_contiguous()):
        raise ValueError(f"workspace has to be contiguous and on {like.device}")


def _workspace(ws, need, device):
    if ws is None:
        return _empty(need, dtype=_U8, device=device), need
    return ws, ws.numel() * ws.element_size()


def _norm_fwd(s, x, gamma, beta, eps, y, mean, rstd):
    t = _type(x)
    rows, width = x.shape
    ldx, device = _matrix(x, rows, width, x, "x"), x.device
    g = _vector(gamma, (width,), x, "gamma")
    b = _vector(beta, (width,), x, "beta")
    _on_gpu(x)
    if y is None:
        y, ldy = _empty(rows, width, dtype=x.dtype, device=device), width
    else:
        ldy = _matrix(y, rows, width, x, "y")
    if mean is None:
        mean = _empty(rows, dtype=_F32, device=device)
    if rstd is None:
        rstd = _empty(rows, dtype=_F32, device=device)
    st = lib().gs_layer_norm_fwd(x.data_ptr(), ldx, g, b, rows, width, eps, t, y.data_ptr(), ldy,
                                 _vector(mean, (rows,), x, "mean"), _vector(rstd, (rows,), x, "rstd"), s)
    if st:
        _check(st, "gs_layer_norm_fwd")
    return y, mean, rstd


def gs_layer_norm_fwd(x, gamma=None, beta=None, eps=1e-5, y=None, mean=None, rstd=None, stream=None):
    """y, mean and rstd of the rows of ``x`` (``mean``, ``rstd``: [rows]
    float32, what the backward pass reads)."""
    return _launch(_norm_fwd, x, stream, gamma, beta, eps, y, mean, rstd)


def _norm_bwd(s, x, dy, gamma, mean, rstd, dres, dx, dgamma, dbeta, workspace):
    t = _type(x)
    rows, width = x.shape
    ldx, device = _matrix(x, rows, width, x, "x"), x.device
    lddy = _matrix(dy, rows, width, x, "dy")
    ldr = 0 if dres is None else _matrix(dres, rows, width, x, "dres")
    if mean is None or rstd is None:
        raise ValueError("the backward pass reads the forward's mean and rstd")
    _scratch(workspace, x)
    _on_gpu(x)
    if dx is None:
        dx, lddx = _empty(rows, width, dtype=x.dtype, device=device), width
    else:
        lddx = _matrix(dx, rows, width, x, "dx")
    if dgamma is None:
        dgamma = _empty(width, dtype=_F32, device=device)
    if dbeta is None:
        dbeta = _empty(width, dtype=_F32, device=device)
    ws, nbytes = _workspace(workspace, gs_workspace_size(GS_OP_LAYER_NORM_BWD, rows, width), device)
    st = lib().gs_layer_norm_bwd(x.data_ptr(), ldx, dy.data_ptr(), lddy, _vector(gamma, (width,), x, "gamma"),
                                 _vector(mean, (rows,), x, "mean"), _vector(rstd, (rows,), x, "rstd"),
                                 _optional(dres), ldr, rows, width, t, dx.data_ptr(), lddx,
                                 _vector(dgamma, (width,), x, "dgamma"), _vector(dbeta, (width,), x, "dbeta"),
                                 ws.data_ptr(), nbytes, s)
    if st:
        _check(st, "gs_layer_norm_bwd")
    return dx, dgamma, dbeta


def gs_layer_norm_bwd(x, dy, gamma, mean, rstd, dres=None, dx=None, dgamma=None, dbeta=None, workspace=None,
                      stream=None):
    """(dx, dgamma, dbeta); ``dres`` is added into dx (the gradient that
    reaches x past the norm)."""
    return _launch(_norm_bwd, x, stream, dy, gamma, mean, rstd, dres, dx, dgamma, dbeta, workspace)


def _fwd(s, x, w, offsets, bias, act, residual, y, z, save_z):
    t = _type(x)
    rows, inner = x.shape
    ldx, device = _matrix(x, rows, inner, x, "x"), x.device
    groups = 0 if offsets is None else _groups(offsets, x)
    ldw, out = _weights(w, groups, x, inner)
    b = _vector(bias, (groups, out) if groups else (out,), x, "bias")
    ldr = 0 if residual is None else _matrix(residual, rows, out, x, "residual")
    _on_gpu(x)
    if y is None:
        y, ldy = _empty(rows, out, dtype=x.dtype, device=device), out
    else:
        ldy = _matrix(y, rows, out, x, "y")
    if z is not None:
        ldz = _matrix(z, rows, out, x, "z")
    elif save_z:
        z, ldz = _empty(rows, out, dtype=x.dtype, device=device), out
    else:
        ldz = 0
    if groups:
        st = lib().gs_grouped_linear_fwd(x.data_ptr(), ldx, w.data_ptr(), ldw, b, offsets.data_ptr(), groups,
                                         _optional(residual), ldr, rows, inner, out, t, act, y.data_ptr(), ldy,
                                         _optional(z), ldz, s)
    else:
        st = lib().gs_linear_fwd(x.data_ptr(), ldx, w.data_ptr(), ldw, b, _optional(residual), ldr, rows, inner, out,
                                 t, act, y.data_ptr(), ldy, _optional(z), ldz, s)
    if st:
        _check(st, "gs_grouped_linear_fwd" if groups else "gs_linear_fwd")
    return y if z is None else (y, z)


def gs_linear_fwd(x, w, bias=None, act=GS_ACT_NONE, residual=None, y=None, z=None, save_z=False, stream=None):
    """y = act(x w^T + bias) + residual; with ``save_z`` (or a ``z`` to
    write) also the value before the activation: (y, z)."""
    return _launch(_fwd, x, stream, w, None, bias, act, residual, y, z, save_z)


def gs_grouped_linear_fwd(x, w, offsets, bias=None, act=GS_ACT_NONE, residual=None, y=None, z=None, save_z=False,
                          stream=None):
    """gs_linear_fwd with w[e], bias[e] for the rows offsets[e] ..
    offsets[e + 1] - 1 (``offsets``: int64 on the device, read there).
    Rows in no group are not written."""
    return _launch(_fwd, x, stream, w, offsets, bias, act, residual, y, z, save_z)


def gs_linear_workspace_size(rows, inner, out, num_groups, type, act) -> int:
    b = _size_t(0)
    _check(lib().gs_linear_workspace_size(rows, inner, out, num_groups, type, act, _byref(b)),
           "gs_linear_workspace_size")
    return b.value


def _bwd(s, x, w, offsets, dy, z, act, dx, dw, db, want_dx, workspace, want_dw):
    t = _type(x)
    rows, inner = x.shape
    ldx, device = _matrix(x, rows, inner, x, "x"), x.device
    groups = 0 if offsets is None else _groups(offsets, x)
    ldw, out = _weights(w, groups, x, inner)
    lddy = _matrix(dy, rows, out, x, "dy")
    if z is None and act != GS_ACT_NONE:
        raise ValueError("the activation's slope needs z, the value before it")
    ldz = 0 if z is None else _matrix(z, rows, out, x, "z")
    _scratch(workspace, x)
    _on_gpu(x)
    if dx is not None:
        lddx = _matrix(dx, rows, inner, x, "dx")
    elif want_dx:
        dx, lddx = _empty(rows, inner, dtype=x.dtype, device=device), inner
    else:
        lddx = 0
    dw_type = t
    if dw is None:
        if want_dw:
            dw = _empty(w.shape, dtype=w.dtype, device=device)
    else:
        dw_type = 2 if dw.dtype == _F32 else t
        if (dw.shape != w.shape or dw.dtype not in (w.dtype, _F32) or not dw.is_contiguous()
                or dw.device != device):
            raise ValueError(f"dw is {dw.dtype} {tuple(dw.shape)}: contiguous {w.dtype} or torch.float32 "
                             f"{tuple(w.shape)} on {device} expected")
    bshape = (groups, out) if groups else (out,)
    if db is None and want_dw:
        db = _empty(bshape, dtype=_F32, device=device)
    ws, nbytes = _workspace(workspace, gs_linear_workspace_size(rows, inner, out, groups, t, act), device)
    head = (x.data_ptr(), ldx, w.data_ptr(), ldw)
    tail = (_optional(z), ldz, dy.data_ptr(), lddy, rows, inner, out, t, act, _optional(dx), lddx, _optional(dw),
            dw_type, _vector(db, bshape, x, "db"), ws.data_ptr(), nbytes, s)
    if groups:
        st = lib().gs_grouped_linear_bwd(*head, offsets.data_ptr(), groups, *tail)
    else:
        st = lib().gs_linear_bwd(*head, *tail)
    if st:
        _check(st, "gs_grouped_linear_bwd" if groups else "gs_linear_bwd")
    return dx, dw, db


def gs_linear_bwd(x, w, dy, z=None, act=GS_ACT_NONE, dx=None, dw=None, db=None, want_dx=True, workspace=None,
                  stream=None, want_dw=True):
    """(dx, dw, db) of gs_linear_fwd for the gradient ``dy`` of y (the
    residual's gradient is dy itself).  ``dw`` is of w's type, or float32
    where such a tensor is passed in; ``want_dx`` false leaves dx out,
    ``want_dw`` false (frozen weights) dw and db, unless they are passed in."""
    return _launch(_bwd, x, stream, w, None, dy, z, act, dx, dw, db, want_dx, workspace, want_dw)


def gs_grouped_linear_bwd(x, w, offsets, dy, z=None, act=GS_ACT_NONE, dx=None, dw=None, db=None, want_dx=True,
                          workspace=None, stream=None, want_dw=True):
    """(dx, dw, db) of gs_grouped_linear_fwd; dw[e] and db[e] are 0 for an
    empty group, rows in no group have no dx."""
    return _launch(_bwd, x, stream, w, offsets, dy, z, act, dx, dw, db, want_dx, workspace, want_dw)
