"""The network operators of libgs: layer norm, the linear layer with bias,
activation and residual in its epilogue, the linear layer whose weights
go by ragged group, rows looked up in a shared table, the gate that picks
groups for a row, rows brought to their groups and back, each forward and
backward, and the sort by group that ragged groups are made by.

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
_F32, _I32, _I64, _U8 = torch.float32, torch.int32, torch.int64, torch.uint8
_ID_BYTES = {_I32: 4, _I64: 8}
_empty = torch.empty
_byref, _size_t = C.byref, C.c_size_t
# the stream's handle without a Stream object, where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


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


def _on_gpu(x, name="x"):
    if not x.is_cuda:
        raise ValueError(f"{name} is on {x.device}: the kernels need a GPU tensor")


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
    if ws is None and need == 0:
        return None, 0
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


# --- shared features and routed rows ---------------------------------------------

def _ids(ids, like_device, name="ids", dims=None):
    """(address, bytes of an element) of a contiguous int32 or int64 tensor."""
    if ids.dtype not in _ID_BYTES or (dims is not None and ids.dim() != dims):
        raise ValueError(f"{name} is {ids.dtype} with {ids.dim()} dimensions: torch.int32 or torch.int64"
                         f"{'' if dims is None else f' with {dims}'} expected")
    if ids.device != like_device or not ids.is_contiguous():
        raise ValueError(f"{name} has to be contiguous and on {like_device}")
    return ids.data_ptr(), _ID_BYTES[ids.dtype]


def _whole(t, dtype, shape, device, name):
    """t, or a new tensor; [rows] and [rows][k] arrays of one element type."""
    if t is None:
        return _empty(shape, dtype=dtype, device=device)
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}: {dtype} {tuple(shape)} expected")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} has to be contiguous and on {device}")
    return t


def gs_group_sort_workspace_size(n, num_groups) -> int:
    b = _size_t(0)
    _check(lib().gs_group_sort_workspace_size(n, num_groups, _byref(b)), "gs_group_sort_workspace_size")
    return b.value


def _group_sort(s, ids, num_groups, offsets, order, place, want_order, want_place, workspace):
    device, n = ids.device, ids.numel()
    at, id_bytes = _ids(ids, device)
    _scratch(workspace, ids)
    need = gs_group_sort_workspace_size(n, num_groups)
    if not ids.is_cuda:
        raise ValueError(f"ids is on {device}: the kernels need a GPU tensor")
    offsets = _whole(offsets, _I64, (num_groups + 1,), device, "offsets")
    if order is not None or want_order:
        order = _whole(order, _I32, (n,), device, "order")
    if place is not None or want_place:
        place = _whole(place, _I32, ids.shape, device, "place")
    ws, nbytes = _workspace(workspace, need, device)
    st = lib().gs_group_sort(at, id_bytes, n, num_groups, offsets.data_ptr(), _optional(order), _optional(place),
                             _optional(ws), nbytes, s)
    if st:
        _check(st, "gs_group_sort")
    return offsets, order, place


def gs_group_sort(ids, num_groups, offsets=None, order=None, place=None, want_order=True, want_place=True,
                  workspace=None, stream=None):
    """(offsets, order, place) of a stable sort of ``ids`` (int32 or int64, any
    shape) by group: ``offsets`` [num_groups + 1] int64 are the groups' bounds
    (what ``gs_grouped_linear_fwd`` reads), ``order`` [n] int32 the entry at
    each position, ``place`` (ids' shape, int32) each entry's position, -1 for
    an id outside [0, num_groups).  None for what is not wanted."""
    return _launch(_group_sort, ids, stream, num_groups, offsets, order, place, want_order, want_place, workspace)


def _embed_fwd(s, table, ids, scale, y):
    t = _type(table, "table")
    num_rows, width = table.shape
    ldt, device = _matrix(table, num_rows, width, table, "table"), table.device
    at, id_bytes = _ids(ids, device)
    rows = ids.numel()
    _on_gpu(table, "table")
    if y is None:
        y, ldy = _empty(rows, width, dtype=table.dtype, device=device), width
    else:
        ldy = _matrix(y, rows, width, table, "y")
    st = lib().gs_embedding_fwd(table.data_ptr(), ldt, num_rows, at, id_bytes, rows, width, scale, t, y.data_ptr(),
                                ldy, s)
    if st:
        _check(st, "gs_embedding_fwd")
    return y


def gs_embedding_fwd(table, ids, scale=1.0, y=None, stream=None):
    """y[i] = scale table[ids[i]] ([ids.numel()][width]; ``ids`` int32 or
    int64); a row of zeros for an id outside the table."""
    return _launch(_embed_fwd, table, stream, ids, scale, y)


def gs_embedding_workspace_size(rows, num_rows, width, type) -> int:
    b = _size_t(0)
    _check(lib().gs_embedding_workspace_size(rows, num_rows, width, type, _byref(b)), "gs_embedding_workspace_size")
    return b.value


def _embed_bwd(s, dy, ids, offsets, order, scale, dtable, workspace):
    t = _type(dy, "dy")
    rows, width = dy.shape
    lddy, device = _matrix(dy, rows, width, dy, "dy"), dy.device
    at, id_bytes = _ids(ids, device)
    if ids.numel() != rows:
        raise ValueError(f"ids holds {ids.numel()} entries, dy {rows} rows")
    num_rows = _groups(offsets, dy)
    if order is None:
        raise ValueError("the backward pass reads gs_group_sort's order")
    _whole(order, _I32, (rows,), device, "order")
    _scratch(workspace, dy)
    need = gs_embedding_workspace_size(rows, num_rows, width, t)
    _on_gpu(dy, "dy")
    dt_type = t
    if dtable is None:
        dtable, lddt = _empty(num_rows, width, dtype=dy.dtype, device=device), width
    else:
        dt_type = 2 if dtable.dtype == _F32 else t
        if dt_type == t:
            lddt = _matrix(dtable, num_rows, width, dy, "dtable")
        else:
            if dtable.device != device:
                raise ValueError(f"dtable is on {dtable.device}, dy on {device}")
            lddt = _matrix(dtable, num_rows, width, dtable, "dtable")
    ws, nbytes = _workspace(workspace, need, device)
    st = lib().gs_embedding_bwd(dy.data_ptr(), lddy, at, id_bytes, offsets.data_ptr(), order.data_ptr(), rows,
                                num_rows, width, scale, t, dtable.data_ptr(), lddt, dt_type, ws.data_ptr(), nbytes, s)
    if st:
        _check(st, "gs_embedding_bwd")
    return dtable


def gs_embedding_bwd(dy, ids, offsets, order, scale=1.0, dtable=None, workspace=None, stream=None):
    """dtable of gs_embedding_fwd for the gradient ``dy`` of y; ``offsets`` and
    ``order`` are those of ``gs_group_sort(ids, rows of the table)``.
    ``dtable`` is of dy's type, or float32 where such a tensor is passed in;
    every row is written."""
    return _launch(_embed_bwd, dy, stream, ids, offsets, order, scale, dtable, workspace)


def _choices(t, dtype, rows, device, name, k=None):
    """k of t, a contiguous [rows][k] tensor."""
    if t.dtype != dtype or t.dim() != 2 or t.shape[0] != rows or (k is not None and t.shape[1] != k):
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}: {dtype} ({rows}, {'k' if k is None else k}) expected")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} has to be contiguous and on {device}")
    return t.shape[1]


def _gate_fwd(s, logits, k, renorm, ids, weights):
    t = _type(logits, "logits")
    rows, groups = logits.shape
    ld, device = _matrix(logits, rows, groups, logits, "logits"), logits.device
    _on_gpu(logits, "logits")
    if not 1 <= k <= groups:
        raise ValueError(f"k = {k} of {groups} groups")
    ids = _whole(ids, _I32, (rows, k), device, "ids")
    weights = _whole(weights, _F32, (rows, k), device, "weights")
    st = lib().gs_gate_fwd(logits.data_ptr(), ld, rows, groups, k, 1 if renorm else 0, t, ids.data_ptr(),
                           weights.data_ptr(), s)
    if st:
        _check(st, "gs_gate_fwd")
    return ids, weights


def gs_gate_fwd(logits, k, renorm=True, ids=None, weights=None, stream=None):
    """(ids, weights), [rows][k] int32 and float32: each row's k largest logits
    and their softmax over themselves (``renorm``) or over the whole row.  A
    logit of minus infinity is never chosen; -1 and 0 where no other is left."""
    return _launch(_gate_fwd, logits, stream, k, renorm, ids, weights)


def _gate_bwd(s, logits, ids, weights, dweights, renorm, dlogits):
    t = _type(logits, "logits")
    rows, groups = logits.shape
    ld, device = _matrix(logits, rows, groups, logits, "logits"), logits.device
    k = _choices(ids, _I32, rows, device, "ids")
    _choices(weights, _F32, rows, device, "weights", k)
    _choices(dweights, _F32, rows, device, "dweights", k)
    _on_gpu(logits, "logits")
    if dlogits is None:
        dlogits, lddl = _empty(rows, groups, dtype=logits.dtype, device=device), groups
    else:
        lddl = _matrix(dlogits, rows, groups, logits, "dlogits")
    st = lib().gs_gate_bwd(logits.data_ptr(), ld, ids.data_ptr(), weights.data_ptr(), dweights.data_ptr(), rows,
                           groups, k, 1 if renorm else 0, t, dlogits.data_ptr(), lddl, s)
    if st:
        _check(st, "gs_gate_bwd")
    return dlogits


def gs_gate_bwd(logits, ids, weights, dweights, renorm=True, dlogits=None, stream=None):
    """dlogits of gs_gate_fwd, whose ``ids`` and ``weights`` it reads, for the
    gradient ``dweights`` of the weights.  A choice that is left out afterwards
    loses its place (-1), not its id: gs_combine_bwd's dweight for it is 0."""
    return _launch(_gate_bwd, logits, stream, ids, weights, dweights, renorm, dlogits)


def _dispatch_fwd(s, x, place, xs):
    t = _type(x)
    rows, width = x.shape
    ldx, device = _matrix(x, rows, width, x, "x"), x.device
    k = _choices(place, _I32, rows, device, "place")
    _on_gpu(x)
    if xs is None:
        xs, ldxs = _empty(rows * k, width, dtype=x.dtype, device=device), width
    else:
        ldxs = _matrix(xs, rows * k, width, x, "xs")
    st = lib().gs_dispatch_fwd(x.data_ptr(), ldx, place.data_ptr(), rows, k, width, t, xs.data_ptr(), ldxs, s)
    if st:
        _check(st, "gs_dispatch_fwd")
    return xs


def gs_dispatch_fwd(x, place, xs=None, stream=None):
    """xs [rows k][width] with xs[place[i][j]] = x[i]; ``place`` is
    gs_group_sort's of [rows][k] ids.  Rows behind the last group are not written."""
    return _launch(_dispatch_fwd, x, stream, place, xs)


def _back(s, x, place, weights, residual, y, weighted):
    """gs_combine_fwd of x = ys, or gs_dispatch_bwd of x = dxs."""
    name = "ys" if weighted else "dxs"
    t = _type(x, name)
    many, width = x.shape
    ldx, device = _matrix(x, many, width, x, name), x.device
    rows = place.shape[0] if place.dim() == 2 else -1
    k = _choices(place, _I32, rows, device, "place")
    if many != rows * k:
        raise ValueError(f"{name} has {many} rows, place {rows} x {k}")
    if weights is not None:
        _choices(weights, _F32, rows, device, "weights", k)
    ldr = 0 if residual is None else _matrix(residual, rows, width, x, "residual" if weighted else "dres")
    _on_gpu(x, name)
    if y is None:
        y, ldy = _empty(rows, width, dtype=x.dtype, device=device), width
    else:
        ldy = _matrix(y, rows, width, x, "y" if weighted else "dx")
    if weighted:
        st = lib().gs_combine_fwd(x.data_ptr(), ldx, place.data_ptr(), _optional(weights), _optional(residual), ldr,
                                  rows, k, width, t, y.data_ptr(), ldy, s)
    else:
        st = lib().gs_dispatch_bwd(x.data_ptr(), ldx, place.data_ptr(), rows, k, width, t, _optional(residual), ldr,
                                   y.data_ptr(), ldy, s)
    if st:
        _check(st, "gs_combine_fwd" if weighted else "gs_dispatch_bwd")
    return y


def gs_dispatch_bwd(dxs, place, dres=None, dx=None, stream=None):
    """dx[i] = sum_j dxs[place[i][j]] (+ dres[i], the gradient that reaches x
    past the heads)."""
    return _launch(_back, dxs, stream, place, None, dres, dx, False)


def gs_combine_fwd(ys, place, weights=None, residual=None, y=None, stream=None):
    """y[i] = sum_j weights[i][j] ys[place[i][j]] (+ residual[i]); places that
    were left out (-1) add nothing."""
    return _launch(_back, ys, stream, place, weights, residual, y, True)


def _combine_bwd(s, dy, ys, place, weights, dys, dweights, want_dys, want_dw):
    t = _type(dy, "dy")
    rows, width = dy.shape
    lddy, device = _matrix(dy, rows, width, dy, "dy"), dy.device
    k = _choices(place, _I32, rows, device, "place")
    if weights is not None:
        _choices(weights, _F32, rows, device, "weights", k)
    if dweights is not None:
        _choices(dweights, _F32, rows, device, "dweights", k)
    want_dw = want_dw or dweights is not None
    if ys is None and want_dw:
        raise ValueError("the weights' gradient reads ys")
    ldys = 0 if ys is None else _matrix(ys, rows * k, width, dy, "ys")
    _on_gpu(dy, "dy")
    if dys is not None:
        lddys = _matrix(dys, rows * k, width, dy, "dys")
    elif want_dys:
        dys, lddys = _empty(rows * k, width, dtype=dy.dtype, device=device), width
    else:
        lddys = 0
    if dweights is None and want_dw:
        dweights = _empty(rows, k, dtype=_F32, device=device)
    st = lib().gs_combine_bwd(dy.data_ptr(), lddy, _optional(ys), ldys, place.data_ptr(), _optional(weights), rows, k,
                              width, t, _optional(dys), lddys, _optional(dweights), s)
    if st:
        _check(st, "gs_combine_bwd")
    return dys, dweights


def gs_combine_bwd(dy, ys, place, weights=None, dys=None, dweights=None, want_dys=True, want_dw=True, stream=None):
    """(dys, dweights) of gs_combine_fwd for the gradient ``dy`` of y (the
    residual's gradient is dy itself); rows of dys behind the last group are
    not written.  ``want_dw`` false leaves dweights out (``ys`` may be None
    then), ``want_dys`` false dys, unless they are passed in."""
    return _launch(_combine_bwd, dy, stream, ys, place, weights, dys, dweights, want_dys, want_dw)
