"""AdamW over a network's tensors in one launch, moments in 32 or in 8 bits.

``gs_adamw`` carries the C entry point's name (``include/gs.h``) and takes
lists of tensors; ``AdamW`` keeps the moments and what a call has to know
about them, as a training program does.  Parameters are contiguous float32
tensors on one GPU; gradients bfloat16, float16 or float32; ``copies`` are the
16-bit (or float32) tensors that kernels read in the parameters' place, written
in the same pass.  Errors as in the network operators: ``ValueError`` or
``GSError``, before any work is enqueued.
"""
from __future__ import annotations

import array
from operator import attrgetter

import torch

from . import GS_ADAMW_BLOCK, _check, lib
from .network import _F32, _I64, _TYPES, _U8, _launch, _on_gpu

# a gs_adamw_tensor as 64-bit words: param, grad, m, v, m_scale, v_scale, copy,
# n, grad_type below copy_type
_WORDS, _GRAD, _COUNT, _KINDS = 9, 1, 7, 8
_address, _dense = torch.Tensor.data_ptr, torch.Tensor.is_contiguous
_nbytes, _dtype = attrgetter("nbytes"), attrgetter("dtype")


def _blocks(n):
    return -(-n // GS_ADAMW_BLOCK)


def _tensor(t, dtypes, n, device, name):
    """The address of a contiguous tensor of n elements."""
    if t.dtype not in dtypes or t.numel() != n:
        raise ValueError(f"{name} is {t.dtype} of {t.numel()} elements: {' or '.join(map(str, dtypes))} of {n} expected")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} has to be contiguous and on {device}")
    return t.data_ptr()


def _entry(table, i, device, param, m, v, m_scale, v_scale, copy):
    """Appends tensor i without a gradient; returns its copy's type as the upper
    half of the last word."""
    n = param.numel()
    if (m_scale is None) != (v_scale is None):
        raise ValueError(f"parameter {i}: one scale of two")
    kinds = (_F32,) if m_scale is None else (_U8,)
    table.append(_tensor(param, (_F32,), n, device, f"parameter {i}"))
    table.append(0)
    table.append(_tensor(m, kinds, n, device, f"m of parameter {i}"))
    table.append(_tensor(v, kinds, n, device, f"v of parameter {i}"))
    for name, scale in (("m", m_scale), ("v", v_scale)):
        table.append(0 if scale is None else
                     _tensor(scale, (_F32,), _blocks(n), device, f"{name}'s scales of parameter {i}"))
    table.append(0 if copy is None else _tensor(copy, tuple(_TYPES), n, device, f"copy of parameter {i}"))
    kind = 0 if copy is None else _TYPES[copy.dtype] << 32
    table.extend((0, kind))
    return kind


def _grads(table, device, sizes, kinds, grads):
    """Fills in the gradients; None: nothing is done for that tensor."""
    at, index = 0, device.index
    for i, g in enumerate(grads):
        if g is None:
            table[at + _COUNT] = 0
        else:
            n, t = sizes[i], _TYPES.get(g.dtype)
            if t is None or g.numel() != n or g.get_device() != index or not g.is_contiguous():
                _tensor(g, tuple(_TYPES), n, device, f"gradient {i}")       # says what is wrong, if it is
            table[at + _GRAD] = g.data_ptr()
            table[at + _COUNT] = n
            table[at + _KINDS] = kinds[i] + t
        at += _WORDS


def _scalar(t, dtype, device, name):
    return None if t is None else _tensor(t, (dtype,), 1, device, name)


def _call(s, first, table, count, numbers, step, grad_scale, seed):
    device = first.device
    step_at = _scalar(step, _I64, device, "step") if isinstance(step, torch.Tensor) else None
    scale_at = _scalar(grad_scale, _F32, device, "grad_scale")
    _on_gpu(first, "parameter 0")
    st = lib().gs_adamw(table.buffer_info()[0], count, *numbers, 0 if step_at is not None else step, step_at, scale_at,
                        seed, s)
    if st:
        _check(st, "gs_adamw")


def gs_adamw(params, grads, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, m_scales=None,
             v_scales=None, copies=None, grad_scale=None, seed=0, stream=None):
    """One AdamW step, in place, over lists of tensors: ``params`` float32,
    ``grads`` (an entry may be None: that tensor is left as it is), moments
    ``m`` and ``v`` (float32, or uint8 codes where ``m_scales[i]`` and
    ``v_scales[i]``, float32 of one for each 256 values, are given), ``copies``
    (entries may be None).  ``step`` counts from 1 on: a number, or a device
    int64 tensor read there (for a captured call).  ``grad_scale``: device
    float32, times which the gradients are taken.  ``seed`` fixes the random
    rounding of moments in 8 bits."""
    count = len(params)
    none = [None] * count
    lists = (grads, m, v, m_scales or none, v_scales or none, copies or none)
    if any(len(x) != count for x in lists):
        raise ValueError(f"{count} parameters with lists of {[len(x) for x in lists]}")
    if count == 0:
        return
    table, device = array.array("Q"), params[0].device
    kinds = [_entry(table, i, device, *row) for i, row in enumerate(zip(params, *lists[1:]))]
    _grads(table, device, [p.numel() for p in params], kinds, grads)
    _launch(_call, params[0], stream, table, count, (lr, beta1, beta2, eps, weight_decay), step, grad_scale, seed)


def _moment(s, codes, scales, moment, dtype, values):
    n, t, index = codes.numel(), _TYPES.get(dtype), codes.get_device()
    if t is None:
        raise ValueError(f"values of {dtype}: bfloat16, float16 or float32 expected")
    if codes.dtype is not _U8 or not codes.is_contiguous():
        _tensor(codes, (_U8,), n, codes.device, "codes")
    if (scales.dtype is not _F32 or scales.numel() != -(-n // GS_ADAMW_BLOCK) or scales.get_device() != index
            or not scales.is_contiguous()):
        _tensor(scales, (_F32,), _blocks(n), codes.device, "scales")
    if index < 0:
        _on_gpu(codes, "codes")
    if values is None:
        values = torch.empty_like(codes, dtype=dtype)
    else:
        _tensor(values, (dtype,), n, codes.device, "values")
    st = lib().gs_adamw_moment(codes.data_ptr(), scales.data_ptr(), n, moment, t, values.data_ptr(), s)
    if st:
        _check(st, "gs_adamw_moment")
    return values


def gs_adamw_moment(codes, scales, moment, dtype=torch.float32, values=None, stream=None):
    """The values (of ``dtype``, in codes' shape) of a moment in 8 bits:
    ``moment`` 1 for m, 2 for v."""
    return _launch(_moment, codes, stream, scales, moment, dtype, values)


class AdamW:
    """The optimiser of a list of float32 parameters.

    ``bits`` 8 holds the moments of tensors of at least ``min_8bit`` elements
    in 8 bits (2 bytes a parameter instead of 8); ``copies[i]`` (or None) is
    written with parameter i's new values.  ``capturable`` keeps the step's
    number on the device, so that a captured ``step`` counts on with each
    replay (``steps``, on the host, does not; without it a capture is refused);
    ``lr`` and the other numbers, which may be set between steps, stay those of
    the capture.
    ``state``: (m, v, m_scale, v_scale) of each tensor to go on from, taken as
    they are (scales None for moments in 32 bits), ``step`` the number of steps
    done.  ``params``, ``copies`` and ``state`` stay the tensors that they are
    from then on; a tensor's storage may be replaced (its ``.data``), and each
    step looks at all of them again."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, bits=32, min_8bit=4096,
                 copies=None, seed=0, capturable=False, state=None, step=0):
        self._params = tuple(params)
        if not self._params:
            raise ValueError("no parameters")
        if bits not in (8, 32):
            raise ValueError(f"bits = {bits}: 8 or 32 expected")
        self.lr, self.betas, self.eps, self.weight_decay, self.seed = lr, betas, eps, weight_decay, seed
        count, device = len(self.params), self.params[0].device
        self._copies = (None,) * count if copies is None else tuple(copies)
        if state is None:
            state = []
            for p in self.params:
                n = p.numel()
                if bits == 8 and n >= min_8bit:
                    state.append(tuple(torch.zeros(n, dtype=_U8, device=device) for _ in range(2))
                                 + tuple(torch.zeros(_blocks(n), device=device) for _ in range(2)))
                else:
                    state.append((torch.zeros(n, device=device), torch.zeros(n, device=device), None, None))
        self._state = tuple(tuple(s) for s in state)
        if len(self.copies) != count or len(self.state) != count:
            raise ValueError(f"{count} parameters, {len(self.copies)} copies, {len(self.state)} states")
        self.steps = step
        # the next step's number: counted on behind a call that was taken
        self.step_dev = torch.tensor([step + 1], dtype=_I64, device=device) if capturable else None
        rows = zip(self.params, self.copies, self.state)
        self._tensors = [t for p, c, s in rows for t in (p, c, *s) if t is not None]
        self._typed = [c for c in self.copies if c is not None]
        self._table, self._held, self._sizes, self._kinds, self._given = None, None, None, None, None

    params = property(attrgetter("_params"))
    copies = property(attrgetter("_copies"))
    state = property(attrgetter("_state"))

    def step(self, grads=None, grad_scale=None, stream=None):
        """One step with ``grads`` (default: each parameter's .grad; None leaves
        a tensor as it is), times the device float32 ``grad_scale``."""
        grads = [p.grad for p in self.params] if grads is None else grads
        count, device = len(self.params), self.params[0].device
        if len(grads) != count:
            raise ValueError(f"{len(grads)} gradients of {count} parameters")
        # the tensors as they are now: storage or layout may have been replaced
        # (float32 and codes go by their bytes alone, a copy by its type too)
        held = [*map(_address, self._tensors), *map(_nbytes, self._tensors), *map(_dense, self._tensors),
                *map(_dtype, self._typed)]
        if held != self._held:
            table = array.array("Q")
            self._kinds = [_entry(table, i, device, p, *s, c)
                           for i, (p, s, c) in enumerate(zip(self.params, self.state, self.copies))]
            self._table, self._held, self._sizes = table, held, [p.numel() for p in self.params]
            self._given = None
        # gradients that are filled where they were have their entries (an address
        # is of one device)
        try:
            given = [*map(_address, grads), *map(_nbytes, grads), *map(_dense, grads), *map(_dtype, grads)]
        except TypeError:       # None among them
            given = None
        if given is None or given != self._given:
            self._given = None
            _grads(self._table, device, self._sizes, self._kinds, grads)
            self._given = given
        numbers = (self.lr, *self.betas, self.eps, self.weight_decay)
        _launch(self._enqueue, self.params[0], stream, numbers, grad_scale)
        self.steps += 1

    def _enqueue(self, s, first, numbers, grad_scale):
        _on_gpu(first, "parameter 0")
        if self.step_dev is None and torch.cuda.is_current_stream_capturing():
            raise ValueError("a captured step would stay the same step in every replay: make the AdamW capturable")
        step = self.steps + 1 if self.step_dev is None else self.step_dev
        _call(s, first, self._table, len(self.params), numbers, step, grad_scale, self.seed)
        if self.step_dev is not None:
            self.step_dev.add_(1)

    def state_dict(self):
        """The moments, as they are held, and the number of steps done."""
        steps = self.steps if self.step_dev is None else int(self.step_dev) - 1
        return {"state": [tuple(None if x is None else x.clone() for x in s) for s in self.state], "steps": steps}

    def load_state_dict(self, d):
        if len(d["state"]) != len(self.state):
            raise ValueError(f"state of {len(d['state'])} tensors for {len(self.state)}")
        for mine, theirs in zip(self.state, d["state"]):
            if any((a is None) != (b is None) or (a is not None and (a.dtype != b.dtype or a.shape != b.shape))
                   for a, b in zip(mine, theirs)):
                raise ValueError("state of other sizes or bits")
        for mine, theirs in zip(self.state, d["state"]):
            for a, b in zip(mine, theirs):
                if a is not None:
                    a.copy_(b)
        self.steps = int(d["steps"])
        if self.step_dev is not None:
            self.step_dev.fill_(self.steps + 1)
