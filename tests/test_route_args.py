"""What the sort, the lookup and the other operators of shared features and
routed rows refuse, on the host (no GPU: nothing is launched on a refusal)."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

import differentiable_gaussian_splatting_dgs_amd as gs

P = C.c_void_p
F = C.c_float


def _sort(ids=P(16), id_bytes=4, n=10, groups=5, offsets=P(16), order=P(16), place=P(16), ws=P(256), ws_bytes=1 << 24):
    return gs.lib().gs_group_sort(ids, id_bytes, n, groups, offsets, order, place, ws, ws_bytes, None)


def _embed(table=P(16), ldt=64, num_rows=9, ids=P(16), id_bytes=8, rows=4, width=64, scale=1.0, typ=0, y=P(16), ldy=64):
    return gs.lib().gs_embedding_fwd(table, ldt, num_rows, ids, id_bytes, rows, width, F(scale), typ, y, ldy, None)


def _embed_bwd(dy=P(16), lddy=64, ids=P(16), id_bytes=8, offsets=P(16), order=P(16), rows=4, num_rows=9, width=64,
               scale=1.0, typ=0, dtable=P(16), lddt=64, dt_type=0, ws=P(256), ws_bytes=1 << 24):
    return gs.lib().gs_embedding_bwd(dy, lddy, ids, id_bytes, offsets, order, rows, num_rows, width, F(scale), typ,
                                     dtable, lddt, dt_type, ws, ws_bytes, None)


@pytest.mark.parametrize("call,kw,word", [
    (_sort, dict(n=-1), b"n ="), (_sort, dict(n=1 << 31), b"n ="), (_sort, dict(groups=0), b"num_groups"),
    (_sort, dict(groups=(1 << 30) + 1), b"num_groups"), (_sort, dict(id_bytes=2), b"id_bytes"),
    (_sort, dict(ids=None), b"ids"), (_sort, dict(ids=P(18)), b"ids"), (_sort, dict(ids=P(20), id_bytes=8), b"ids"),
    (_sort, dict(offsets=None), b"offsets"), (_sort, dict(offsets=P(12)), b"offsets"),
    (_sort, dict(order=P(18)), b"order"), (_sort, dict(place=P(17)), b"place"),
    (_sort, dict(n=100_000, ws=None), b"workspace"), (_sort, dict(ws=P(128)), b"workspace"),
    (_sort, dict(n=100_000, ws_bytes=256), b"workspace_bytes"),
    (_embed, dict(typ=3), b"type"), (_embed, dict(rows=-1), b"rows"), (_embed, dict(rows=1 << 31), b"rows"),
    (_embed, dict(num_rows=0), b"num_rows"), (_embed, dict(num_rows=(1 << 30) + 1), b"num_rows"),
    (_embed, dict(width=0), b"width"), (_embed, dict(width=65537), b"width"), (_embed, dict(ldt=63), b"table"),
    (_embed, dict(ldy=63), b"y"), (_embed, dict(table=None), b"table"), (_embed, dict(table=P(17)), b"table"),
    (_embed, dict(y=None), b"y"), (_embed, dict(ids=None), b"ids"), (_embed, dict(id_bytes=1), b"id_bytes"),
    (_embed, dict(scale=float("nan")), b"scale"), (_embed, dict(scale=float("inf")), b"scale"),
    (_embed_bwd, dict(typ=-1), b"type"), (_embed_bwd, dict(lddy=10), b"dy"), (_embed_bwd, dict(dy=None), b"dy"),
    (_embed_bwd, dict(ids=None), b"ids"), (_embed_bwd, dict(offsets=None), b"offsets"),
    (_embed_bwd, dict(offsets=P(20)), b"offsets"), (_embed_bwd, dict(order=None), b"order"),
    (_embed_bwd, dict(order=P(18)), b"order"), (_embed_bwd, dict(dt_type=1), b"dtable_type"),
    (_embed_bwd, dict(dtable=None), b"dtable"), (_embed_bwd, dict(lddt=63), b"dtable"),
    (_embed_bwd, dict(dtable=P(18), dt_type=2), b"dtable"), (_embed_bwd, dict(scale=float("nan")), b"scale"),
    (_embed_bwd, dict(ws=None), b"workspace"), (_embed_bwd, dict(ws=P(64)), b"workspace"),
    (_embed_bwd, dict(ws_bytes=0), b"workspace_bytes"),
])
def test_refused(call, kw, word):
    assert call(**kw) == gs.GS_ERR_INVALID_ARG
    assert word in gs.lib().gs_last_error(), gs.lib().gs_last_error()


def test_nothing_to_do():
    assert _embed(rows=0, table=None, y=None, ids=None) == gs.GS_OK


def test_workspace_sizes():
    for n in (0, 1, 2048, 1_000_000):
        for groups in (1, 1000, 100_000):
            assert gs.gs_group_sort_workspace_size(n, groups) >= (4 * n if groups > 10_000 else 0)
    assert gs.gs_group_sort_workspace_size(100, 64) == 0
    assert gs.gs_embedding_workspace_size(0, 1, 1, 0) >= 256
    with pytest.raises(gs.GSError, match="num_groups"):
        gs.gs_group_sort_workspace_size(4, 0)
    with pytest.raises(gs.GSError, match="width"):
        gs.gs_embedding_workspace_size(4, 4, 0, 0)


def _t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def _ids(*shape, dtype=torch.int64):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("call,match", [
    (lambda: gs.gs_group_sort(_t(4), 3), "int32 or torch.int64"),
    (lambda: gs.gs_group_sort(_ids(8)[::2], 3), "contiguous"),
    (lambda: gs.gs_group_sort(_ids(8), 3), "GPU tensor"),
    (lambda: gs.gs_embedding_fwd(_t(4), _ids(3)), "dimensions"),
    (lambda: gs.gs_embedding_fwd(_t(4, 8, dtype=torch.float64), _ids(3)), "float64"),
    (lambda: gs.gs_embedding_fwd(_t(4, 8).t(), _ids(3)), "stride"),
    (lambda: gs.gs_embedding_fwd(_t(4, 8), _t(3)), "int32"),
    (lambda: gs.gs_embedding_fwd(_t(4, 8), _ids(3)), "GPU tensor"),
    (lambda: gs.gs_embedding_bwd(_t(4, 8), _ids(3), _ids(10), _ids(4, dtype=torch.int32)), "entries"),
    (lambda: gs.gs_embedding_bwd(_t(4, 8), _ids(4), _t(10), _ids(4, dtype=torch.int32)), "offsets"),
    (lambda: gs.gs_embedding_bwd(_t(4, 8), _ids(4), _ids(10), _ids(4)), "order"),
    (lambda: gs.gs_embedding_bwd(_t(4, 8), _ids(4), _ids(10), None), "order"),
    (lambda: gs.gs_embedding_bwd(_t(4, 8), _ids(4), _ids(10), _ids(4, dtype=torch.int32),
                                 workspace=_ids(64)[::2]), "workspace"),
    (lambda: gs.gs_embedding_bwd(_t(4, 8), _ids(4), _ids(10), _ids(4, dtype=torch.int32)), "GPU tensor"),
])
def test_binding_refuses(call, match):
    with pytest.raises(ValueError, match=match):
        call()


# --- the gate and routed rows ------------------------------------------------------

def _gate(logits=P(16), ld=64, rows=4, groups=64, k=2, renorm=1, typ=0, ids=P(16), weights=P(16)):
    return gs.lib().gs_gate_fwd(logits, ld, rows, groups, k, renorm, typ, ids, weights, None)


def _gate_bwd(logits=P(16), ld=64, ids=P(16), weights=P(16), dweights=P(16), rows=4, groups=64, k=2, renorm=1, typ=0,
              dlogits=P(16), lddl=64):
    return gs.lib().gs_gate_bwd(logits, ld, ids, weights, dweights, rows, groups, k, renorm, typ, dlogits, lddl, None)


def _dispatch(x=P(16), ldx=64, place=P(16), rows=4, k=2, width=64, typ=0, xs=P(16), ldxs=64):
    return gs.lib().gs_dispatch_fwd(x, ldx, place, rows, k, width, typ, xs, ldxs, None)


def _dispatch_bwd(dxs=P(16), ld=64, place=P(16), rows=4, k=2, width=64, typ=0, dres=None, ldr=0, dx=P(16), lddx=64):
    return gs.lib().gs_dispatch_bwd(dxs, ld, place, rows, k, width, typ, dres, ldr, dx, lddx, None)


def _combine(ys=P(16), ld=64, place=P(16), weights=P(16), res=None, ldr=0, rows=4, k=2, width=64, typ=0, y=P(16),
             ldy=64):
    return gs.lib().gs_combine_fwd(ys, ld, place, weights, res, ldr, rows, k, width, typ, y, ldy, None)


def _combine_bwd(dy=P(16), lddy=64, ys=P(16), ldys=64, place=P(16), weights=P(16), rows=4, k=2, width=64, typ=0,
                 dys=P(16), lddys=64, dw=P(16)):
    return gs.lib().gs_combine_bwd(dy, lddy, ys, ldys, place, weights, rows, k, width, typ, dys, lddys, dw, None)


@pytest.mark.parametrize("call,kw,word", [
    (_gate, dict(typ=3), b"type"), (_gate, dict(rows=-1), b"rows"), (_gate, dict(groups=0), b"groups"),
    (_gate, dict(groups=1025, ld=2000), b"groups"), (_gate, dict(k=0), b"k ="), (_gate, dict(k=17), b"k ="),
    (_gate, dict(groups=4, k=5), b"k ="), (_gate, dict(ld=63), b"logits"), (_gate, dict(logits=None), b"logits"),
    (_gate, dict(logits=P(17)), b"logits"), (_gate, dict(ids=None), b"ids"), (_gate, dict(ids=P(18)), b"ids"),
    (_gate, dict(weights=None), b"weights"), (_gate, dict(weights=P(18)), b"weights"),
    (_gate_bwd, dict(typ=-1), b"type"), (_gate_bwd, dict(k=0), b"k ="), (_gate_bwd, dict(dlogits=None), b"dlogits"),
    (_gate_bwd, dict(lddl=9), b"dlogits"), (_gate_bwd, dict(ld=9), b"logits"), (_gate_bwd, dict(ids=None), b"ids"),
    (_gate_bwd, dict(dweights=None), b"dweights"), (_gate_bwd, dict(dweights=P(18)), b"dweights"),
    (_dispatch, dict(typ=7), b"type"), (_dispatch, dict(rows=1 << 31), b"rows"), (_dispatch, dict(k=0), b"k ="),
    (_dispatch, dict(k=17), b"k ="), (_dispatch, dict(rows=1 << 30, k=2), b"rows"),
    (_dispatch, dict(width=0), b"width"), (_dispatch, dict(width=65537), b"width"), (_dispatch, dict(ldx=63), b"x"),
    (_dispatch, dict(ldxs=63), b"xs"), (_dispatch, dict(x=None), b"x"), (_dispatch, dict(xs=None), b"xs"),
    (_dispatch, dict(place=None), b"place"), (_dispatch, dict(place=P(18)), b"place"),
    (_dispatch_bwd, dict(dxs=None), b"dxs"), (_dispatch_bwd, dict(dx=None), b"dx"),
    (_dispatch_bwd, dict(dres=P(16), ldr=1), b"residual"), (_dispatch_bwd, dict(lddx=2), b"dx"),
    (_combine, dict(ys=None), b"ys"), (_combine, dict(y=None), b"y"), (_combine, dict(weights=P(18)), b"weights"),
    (_combine, dict(res=P(17), ldr=64), b"residual"), (_combine, dict(ldy=63), b"y"),
    (_combine, dict(res=P(16), ldr=65), b"in place"), (_dispatch_bwd, dict(dres=P(16), ldr=66), b"in place"),
    (_combine_bwd, dict(dy=None), b"dy"), (_combine_bwd, dict(ys=None), b"ys"), (_combine_bwd, dict(lddys=1), b"dys"),
    (_combine_bwd, dict(dw=P(18)), b"dweights"), (_combine_bwd, dict(place=None), b"place"),
])
def test_routing_refused(call, kw, word):
    assert call(**kw) == gs.GS_ERR_INVALID_ARG
    assert word in gs.lib().gs_last_error(), gs.lib().gs_last_error()


def test_routing_nothing_to_do():
    for call in (_gate, _gate_bwd, _dispatch, _dispatch_bwd, _combine, _combine_bwd):
        assert call(rows=0) == gs.GS_OK
    assert _combine_bwd(dys=None, dw=None) == gs.GS_OK


I4 = torch.int32


@pytest.mark.parametrize("call,match", [
    (lambda: gs.gs_gate_fwd(_t(4), 2), "dimensions"), (lambda: gs.gs_gate_fwd(_t(8, 4).t(), 2), "stride"),
    (lambda: gs.gs_gate_fwd(_t(4, 8), 2), "GPU tensor"),
    (lambda: gs.gs_gate_bwd(_t(4, 8), _ids(4, 2), _t(4, 2), _t(4, 2)), "ids"),
    (lambda: gs.gs_gate_bwd(_t(4, 8), _ids(4, 2, dtype=I4), _t(4, 3), _t(4, 2)), "weights"),
    (lambda: gs.gs_gate_bwd(_t(4, 8), _ids(4, 2, dtype=I4), _t(4, 2), _t(3, 2)), "dweights"),
    (lambda: gs.gs_gate_bwd(_t(4, 8), _ids(4, 2, dtype=I4), _t(4, 2), _t(4, 2)), "GPU tensor"),
    (lambda: gs.gs_dispatch_fwd(_t(4, 8), _ids(4, 2)), "place"),
    (lambda: gs.gs_dispatch_fwd(_t(4, 8), _ids(5, 2, dtype=I4)), "place"),
    (lambda: gs.gs_dispatch_fwd(_t(4, 8), _ids(4, dtype=I4)), "place"),
    (lambda: gs.gs_dispatch_fwd(_t(4, 8), _ids(4, 2, dtype=I4)), "GPU tensor"),
    (lambda: gs.gs_dispatch_bwd(_t(7, 8), _ids(4, 2, dtype=I4)), "rows"),
    (lambda: gs.gs_dispatch_bwd(_t(8, 8), _ids(4, 2, dtype=I4), dres=_t(4, 7)), "dres"),
    (lambda: gs.gs_dispatch_bwd(_t(8, 8), _ids(8, dtype=I4)), "place"),
    (lambda: gs.gs_dispatch_bwd(_t(8, 8), _ids(4, 2, dtype=I4)), "GPU tensor"),
    (lambda: gs.gs_combine_fwd(_t(9, 8), _ids(4, 2, dtype=I4)), "rows"),
    (lambda: gs.gs_combine_fwd(_t(8, 8), _ids(4, 2, dtype=I4), _t(4, 3)), "weights"),
    (lambda: gs.gs_combine_fwd(_t(8, 8), _ids(4, 2, dtype=I4), _t(2, 4).t()), "contiguous"),
    (lambda: gs.gs_combine_fwd(_t(8, 8), _ids(4, 2, dtype=I4)), "GPU tensor"),
    (lambda: gs.gs_combine_bwd(_t(4, 8), None, _ids(4, 2, dtype=I4)), "reads ys"),
    (lambda: gs.gs_combine_bwd(_t(4, 8), _t(7, 8), _ids(4, 2, dtype=I4)), "ys"),
    (lambda: gs.gs_combine_bwd(_t(4, 8), _t(8, 8), _ids(4, 2, dtype=I4)), "GPU tensor"),
])
def test_routing_binding_refuses(call, match):
    with pytest.raises(ValueError, match=match):
        call()


# --- AdamW -----------------------------------------------------------------------------

def _adamw(count=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, step=1, step_dev=None, scale=None, tensors=True, **kw):
    t = gs.gs_adamw_tensor(param=1 << 20, grad=1 << 21, m=1 << 22, v=1 << 23, n=0, grad_type=2, copy_type=2)
    for k, v in kw.items():
        setattr(t, k, v)
    return gs.lib().gs_adamw(C.byref(t) if tensors else None, count, lr, b1, b2, eps, wd, step, step_dev, scale, 0, None)


NAN = float("nan")


@pytest.mark.parametrize("kw,word", [
    (dict(count=-1), b"count"), (dict(tensors=False), b"tensors"), (dict(lr=NAN), b"lr"),
    (dict(wd=float("inf")), b"weight_decay"), (dict(b1=1.0), b"beta"), (dict(b1=-0.1), b"beta"), (dict(b2=NAN), b"beta"),
    (dict(eps=0.0), b"eps"), (dict(eps=1e-60), b"eps"), (dict(eps=NAN), b"eps"), (dict(eps=1e60), b"eps"),
    (dict(step=0), b"step"), (dict(step_dev=P(12)), b"step_dev"), (dict(scale=P(6)), b"grad_scale"),
    (dict(n=-1), b"n ="), (dict(n=(1 << 33) + 1), b"n ="), (dict(n=4, grad_type=3), b"grad_type"),
    (dict(n=4, param=None), b"param"), (dict(n=4, param=2), b"param"), (dict(n=4, grad=None), b"grad"),
    (dict(n=4, grad=6), b"grad"), (dict(n=4, m=None), b"m or v"), (dict(n=4, v=10), b"m or v"),
    (dict(n=4, m_scale=64), b"scale"), (dict(n=4, v_scale=64), b"scale"), (dict(n=4, m_scale=66, v_scale=128), b"scale"),
    (dict(n=4, copy=1 << 24, copy_type=9), b"copy_type"), (dict(n=4, copy=2, copy_type=2), b"copy"),
    (dict(n=4, m=1 << 20), b"overlap"), (dict(n=1 << 20, m=(1 << 20) + 64), b"overlap"),
    (dict(n=4, copy=(1 << 23) + 14, copy_type=0), b"overlap"),
    (dict(n=600, m_scale=1 << 24, v_scale=(1 << 24) + 8), b"overlap"),
])
def test_adamw_refused(kw, word):
    assert _adamw(**kw) == gs.GS_ERR_INVALID_ARG
    assert word in gs.lib().gs_last_error(), gs.lib().gs_last_error()


@pytest.mark.parametrize("count", [1, 2, 63, 64, 65, 200])
def test_adamw_overlap_among_many(count):
    """All six written ranges of every tensor are looked at: only the last
    tensor's copy lies where the first one's parameter is."""
    size = 1 << 12
    t = (gs.gs_adamw_tensor * count)()
    for i in range(count):
        at = (1 << 30) + i * 8 * size
        for k, name in enumerate(("param", "m", "v", "m_scale", "v_scale", "copy", "grad")):
            setattr(t[i], name, at + k * size)
        t[i].n, t[i].grad_type, t[i].copy_type = 256, 2, 0
    t[count - 1].copy = 1 << 30
    assert gs.lib().gs_adamw(t, count, 1e-3, 0.9, 0.999, 1e-8, 0.0, 1, None, None, 0, None) == gs.GS_ERR_INVALID_ARG
    assert b"overlap" in gs.lib().gs_last_error()


def test_adamw_nothing_to_do():
    assert _adamw(count=0, tensors=False) == gs.GS_OK
    assert _adamw(n=0, param=None, grad=None, m=None, v=None) == gs.GS_OK
    gs.gs_adamw([], [], [], [], 1, 1e-3)


@pytest.mark.parametrize("kw,word", [
    (dict(n=-1), b"n ="), (dict(moment=0), b"moment"), (dict(moment=3), b"moment"), (dict(typ=3), b"type"),
    (dict(codes=None), b"codes"), (dict(scales=None), b"scales"), (dict(scales=P(18)), b"scales"),
    (dict(values=None), b"values"), (dict(values=P(17)), b"values"),
])
def test_adamw_moment_refused(kw, word):
    a = dict(codes=P(16), scales=P(16), n=4, moment=1, typ=0, values=P(16)) | kw
    assert gs.lib().gs_adamw_moment(a["codes"], a["scales"], a["n"], a["moment"], a["typ"], a["values"],
                                    None) == gs.GS_ERR_INVALID_ARG
    assert word in gs.lib().gs_last_error()


U1 = torch.uint8


@pytest.mark.parametrize("call,match", [
    (lambda: gs.gs_adamw([_t(4)], [_t(4)], [_t(4)], [], 1, 1e-3), "lists"),
    (lambda: gs.gs_adamw([_t(4, dtype=torch.bfloat16)], [_t(4)], [_t(4)], [_t(4)], 1, 1e-3), "parameter 0"),
    (lambda: gs.gs_adamw([_t(4, 4).t()[1:]], [_t(12)], [_t(12)], [_t(12)], 1, 1e-3), "contiguous"),
    (lambda: gs.gs_adamw([_t(4)], [_t(5)], [_t(4)], [_t(4)], 1, 1e-3), "gradient 0"),
    (lambda: gs.gs_adamw([_t(4)], [_t(4, dtype=torch.float64)], [_t(4)], [_t(4)], 1, 1e-3), "gradient 0"),
    (lambda: gs.gs_adamw([_t(4)], [_t(4)], [_t(4, dtype=U1)], [_t(4)], 1, 1e-3), "m of"),
    (lambda: gs.gs_adamw([_t(4)], [_t(4)], [_t(4, dtype=U1)], [_t(4, dtype=U1)], 1, 1e-3, m_scales=[_t(1)]), "scale"),
    (lambda: gs.gs_adamw([_t(300)], [_t(300)], [_t(300, dtype=U1)], [_t(300, dtype=U1)], 1, 1e-3, m_scales=[_t(1)],
                         v_scales=[_t(2)]), "scales"),
    (lambda: gs.gs_adamw([_t(4)], [_t(4)], [_t(4)], [_t(4)], 1, 1e-3, copies=[_t(3)]), "copy"),
    (lambda: gs.gs_adamw([_t(4)], [_t(4)], [_t(4)], [_t(4)], _t(1), 1e-3), "step"),
    (lambda: gs.gs_adamw([_t(4)], [_t(4)], [_t(4)], [_t(4)], 1, 1e-3, grad_scale=_t(2)), "grad_scale"),
    (lambda: gs.gs_adamw([_t(4)], [_t(4)], [_t(4)], [_t(4)], 1, 1e-3), "GPU tensor"),
    (lambda: gs.gs_adamw_moment(_t(4), _t(1), 1), "codes"), (lambda: gs.gs_adamw_moment(_t(4, dtype=U1), _t(2), 1), "scales"),
    (lambda: gs.gs_adamw_moment(_t(4, dtype=U1), _t(1), 1, torch.int32), "int32"),
    (lambda: gs.gs_adamw_moment(_t(4, dtype=U1), _t(1), 1), "GPU tensor"),
    (lambda: gs.AdamW([]), "no parameters"), (lambda: gs.AdamW([_t(4)], bits=16), "bits"),
    (lambda: gs.AdamW([_t(4)], copies=[None, None]), "copies"),
    (lambda: gs.AdamW([_t(4)]).step([]), "gradients"), (lambda: gs.AdamW([_t(4)]).step([_t(4)]), "GPU tensor"),
])
def test_adamw_binding_refuses(call, match):
    with pytest.raises(ValueError, match=match):
        call()


@pytest.mark.parametrize("change,match", [
    (lambda p, c, s: setattr(p, "data", p.data.t()), "contiguous"),
    (lambda p, c, s: setattr(p, "data", p.data[:2]), "m of parameter 0"),
    (lambda p, c, s: setattr(p, "data", p.data.bfloat16()), "bfloat16"),
    (lambda p, c, s: setattr(c, "data", c.data.t()), "copy of parameter 0 has to be contiguous"),
    (lambda p, c, s: setattr(c, "data", c.data[:1]), "copy of parameter 0"),
    (lambda p, c, s: setattr(c, "data", c.data.view(torch.int16)), "copy of parameter 0 is torch.int16"),
    (lambda p, c, s: setattr(s, "data", s.data[::2]), "m of parameter 0"),
    (lambda p, c, s: setattr(s, "data", s.data[:7]), "m of parameter 0"),
])
def test_adamw_layouts_are_looked_at_again(change, match):
    """A tensor that becomes another layout, size or type at the same address
    is refused as it would have been at first (without a GPU a good call ends
    with the refusal of CPU tensors)."""
    p, c, g = _t(4, 4), _t(4, 4, dtype=torch.bfloat16), _t(4, 4)
    m = _t(16)
    opt = gs.AdamW([p], copies=[c], state=[(m, _t(16), None, None)])
    with pytest.raises(ValueError, match="GPU tensor"):
        opt.step([g])
    change(p, c, m)
    with pytest.raises(ValueError, match=match):
        opt.step([g])


def test_adamw_lists_are_fixed():
    """What the step works on is chosen once: neither the lists nor an entry of
    theirs can be replaced behind its back."""
    params, copies = [_t(4), _t(3)], [None, _t(3)]
    opt = gs.AdamW(params, copies=copies, bits=8, min_8bit=4)
    params[0], copies[1] = _t(5), None
    assert opt.params[0].numel() == 4 and opt.copies[1].numel() == 3
    assert [s[2] is None for s in opt.state] == [False, True]
    for name in ("params", "copies", "state"):
        with pytest.raises(TypeError):
            getattr(opt, name)[0] = None
        with pytest.raises(AttributeError):
            setattr(opt, name, [])


@pytest.mark.parametrize("kw,word", [
    (dict(eps=1.17e-38), b"eps"), (dict(eps=1e-40), b"eps"), (dict(eps=5e37), b"eps"),
    (dict(lr=1e38), b"lr"), (dict(lr=-1e38), b"lr"), (dict(lr=1e39), b"lr"),
    (dict(lr=1e20, wd=1e20), b"weight_decay"), (dict(lr=1e30, b1=1 - 2.0 ** -53), b"lr"),
])
def test_adamw_numbers_that_fp32_cannot_hold(kw, word):
    """The update works in fp32: a reciprocal of eps, lr over the first step's
    1 - beta1 and the decay's factor have to be normal numbers there."""
    assert _adamw(**kw) == gs.GS_ERR_INVALID_ARG
    assert word in gs.lib().gs_last_error(), gs.lib().gs_last_error()


@pytest.mark.parametrize("kw", [dict(eps=2.0 ** -126), dict(eps=1e-15), dict(eps=1e30), dict(eps=2.0 ** 125), dict(lr=1e30),
                                dict(lr=-1.0), dict(lr=0.0), dict(lr=1e-300), dict(b1=0.0, b2=0.0)])
def test_adamw_numbers_that_are_taken(kw):
    assert _adamw(**kw) == gs.GS_OK
