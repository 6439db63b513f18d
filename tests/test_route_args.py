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
    (_sort, dict(ws=None), b"workspace"), (_sort, dict(ws=P(128)), b"workspace"),
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
            assert gs.gs_group_sort_workspace_size(n, groups) >= 256
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
