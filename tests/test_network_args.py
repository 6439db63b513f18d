"""What the network operators refuse, on the host (no GPU: nothing is
launched on a refusal), and their workspace sizes."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

import differentiable_gaussian_splatting_dgs_amd as gs

P = C.c_void_p
F = C.c_float


def _norm_fwd(x=P(16), ldx=64, rows=4, width=64, eps=1e-5, typ=0, y=P(16), ldy=64, gamma=P(16), mean=P(16)):
    return gs.lib().gs_layer_norm_fwd(x, ldx, gamma, P(16), rows, width, F(eps), typ, y, ldy, mean, P(16), None)


def _norm_bwd(x=P(16), ldx=64, dy=P(16), lddy=64, rows=4, width=64, typ=0, dx=P(16), lddx=64, mean=P(16), dres=None,
              lddres=0, ws=P(256), ws_bytes=1 << 20):
    return gs.lib().gs_layer_norm_bwd(x, ldx, dy, lddy, P(16), mean, P(16), dres, lddres, rows, width, typ, dx, lddx,
                                      P(16), P(16), ws, ws_bytes, None)


def _fwd(x=P(16), ldx=64, w=P(16), ldw=64, bias=P(16), residual=None, ldr=0, rows=4, inner=64, out=32, typ=0, act=0,
         y=P(16), ldy=32, z=None, ldz=0):
    return gs.lib().gs_linear_fwd(x, ldx, w, ldw, bias, residual, ldr, rows, inner, out, typ, act, y, ldy, z, ldz,
                                  None)


def _bwd(x=P(16), ldx=64, w=P(16), ldw=64, z=P(16), ldz=32, dy=P(16), lddy=32, rows=4, inner=64, out=32, typ=0, act=1,
         dx=P(16), lddx=64, dw=P(16), dw_type=0, db=P(16), ws=P(256), ws_bytes=1 << 24):
    return gs.lib().gs_linear_bwd(x, ldx, w, ldw, z, ldz, dy, lddy, rows, inner, out, typ, act, dx, lddx, dw, dw_type,
                                  db, ws, ws_bytes, None)


def _grouped(offsets=P(16), groups=3, rows=4):
    return gs.lib().gs_grouped_linear_fwd(P(16), 64, P(16), 64, None, offsets, groups, None, 0, rows, 64, 32, 0, 0,
                                          P(16), 32, None, 0, None)


@pytest.mark.parametrize("call,kw,word", [
    (_norm_fwd, dict(typ=3), b"type"), (_norm_fwd, dict(typ=-1), b"type"),
    (_norm_fwd, dict(rows=-1), b"rows"), (_norm_fwd, dict(rows=1 << 31), b"rows"),
    (_norm_fwd, dict(width=0), b"width"), (_norm_fwd, dict(width=gs.GS_MAX_NET_DIM + 1), b"width"),
    (_norm_fwd, dict(eps=-1.0), b"eps"), (_norm_fwd, dict(eps=float("nan")), b"eps"),
    (_norm_fwd, dict(x=None), b"x is NULL"), (_norm_fwd, dict(x=P(17)), b"x not aligned"),
    (_norm_fwd, dict(x=P(18), typ=2), b"x not aligned"), (_norm_fwd, dict(ldx=63), b"leading dimension"),
    (_norm_fwd, dict(ldx=0), b"leading dimension"), (_norm_fwd, dict(ldy=1), b"leading dimension"),
    (_norm_fwd, dict(y=None), b"y is NULL"), (_norm_fwd, dict(gamma=P(18)), b"gamma"),
    (_norm_fwd, dict(mean=P(17)), b"mean"),
    (_norm_bwd, dict(dy=None), b"dy is NULL"), (_norm_bwd, dict(lddy=5), b"leading dimension"),
    (_norm_bwd, dict(mean=None), b"mean"), (_norm_bwd, dict(dres=P(16), lddres=2), b"dres"),
    (_norm_bwd, dict(lddx=3), b"dx"), (_norm_bwd, dict(ws=None), b"workspace"),
    (_norm_bwd, dict(ws=P(264)), b"workspace"), (_norm_bwd, dict(ws_bytes=255), b"workspace_bytes"),
    (_norm_bwd, dict(typ=9), b"type"), (_norm_bwd, dict(width=-4), b"width"),
    (_fwd, dict(typ=5), b"type"), (_fwd, dict(act=4), b"act"), (_fwd, dict(act=-1), b"act"),
    (_fwd, dict(rows=-2), b"rows"), (_fwd, dict(inner=0), b"in ="), (_fwd, dict(out=0), b"out ="),
    (_fwd, dict(out=gs.GS_MAX_NET_DIM + 1), b"out ="), (_fwd, dict(ldx=8), b"x: leading"),
    (_fwd, dict(ldw=63), b"w: leading"), (_fwd, dict(ldy=31), b"y: leading"), (_fwd, dict(x=None), b"x is NULL"),
    (_fwd, dict(w=None), b"w is NULL"), (_fwd, dict(w=P(3)), b"w not aligned"), (_fwd, dict(y=None), b"y is NULL"),
    (_fwd, dict(bias=P(2)), b"bias"), (_fwd, dict(residual=P(16), ldr=4), b"residual"),
    (_fwd, dict(z=P(16), ldz=4), b"z: leading"), (_fwd, dict(z=P(1), ldz=32), b"z not aligned"),
    (_fwd, dict(rows=(1 << 31) - 1, inner=64, out=65536, ldy=65536), b"launch grid"),
    (_bwd, dict(z=None), b"z is NULL"), (_bwd, dict(ldz=3), b"z: leading"), (_bwd, dict(dy=None), b"dy is NULL"),
    (_bwd, dict(lddy=31), b"dy: leading"), (_bwd, dict(lddx=63), b"dx: leading"), (_bwd, dict(dw_type=1), b"dw_type"),
    (_bwd, dict(dw=P(18), dw_type=2), b"dw not aligned"), (_bwd, dict(db=P(18)), b"db"),
    (_bwd, dict(ws=None), b"workspace"), (_bwd, dict(ws=P(16)), b"workspace"),
    (_bwd, dict(ws_bytes=16), b"workspace_bytes"), (_bwd, dict(x=None), b"x is NULL"),
    (_bwd, dict(w=None), b"w is NULL"), (_bwd, dict(act=7), b"act"),
    (_grouped, dict(offsets=None), b"offsets"), (_grouped, dict(offsets=P(4)), b"offsets"),
    (_grouped, dict(groups=0), b"num_groups"), (_grouped, dict(groups=-1), b"num_groups"),
    (_grouped, dict(groups=gs.GS_MAX_NET_GROUPS + 1), b"num_groups"),
])
def test_refused_on_the_host(call, kw, word):
    assert call(**kw) == gs.GS_ERR_INVALID_ARG
    assert word in gs.lib().gs_last_error()


def test_no_rows_need_no_matrices():
    assert _norm_fwd(rows=0, x=None, y=None) == gs.GS_OK
    assert _fwd(rows=0, x=None, w=None, y=None) == gs.GS_OK
    assert _grouped(rows=0) == gs.GS_OK


def test_workspace_sizes():
    n = gs.gs_workspace_size(gs.GS_OP_LAYER_NORM_BWD, 1000, 64)
    assert n >= 2 * 64 * 4 and n % 256 == 0
    assert gs.gs_workspace_size(gs.GS_OP_LAYER_NORM_BWD, 1 << 30, 256) <= 4096 * 2 * 256 * 4
    # dz of an activation needs its rows, and no activation does not
    size = gs.gs_linear_workspace_size
    assert size(1 << 20, 64, 64, 0, gs.GS_TYPE_BF16, gs.GS_ACT_GELU) >= (1 << 20) * 64 * 2
    assert size(1 << 20, 64, 64, 0, gs.GS_TYPE_BF16, gs.GS_ACT_NONE) < (1 << 20) * 64 * 2
    assert size(0, 64, 64, 0, gs.GS_TYPE_F32, gs.GS_ACT_NONE) >= 256
    assert size(0, 64, 64, 9, gs.GS_TYPE_F32, gs.GS_ACT_GELU) >= 256
    # many rows: partial sums do not grow with them
    big = size(1 << 28, 64, 64, 0, gs.GS_TYPE_BF16, gs.GS_ACT_NONE)
    assert 0 < big < 1 << 28
    assert size(1 << 28, 64, 64, 1000, gs.GS_TYPE_F32, gs.GS_ACT_NONE) < 1 << 30
    for bad in (dict(rows=-1), dict(inner=0), dict(num_groups=-1), dict(num_groups=5000), dict(type=4), dict(act=9)):
        args = dict(rows=10, inner=8, out=8, num_groups=0, type=0, act=0) | bad
        with pytest.raises(gs.GSError):
            size(**args)


def test_the_binding_checks_what_only_tensors_show():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        gs.gs_layer_norm_fwd(x)
    with pytest.raises(ValueError, match="GPU"):
        gs.gs_linear_fwd(x, torch.zeros(3, 8))
    with pytest.raises(ValueError, match="float64"):
        gs.gs_linear_fwd(x.double(), torch.zeros(3, 8))
    with pytest.raises(ValueError, match="dimensions"):
        gs.gs_layer_norm_fwd(torch.zeros(8))
    with pytest.raises(ValueError, match="w is"):
        gs.gs_linear_fwd(x, torch.zeros(3, 9))
    with pytest.raises(ValueError, match="w is"):
        gs.gs_linear_fwd(x, torch.zeros(3, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="last stride"):
        gs.gs_linear_fwd(torch.zeros(8, 4).t(), torch.zeros(3, 8))
    with pytest.raises(ValueError, match="bias"):
        gs.gs_linear_fwd(x, torch.zeros(3, 8), torch.zeros(4))
    with pytest.raises(ValueError, match="residual"):
        gs.gs_linear_fwd(x, torch.zeros(3, 8), residual=torch.zeros(4, 4))
    with pytest.raises(ValueError, match="offsets"):
        gs.gs_grouped_linear_fwd(x, torch.zeros(2, 3, 8), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="groups"):
        gs.gs_grouped_linear_fwd(x, torch.zeros(5, 3, 8), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="without a gap"):
        gs.gs_grouped_linear_fwd(x, torch.zeros(2, 6, 8)[:, :3], torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="needs z"):
        gs.gs_linear_bwd(x, torch.zeros(3, 8), torch.zeros(4, 3), None, gs.GS_ACT_RELU)
    with pytest.raises(ValueError, match="dy"):
        gs.gs_linear_bwd(x, torch.zeros(3, 8), torch.zeros(4, 5))


@pytest.mark.parametrize("workspace", [torch.empty(1 << 16, dtype=torch.uint8, device="meta"),
                                       torch.zeros(1 << 16, 2, dtype=torch.uint8)[:, 0],
                                       torch.zeros(64, 64).t()], ids=["device", "strided", "transposed"])
def test_the_binding_checks_workspaces(workspace):
    """On another device than x, or with gaps: refused before anything else
    sees its address."""
    x, dy, w, v = torch.zeros(4, 8), torch.zeros(4, 3), torch.zeros(3, 8), torch.ones(4)
    offsets = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: gs.gs_layer_norm_bwd(x, x, None, v, v, workspace=workspace),
                 lambda: gs.gs_linear_bwd(x, w, dy, workspace=workspace),
                 lambda: gs.gs_grouped_linear_bwd(x, torch.zeros(2, 3, 8), offsets, dy, workspace=workspace)):
        with pytest.raises(ValueError, match="workspace"):
            call()


def test_the_binding_checks_streams():
    """A stream of another device than x: refused, nothing is called."""
    from types import SimpleNamespace

    from differentiable_gaussian_splatting_dgs_amd import network
    x = SimpleNamespace(device=torch.device("cuda", 0), get_device=lambda: 0)
    stream = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    called = []
    with pytest.raises(ValueError, match="stream"):
        network._launch(lambda *a: called.append(a), x, stream)
    assert not called


def test_the_package_imports_without_torch_internals():
    """A torch without CUDA's internal functions (a build for the CPU) imports
    the package."""
    import subprocess
    import sys
    code = ("import torch\n"
            "del torch._C._cuda_getCurrentRawStream\n"
            "import differentiable_gaussian_splatting_dgs_amd as gs\n"
            "assert callable(gs.gs_linear_fwd)\n")
    root = __file__.rsplit("/", 2)[0]
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("offsets", [[5, 10], [-1, 4], [0, 6, 4], [3], [], [[0, 4]]])
def test_the_decoder_refuses_blocks_that_leave_rows_out(offsets):
    """Rows of no block have no attributes: blocks begin at 0 and follow each
    other."""
    from differentiable_gaussian_splatting_dgs_amd.decoder import AttributeDecoder
    with pytest.raises(ValueError, match="offsets"):
        AttributeDecoder(offsets, width=8, hidden=8, device="cpu")


def test_the_decoder_takes_blocks_that_cover_the_rows():
    from differentiable_gaussian_splatting_dgs_amd.decoder import AttributeDecoder
    dec = AttributeDecoder(torch.tensor([0, 3, 3, 9]), width=8, hidden=8, device="cpu")
    assert dec.masters["features"].shape == (9, 8) and dec.offsets.dtype == torch.int64


def test_the_decoder_refuses_the_steps_parameters_as_base():
    """train_views writes base + attributes into the step's parameters: with
    those as the base, every pass would add to the last."""
    from types import SimpleNamespace

    from differentiable_gaussian_splatting_dgs_amd.decoder import AttributeDecoder
    dec = AttributeDecoder([0, 4], width=8, hidden=8, device="cpu")
    step = SimpleNamespace(params=torch.zeros(59, 4))
    for base in (step.params, step.params[:, :]):
        with pytest.raises(ValueError, match="base"):
            dec.train_views(step, base)
