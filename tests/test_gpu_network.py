"""The network operators (layer norm, linear layer, grouped linear layer)
against their definitions in 64 bits, on the GPU.

Tolerances are bounds, element by element, made of the roundings that happen
(u: half a step of the storage type; 2^-24: of fp32):
 - a stored result is off by u of itself (plus half the smallest fp16 number);
 - an fp32 sum of n terms, in any order, by (n + 4) 2^-24 of the sum of
   their absolute values (the matrix instructions' inner sums included, for
   which the factor is doubled);
 - the activations of 16-bit storage by 2^-19 of their argument (native
   exponential and reciprocal, and 1.5e-7 of the error function);
 - dz is stored with u of itself before it enters the products."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EPS32 = 2.0 ** -24
TYPES = ["bf16", "fp16", "fp32"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def gs():
    import differentiable_gaussian_splatting_dgs_amd as mod
    return mod


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _u(t):
    return torch.finfo(t).eps / 2


def _tiny(t):
    return 2.0 ** -25 if t == torch.float16 else 0.0


def _rand(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _strided(t, extra, shift=0):
    """t's values with a leading dimension `extra` longer, the padding NaN,
    the first element `shift` elements into its allocation."""
    rows, width = t.shape
    buf = torch.full((rows * (width + extra) + shift,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[shift:].as_strided((rows, width), (width + extra, 1))
    v.copy_(t)
    return v


def _close(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    # the same infinities and NaN are equal
    bad &= ~((got == want) | (got.isnan() & want.isnan()))
    n = int(bad.sum())
    if n:
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{what}: {n} of {bad.numel()} off, first at {i}: {got.flatten()[i].item()} for "
                             f"{want.flatten()[i].item()}, tolerance {torch.as_tensor(tol).expand_as(want).flatten()[i].item()}")


# --- layer norm ---------------------------------------------------------------

NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (130, 255), (17, 256), (9, 515), (33, 1024), (6, 1537), (4, 2049), (3, 4100),
               (2, 9001), (2, 20000)]
# additions on the way of one row's sum: chunks a lane times their values,
# then the lanes
NORM_DEPTH = 400


def _norm_fwd_check(gs, x, gamma, beta, eps, **kw):
    y, mean, rstd = gs.gs_layer_norm_fwd(x, gamma, beta, eps, **kw)
    xd = x.double()
    m = xd.mean(1)
    c = xd - m[:, None]
    r = 1.0 / ((c * c).mean(1) + eps).sqrt()
    e = NORM_DEPTH * EPS32
    absm = xd.abs().mean(1)
    _close(mean, m, e * absm + 1e-30, "mean")
    off = 2 * e * (1 + absm * r)
    _close(rstd, r, off * r, "rstd")
    g = gamma.double() if gamma is not None else torch.ones(x.shape[1], dtype=torch.float64, device=x.device)
    b = beta.double() if beta is not None else torch.zeros_like(g)
    xh = c * r[:, None]
    want = xh * g + b
    t = x.dtype
    _close(y, want, _u(t) * want.abs() + _tiny(t) + g.abs() * (1 + xh.abs()) * 2 * off[:, None]
           + 4 * EPS32 * (b.abs() + (g * xh).abs()), "y")
    return y, mean, rstd


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,width", NORM_SHAPES)
def test_layer_norm_forward(gs, name, rows, width):
    gen, t = _gen(rows * 31 + width), _dtype(name)
    x = _rand(gen, rows, width, scale=1.5, dtype=t) + 0.5
    gamma, beta = 1 + _rand(gen, width, scale=0.2), _rand(gen, width)
    _norm_fwd_check(gs, x, gamma, beta, 1e-5)
    _norm_fwd_check(gs, x, None, None, 1e-3)
    # padding of NaN, and a first element that no 16 bytes divide
    xs = _strided(x, 5, 1)
    y = _strided(torch.zeros_like(x), 3, 1)
    _norm_fwd_check(gs, xs, gamma, None, 1e-5, y=y)
    assert y.stride(0) == width + 3


def test_layer_norm_constant_and_bad_rows(gs):
    x = torch.zeros(8, 96, device="cuda")
    x[1] = 3.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = torch.arange(96, device="cuda") * 1e-3
    y, mean, rstd = gs.gs_layer_norm_fwd(x, None, None, 1e-5)
    assert torch.equal(y[0], torch.zeros(96, device="cuda")) and torch.equal(y[1], torch.zeros(96, device="cuda"))
    assert y[2].isnan().all() and y[3].isnan().all()
    assert y[4:].isfinite().all() and mean[1].item() == 3.0
    # the same bits as without the bad rows beside them
    y2, _, _ = gs.gs_layer_norm_fwd(x[4:].contiguous(), None, None, 1e-5)
    assert torch.equal(y[4:], y2)


def _norm_bwd_want(x, dy, gamma, mean, rstd, dres):
    xd, dyd = x.double(), dy.double()
    g1 = gamma.double() if gamma is not None else torch.ones(x.shape[1], dtype=torch.float64, device=x.device)
    r = rstd.double()[:, None]
    xh = (xd - mean.double()[:, None]) * r
    g = dyd * g1
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    e = NORM_DEPTH * EPS32
    near = r * (8 * EPS32 * (g.abs() + xh.abs() * (g * xh).mean(1, keepdim=True).abs())
                + 2 * e * g.abs().mean(1, keepdim=True) + xh.abs() * 2 * e * (g * xh).abs().mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
        near = near + 2 * EPS32 * dres.double().abs()
    return dx, near, dyd * xh, dyd


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,width", NORM_SHAPES + [(3001, 64), (2500, 259)])
def test_layer_norm_backward(gs, name, rows, width):
    gen, t = _gen(rows * 37 + width), _dtype(name)
    x = _rand(gen, rows, width, scale=1.5, dtype=t) + 0.5
    dy, dres = _rand(gen, rows, width, dtype=t), _rand(gen, rows, width, dtype=t)
    gamma = 1 + _rand(gen, width, scale=0.2)
    _, mean, rstd = gs.gs_layer_norm_fwd(x, gamma, None, 1e-5)
    for g, res, xs, ds in ((gamma, None, x, dy), (None, dres, _strided(x, 5, 1), _strided(dy, 2, 3))):
        dx, dgamma, dbeta = gs.gs_layer_norm_bwd(xs, ds, g, mean, rstd, dres=res)
        want, near, a, b = _norm_bwd_want(x, dy, g, mean, rstd, res)
        _close(dx, want, _u(t) * want.abs() + _tiny(t) + near, "dx")
        _close(dgamma, a.sum(0), (rows + 8) * EPS32 * a.abs().sum(0), "dgamma")
        _close(dbeta, b.sum(0), (rows + 8) * EPS32 * b.abs().sum(0), "dbeta")


def test_layer_norm_no_rows(gs):
    x = torch.zeros(0, 48, device="cuda")
    e = torch.zeros(0, device="cuda")
    y, mean, rstd = gs.gs_layer_norm_fwd(x)
    assert y.shape == (0, 48)
    dg = torch.full((48,), 7.0, device="cuda")
    db = torch.full((48,), 7.0, device="cuda")
    gs.gs_layer_norm_bwd(x, x, None, e, e, dgamma=dg, dbeta=db)
    assert not dg.any() and not db.any()


def test_layer_norm_gradient_against_differences(gs):
    gen = _gen(5)
    x, v = _rand(gen, 6, 40), _rand(gen, 6, 40)
    gamma, beta = 1 + _rand(gen, 40, scale=0.2), _rand(gen, 40)
    _, mean, rstd = gs.gs_layer_norm_fwd(x, gamma, beta, 1e-5)
    dx, dg, db = gs.gs_layer_norm_bwd(x, v, gamma, mean, rstd)

    def f(x, gamma, beta):
        c = x - x.mean(1, keepdim=True)
        return ((c / ((c * c).mean(1, keepdim=True) + 1e-5).sqrt() * gamma + beta) * v.double()).sum()
    at = [t.double() for t in (x, gamma, beta)]
    for k, grad in enumerate((dx, dg, db)):
        d = _rand(gen, *at[k].shape).double()
        h = 1e-4
        up, dn = list(at), list(at)
        up[k], dn[k] = at[k] + h * d, at[k] - h * d
        diff = (f(*up) - f(*dn)) / (2 * h)
        mine = (grad.double() * d).sum()
        # h^2 of third derivatives (below 100 here), 64-bit rounding / h, and fp32 roundings of the gradient
        tol = 100 * h * h * float(d.abs().sum()) + 1e-9 + 64 * EPS32 * float((grad.double().abs() * d.abs()).sum())
        assert abs(float(diff - mine)) <= tol, (k, float(diff), float(mine), tol)


# --- linear layer ---------------------------------------------------------------

ACTS = ["none", "relu", "silu", "gelu"]


def _act_id(gs, act):
    return {"none": gs.GS_ACT_NONE, "relu": gs.GS_ACT_RELU, "silu": gs.GS_ACT_SILU, "gelu": gs.GS_ACT_GELU}[act]


def _act(v, act):
    return {"none": lambda: v, "relu": lambda: torch.where(v < 0, torch.zeros_like(v), v),
            "silu": lambda: v * torch.sigmoid(v), "gelu": lambda: 0.5 * v * torch.erfc(-v / math.sqrt(2))}[act]()


def _slope(v, act):
    if act == "none":
        return torch.ones_like(v)
    if act == "relu":
        return (v > 0).double()
    if act == "silu":
        p = torch.sigmoid(v)
        return p * (1 + v * (1 - p))
    return 0.5 * torch.erfc(-v / math.sqrt(2)) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)


def _spans(offsets, rows, groups):
    """The groups as the library reads any list: clamped, never falling."""
    if offsets is None:
        return [(0, rows)]
    out, low = [], min(max(offsets[0], 0), rows)
    for v in offsets[1:]:
        high = max(low, min(max(v, 0), rows))
        out.append((low, high))
        low = high
    return out


def _linear_fwd_check(gs, x, w, bias, act, residual, offsets=None, **kw):
    t, rows, out = x.dtype, x.shape[0], w.shape[-2]
    spans = _spans(offsets, rows, None)
    y = torch.full((rows, out), 77.0, dtype=t, device="cuda") if kw.get("y") is None else kw.pop("y")
    z = torch.full((rows, out), 77.0, dtype=t, device="cuda") if kw.get("z") is None else kw.pop("z")
    if offsets is None:
        gs.gs_linear_fwd(x, w, bias, _act_id(gs, act), residual=residual, y=y, z=z, **kw)
    else:
        off = torch.tensor(offsets, dtype=torch.int64, device="cuda")
        gs.gs_grouped_linear_fwd(x, w, off, bias, _act_id(gs, act), residual=residual, y=y, z=z, **kw)
    k = x.shape[1]
    covered = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e, (a, b) in enumerate(spans):
        if a == b:
            continue
        covered[a:b] = True
        we = w[e].double() if offsets is not None else w.double()
        be = None if bias is None else (bias[e] if offsets is not None else bias).double()
        xe = x[a:b].double()
        v = xe @ we.t()
        near = 2 * (k + 4) * EPS32 * (xe.abs() @ we.abs().t())
        if be is not None:
            v = v + be
            near = near + 2 * EPS32 * (be.abs() + v.abs())
        _close(z[a:b], v, _u(t) * v.abs() + near + _tiny(t), f"z of group {e}")
        want = _act(v, act)
        near = 1.2 * near + (2 ** -19 if act in ("silu", "gelu") else 0.0) * v.abs()
        if residual is not None:
            r = residual[a:b].double()
            want = want + r
            near = near + 2 * EPS32 * r.abs()
        _close(y[a:b], want, _u(t) * want.abs() + near + _tiny(t), f"y of group {e}")
    assert (y[~covered] == 77.0).all() and (z[~covered] == 77.0).all(), "rows of no group were written"
    return y, z


def _linear_bwd_check(gs, x, w, dy, z, act, offsets=None, dw=None, **kw):
    t, rows, out, k = x.dtype, x.shape[0], w.shape[-2], x.shape[1]
    spans = _spans(offsets, rows, None)
    dx = torch.full((rows, k), 77.0, dtype=t, device="cuda")
    if offsets is None:
        _, dw, db = gs.gs_linear_bwd(x, w, dy, z, _act_id(gs, act), dx=dx, dw=dw, **kw)
    else:
        off = torch.tensor(offsets, dtype=torch.int64, device="cuda")
        _, dw, db = gs.gs_grouped_linear_bwd(x, w, off, dy, z, _act_id(gs, act), dx=dx, dw=dw, **kw)
    u = _u(t)
    covered = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e, (a, b) in enumerate(spans):
        covered[a:b] = True
        we, dwe, dbe = (w[e], dw[e], db[e]) if offsets is not None else (w, dw, db)
        we, xe, g = we.double(), x[a:b].double(), dy[a:b].double()
        off_z = torch.zeros_like(g)
        if act != "none":
            off_z = 2 ** -18 * g.abs()     # the slope, whose value is at most 1.13
            g = g * _slope(z[a:b].double(), act)
        stored = off_z + (u * g.abs() + _tiny(t) if act != "none" else 0.0)
        want = g @ we
        _close(dx[a:b], want, u * want.abs() + _tiny(t) + stored @ we.abs()
               + 2 * (out + 4) * EPS32 * (g.abs() @ we.abs()), f"dx of group {e}")
        want = g.t() @ xe
        _close(dwe, want, _u(dwe.dtype) * want.abs() + _tiny(dwe.dtype) + stored.t() @ xe.abs()
               + 2 * (b - a + 4) * EPS32 * (g.abs().t() @ xe.abs()), f"dw of group {e}")
        _close(dbe, g.sum(0), off_z.sum(0) + (b - a + 4) * EPS32 * g.abs().sum(0), f"db of group {e}")
    assert (dx[~covered] == 77.0).all(), "rows of no group were written"


LINEAR_SHAPES = [(1, 1, 1), (2, 3, 5), (7, 64, 64), (1, 256, 130), (19, 59, 48), (65, 129, 127), (128, 128, 128),
                 (130, 72, 59), (257, 200, 320), (600, 48, 264), (33, 1031, 40), (16, 512, 1024)]


# rows enough for the kernels that keep their weights, at every width of theirs
MANY_ROWS = [(20000, 40, 136), (9000, 264, 520), (33001, 64, 64), (66001, 128, 128), (132001, 256, 256),
             (33000, 24, 256), (66000, 96, 120), (100003, 184, 512), (132001, 192, 48), (33000, 56, 104), (66000, 72, 264), (40001, 104, 56),
             (40000, 104, 200), (40003, 200, 104)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,inner,out", LINEAR_SHAPES + MANY_ROWS + [(52000, 520, 256), (9000, 512, 1800)])
def test_linear_forward(gs, name, rows, inner, out):
    gen, t = _gen(rows + 7 * inner + 13 * out), _dtype(name)
    x, w = _rand(gen, rows, inner, dtype=t), _rand(gen, out, inner, scale=2 * inner ** -0.5, dtype=t)
    bias, residual = _rand(gen, out), _rand(gen, rows, out, dtype=t)
    act = ACTS[(rows + inner + out) % 4]
    _linear_fwd_check(gs, x, w, bias, act, residual)
    # padding of NaN everywhere, nothing aligned, no bias or residual
    y, z = _strided(torch.zeros_like(residual), 3, 1), _strided(torch.zeros_like(residual), 1, 5)
    _linear_fwd_check(gs, _strided(x, 3, 1), _strided(w, 1, 3), None, "none", _strided(residual, 2, 1), y=y, z=z)
    # aligned padding (the 16-byte path), rows of which end inside a chunk
    pad = -inner % 8 + 8
    _linear_fwd_check(gs, _strided(x, pad), _strided(w, pad), bias, "none", None)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("act", ACTS)
def test_linear_activations(gs, name, act):
    gen, t = _gen(3), _dtype(name)
    # arguments from -40 to 40, zero among them
    x = torch.linspace(-40, 40, 321, device="cuda").reshape(321, 1).to(t)
    w = torch.ones(9, 1, device="cuda", dtype=t)
    _, z = _linear_fwd_check(gs, x, w, None, act, None)
    dy = _rand(gen, 321, 9, dtype=t)
    _linear_bwd_check(gs, x, w, dy, z, act)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,inner,out", LINEAR_SHAPES + MANY_ROWS + [(5000, 256, 250), (52000, 512, 256), (33001, 512, 512), (70001, 504, 256)])
def test_linear_backward(gs, name, rows, inner, out):
    gen, t = _gen(rows + 17 * inner + 13 * out), _dtype(name)
    x, w = _rand(gen, rows, inner, dtype=t), _rand(gen, out, inner, scale=2 * inner ** -0.5, dtype=t)
    dy, z = _rand(gen, rows, out, dtype=t), _rand(gen, rows, out, dtype=t)
    act = ACTS[1 + (rows + inner + out) % 3]
    _linear_bwd_check(gs, x, w, dy, z, act)
    _linear_bwd_check(gs, _strided(x, 3, 1), _strided(w, 1, 3), _strided(dy, 2, 1), _strided(z, 5, 3), act)
    _linear_bwd_check(gs, x, w, dy, None, "none", dw=torch.empty(out, inner, device="cuda"))
    _linear_bwd_check(gs, _strided(x, -inner % 8 + 8), w, _strided(dy, -out % 8 + 8), None, "none")
    _linear_bwd_check(gs, _strided(x, -inner % 8 + 8), w, _strided(dy, -out % 8 + 8), _strided(z, -out % 8 + 8), act)


def test_linear_gradient_against_differences(gs):
    gen = _gen(11)
    x, w, bias, v = _rand(gen, 9, 21), _rand(gen, 13, 21, scale=0.3), _rand(gen, 13), _rand(gen, 9, 13)
    for act in ACTS:
        _, z = gs.gs_linear_fwd(x, w, bias, _act_id(gs, act), save_z=True)
        grads = gs.gs_linear_bwd(x, w, v, z, _act_id(gs, act))
        at = [t.double() for t in (x, w, bias)]

        def f(x, w, b):
            return (_act(x @ w.t() + b, act) * v.double()).sum()
        for k, grad in enumerate(grads):
            d, h = _rand(gen, *at[k].shape).double(), 1e-5
            up, dn = list(at), list(at)
            up[k], dn[k] = at[k] + h * d, at[k] - h * d
            if act == "relu":   # the inputs hold no corner between the two points
                assert torch.equal(up[0] @ up[1].t() + up[2] > 0, dn[0] @ dn[1].t() + dn[2] > 0)
            diff = (f(*up) - f(*dn)) / (2 * h)
            mine = (grad.double() * d).sum()
            # third derivatives below 10 a unit of argument cubed; 64-bit rounding / h; fp32 sums
            tol = 1e4 * h * h * float(d.abs().sum()) + 1e-8 + 64 * EPS32 * float((grad.double().abs() * d.abs()).sum())
            assert abs(float(diff - mine)) <= tol, (act, k, float(diff), float(mine), tol)


def test_linear_no_rows(gs):
    x = torch.zeros(0, 24, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(40, 24, device="cuda", dtype=torch.bfloat16)
    dy = torch.zeros(0, 40, device="cuda", dtype=torch.bfloat16)
    assert gs.gs_linear_fwd(x, w).shape == (0, 40)
    dx, dw, db = gs.gs_linear_bwd(x, w, dy, dw=torch.full((40, 24), 5.0, device="cuda"),
                                  db=torch.full((40,), 5.0, device="cuda"))
    assert dx.shape == (0, 24) and not dw.any() and not db.any()
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    w3 = torch.ones(3, 40, 24, device="cuda", dtype=torch.bfloat16)
    assert gs.gs_grouped_linear_fwd(x, w3, off).shape == (0, 40)
    _, dw, db = gs.gs_grouped_linear_bwd(x, w3, off, dy)
    assert not dw.any() and not db.any()


def test_linear_bad_values_stay_in_their_row(gs):
    """NaN and infinities of one row reach that row's results alone, and the
    sums over rows."""
    gen = _gen(2)
    for t in (torch.bfloat16, torch.float32):
        x, w = _rand(gen, 200, 96, dtype=t), _rand(gen, 72, 96, scale=0.1, dtype=t)
        clean = gs.gs_linear_fwd(x, w, None, gs.GS_ACT_GELU)
        x2 = x.clone()
        x2[17, 3], x2[100, 95] = float("nan"), float("inf")
        y = gs.gs_linear_fwd(x2, w, None, gs.GS_ACT_GELU)
        keep = torch.ones(200, dtype=torch.bool, device="cuda")
        keep[17] = keep[100] = False
        assert y[17].isnan().all() and not y[100].isfinite().all()
        assert torch.equal(y[keep], clean[keep])


def test_linear_residual_in_place(gs):
    gen = _gen(8)
    x, w = _rand(gen, 300, 64, dtype=torch.bfloat16), _rand(gen, 64, 64, scale=0.1, dtype=torch.bfloat16)
    r = _rand(gen, 300, 64, dtype=torch.bfloat16)
    want = gs.gs_linear_fwd(x, w, None, gs.GS_ACT_SILU, residual=r)
    gs.gs_linear_fwd(x, w, None, gs.GS_ACT_SILU, residual=r, y=r)
    assert torch.equal(r, want)


def test_linear_beyond_32_bit_offsets(gs):
    """Rows whose elements lie past 2^31 elements and 2^32 bytes."""
    rows, inner, out = (1 << 20) + 77, 2056, 24
    gen, t = _gen(4), torch.bfloat16
    x = torch.empty(rows, inner, device="cuda", dtype=t).normal_(generator=gen)
    w = _rand(gen, out, inner, scale=0.02, dtype=t)
    dy = _rand(gen, rows, out, dtype=t)
    y = gs.gs_linear_fwd(x, w)
    dx, dw, db = gs.gs_linear_bwd(x, w, dy)
    ny, mean, rstd = gs.gs_layer_norm_fwd(x)
    for a, b in ((0, 200), (rows // 2, rows // 2 + 200), (rows - 300, rows)):
        xe = x[a:b].double()
        want = xe @ w.double().t()
        _close(y[a:b], want, _u(t) * want.abs() + 2 * (inner + 4) * EPS32 * (xe.abs() @ w.double().abs().t()), "y")
        want = dy[a:b].double() @ w.double()
        _close(dx[a:b], want, _u(t) * want.abs() + 2 * (out + 4) * EPS32 * (dy[a:b].double().abs() @ w.double().abs()),
               "dx")
        c = xe - xe.mean(1, keepdim=True)
        want = c / ((c * c).mean(1, keepdim=True) + 1e-5).sqrt()
        _close(ny[a:b], want, _u(t) * want.abs() + (1 + want.abs()) * 8 * NORM_DEPTH * EPS32, "norm")
    want = torch.zeros(out, inner, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for a in range(0, rows, 1 << 16):
        g, xe = dy[a:a + (1 << 16)].double(), x[a:a + (1 << 16)].double()
        want += g.t() @ xe
        size += g.abs().t() @ xe.abs()
    # a sum of a million terms: roundings of either sign, so 8 of them on the whole of it rather than one a term
    _close(dw, want, _u(t) * want.abs() + 8 * EPS32 * size, "dw")


# --- grouped linear layer ----------------------------------------------------------

GROUPS = {
    "one": [0, 150],
    "even": [0, 64, 128, 192],
    "ragged": [0, 1, 1, 130, 131, 300, 300, 463],
    "empty ends": [0, 0, 0, 77, 77, 77],
    "gap": [5, 40, 90],            # rows 0-4 and 90-99 belong to nobody
    "none": [0, 0, 0, 0],
}


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("case", sorted(GROUPS))
@pytest.mark.parametrize("inner,out", [(40, 64), (129, 59), (256, 136)])
def test_grouped_linear(gs, name, case, inner, out):
    offsets = GROUPS[case]
    groups, rows = len(offsets) - 1, max(offsets[-1] + (10 if case == "gap" else 0), 3)
    gen, t = _gen(inner + out), _dtype(name)
    x, w = _rand(gen, rows, inner, dtype=t), _rand(gen, groups, out, inner, scale=2 * inner ** -0.5, dtype=t)
    bias, residual = _rand(gen, groups, out), _rand(gen, rows, out, dtype=t)
    dy, z = _rand(gen, rows, out, dtype=t), _rand(gen, rows, out, dtype=t)
    _linear_fwd_check(gs, x, w, bias, "gelu", residual, offsets)
    _linear_fwd_check(gs, _strided(x, 3, 1), w, None, "none", None, offsets)
    _linear_bwd_check(gs, x, w, dy, z, "silu", offsets)
    _linear_bwd_check(gs, _strided(x, 3, 1), w, _strided(dy, 1, 1), None, "none", offsets)


@pytest.mark.parametrize("name", ["bf16", "fp32"])
def test_grouped_linear_many_groups(gs, name):
    """More groups than a wave has lanes, most of them empty or of one row,
    one of many; and rows that do not fill them."""
    gen, t = _gen(77), _dtype(name)
    rng = np.random.default_rng(3)
    sizes = rng.integers(0, 3, 200)
    sizes[150] = 2000
    sizes[:70] = 0
    offsets = [0] + np.cumsum(sizes).tolist()
    rows = offsets[-1] + 13
    x, w = _rand(gen, rows, 72, dtype=t), _rand(gen, 200, 88, 72, scale=0.2, dtype=t)
    bias = _rand(gen, 200, 88)
    dy, z = _rand(gen, rows, 88, dtype=t), _rand(gen, rows, 88, dtype=t)
    _linear_fwd_check(gs, x, w, bias, "relu", None, offsets)
    _linear_bwd_check(gs, x, w, dy, z, "gelu", offsets)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("inner,out", [(64, 256), (256, 64), (120, 136), (512, 248)])
def test_grouped_linear_many_rows(gs, name, inner, out):
    gen, t = _gen(79), _dtype(name)
    offsets = [3, 50000, 50000, 50001, 90000, 90040, 90040, 132000]
    rows = 132050
    x, w = _rand(gen, rows, inner, dtype=t), _rand(gen, 7, out, inner, scale=0.2, dtype=t)
    bias, residual = _rand(gen, 7, out), _rand(gen, rows, out, dtype=t)
    dy, z = _rand(gen, rows, out, dtype=t), _rand(gen, rows, out, dtype=t)
    _linear_fwd_check(gs, x, w, bias, "gelu", residual, offsets)
    _linear_bwd_check(gs, x, w, dy, z, "silu", offsets)


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("groups,inner,out", [(7, 600, 512), (64, 512, 512), (1, 1000, 760)])
def test_grouped_linear_backward_in_one_launch(gs, name, groups, inner, out):
    """Rows and columns enough for dx and dw in the largest tiles together:
    groups that are cut and joined, empty ones, rows of nobody."""
    gen, t = _gen(80 + groups), _dtype(name)
    sizes = np.random.default_rng(groups).integers(0, 2 * 40000 // groups, groups)
    sizes[groups // 2] = 0 if groups > 1 else 40000
    offsets = [2] + (2 + np.cumsum(sizes)).tolist()
    rows = max(offsets[-1] + 3, 39000)
    x, w = _rand(gen, rows, inner, dtype=t), _rand(gen, groups, out, inner, scale=0.1, dtype=t)
    dy, z = _rand(gen, rows, out, dtype=t), _rand(gen, rows, out, dtype=t)
    _linear_bwd_check(gs, x, w, dy, z, "silu", offsets)
    _linear_bwd_check(gs, x, w, dy, None, "none", offsets)
    # dw alone, in a launch of its own, has the same bits
    off = torch.tensor(offsets, dtype=torch.int64, device="cuda")
    _, dw, _ = gs.gs_grouped_linear_bwd(x, w, off, dy, z, gs.GS_ACT_SILU)
    only = torch.empty_like(dw)
    gs.gs_grouped_linear_bwd(x, w, off, dy, z, gs.GS_ACT_SILU, dw=only, want_dx=False)
    assert torch.equal(only, dw)


def test_grouped_linear_any_offsets_are_safe(gs):
    """Bounds below 0, past the rows and falling: clamped, and a bound below
    an earlier one counts as that one."""
    gen, t = _gen(78), torch.bfloat16
    offsets = [-5, 30, 20, 1 << 40, 50, -(1 << 50), 100]
    x, w = _rand(gen, 90, 64, dtype=t), _rand(gen, 6, 40, 64, scale=0.2, dtype=t)
    dy = _rand(gen, 90, 40, dtype=t)
    assert _spans(offsets, 90, 6) == [(0, 30), (30, 30), (30, 90), (90, 90), (90, 90), (90, 90)]
    _linear_fwd_check(gs, x, w, None, "none", None, offsets)
    _linear_bwd_check(gs, x, w, dy, None, "none", offsets)


# --- streams, graphs, repeats ---------------------------------------------------------

def _layer(gs, x, w, w3, off, gamma, beta, dy):
    """Everything once: the outputs of a small network forward and backward."""
    h, mean, rstd = gs.gs_layer_norm_fwd(x, gamma, beta)
    y1, z1 = gs.gs_linear_fwd(h, w, None, gs.GS_ACT_GELU, residual=x, save_z=True)
    y2, z2 = gs.gs_grouped_linear_fwd(y1, w3, off, None, gs.GS_ACT_SILU, save_z=True)
    d1, dw3, db3 = gs.gs_grouped_linear_bwd(y1, w3, off, dy, z2, gs.GS_ACT_SILU)
    d0, dw, db = gs.gs_linear_bwd(h, w, d1, z1, gs.GS_ACT_GELU)
    dx, dg, dbt = gs.gs_layer_norm_bwd(x, d0, gamma, mean, rstd, dres=d1)
    return [y1, y2, dx, dw3, db3, dw, db, dg, dbt]


def _layer_inputs(rows=3000, seed=21):
    gen, t = _gen(seed), torch.bfloat16
    off = torch.tensor([0, rows // 3, rows // 3, rows - 5, rows], dtype=torch.int64, device="cuda")
    return (_rand(gen, rows, 96, dtype=t), _rand(gen, 96, 96, scale=0.1, dtype=t),
            _rand(gen, 4, 59, 96, scale=0.1, dtype=t), off, 1 + _rand(gen, 96, scale=0.1), _rand(gen, 96),
            _rand(gen, rows, 59, dtype=t))


def test_repeats_and_streams_give_the_same_bits(gs):
    args = _layer_inputs()
    first = _layer(gs, *args)
    for a, b in zip(first, _layer(gs, *args)):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _layer(gs, *args)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    # a stream handed to the call, its tensors made on another one
    x, w = args[0], args[1]
    torch.cuda.synchronize()
    y = gs.gs_linear_fwd(x, w, None, gs.GS_ACT_GELU, residual=x, stream=side)
    side.synchronize()
    assert torch.equal(y, gs.gs_linear_fwd(x, w, None, gs.GS_ACT_GELU, residual=x))


def test_graph_replays_match_the_eager_calls(gs):
    args = _layer_inputs()
    _layer(gs, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _layer(gs, *args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _layer(gs, *args)
    for seed in (31, 32, 33, 34):
        fresh = _layer_inputs(seed=seed)
        for a, b in zip(args, fresh):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, _layer(gs, *fresh)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [37, 900, 140000])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_linear_backward_in_parts(gs, rows, act):
    """Each of dx, dw and db alone (the others NULL) has the bits it has
    beside the others; db without dw within fp32 roundings of it."""
    gen, t = _gen(rows), torch.bfloat16
    x, w = _rand(gen, rows, 72, dtype=t), _rand(gen, 40, 72, scale=0.2, dtype=t)
    dy, z = _rand(gen, rows, 40, dtype=t), _rand(gen, rows, 40, dtype=t)
    dx, dw, db = gs.gs_linear_bwd(x, w, dy, z, _act_id(gs, act))
    ws = torch.empty(gs.gs_linear_workspace_size(rows, 72, 40, 0, gs.GS_TYPE_BF16, _act_id(gs, act)),
                     dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream

    def call(dx=None, dw=None, db=None, x=x, w=w):
        st = gs.lib().gs_linear_bwd(None if x is None else x.data_ptr(), 72, None if w is None else w.data_ptr(), 72,
                                    z.data_ptr(), 40, dy.data_ptr(), 40, rows, 72, 40, 0, _act_id(gs, act),
                                    None if dx is None else dx.data_ptr(), 72, None if dw is None else dw.data_ptr(),
                                    0, None if db is None else db.data_ptr(), ws.data_ptr(), ws.numel(), s)
        assert st == gs.GS_OK, gs.gs_last_error()
    a, b, c = torch.zeros_like(dx), torch.zeros_like(dw), torch.zeros_like(db)
    call(dx=a, x=None)
    call(dw=b, w=None)
    call(db=c, x=None, w=None)
    call()
    assert torch.equal(a, dx) and torch.equal(b, dw)
    g = dy.double() * _slope(z.double(), act)
    _close(c, g.sum(0), 2 ** -18 * dy.double().abs().sum(0) + (rows + 4) * EPS32 * g.abs().sum(0), "db")
    # the norm's parts
    y, mean, rstd = gs.gs_layer_norm_fwd(x)
    ex, eg, eb = gs.gs_layer_norm_bwd(x, y, None, mean, rstd)
    ws = torch.empty(gs.gs_workspace_size(gs.GS_OP_LAYER_NORM_BWD, rows, 72), dtype=torch.uint8, device="cuda")
    for parts in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        out = [torch.zeros_like(v) if p else None for v, p in zip((ex, eg, eb), parts)]
        px, pg, pb = (None if v is None else v.data_ptr() for v in out)
        assert gs.lib().gs_layer_norm_bwd(x.data_ptr(), 72, y.data_ptr(), 72, None, mean.data_ptr(), rstd.data_ptr(),
                                          None, 0, rows, 72, 0, px, 72, pg, pb, ws.data_ptr(), ws.numel(),
                                          s) == gs.GS_OK
        for v, want in zip(out, (ex, eg, eb)):
            assert v is None or torch.equal(v, want)


# --- workspaces that hold anything ------------------------------------------------------

def _filled_workspace(gs, rows, inner, out, groups, t, act, byte):
    """A workspace whose every byte is `byte` (255: NaN wherever it is read
    as a number)."""
    kind = {torch.bfloat16: gs.GS_TYPE_BF16, torch.float16: gs.GS_TYPE_F16, torch.float32: gs.GS_TYPE_F32}[t]
    size = gs.gs_linear_workspace_size(rows, inner, out, groups, kind, _act_id(gs, act))
    return torch.full((size,), byte, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("inner,out", [(64, 64), (128, 72), (56, 256), (256, 256)])
@pytest.mark.parametrize("offsets", [[9, 9, 9], [35000, 35001], [7, 1007], [0, 6000], [20000, 23000, 23000, 25000],
                                     [1] + [39000 + 20 * e for e in range(40)]],
                         ids=["no rows", "one row", "a thousand", "six thousand", "three groups", "forty groups"])
def test_grouped_backward_of_few_rows_among_many(gs, name, inner, out, offsets):
    """Groups that cover a small part of the rows, in a workspace of NaN: dw
    and db hold the covered rows alone, whatever the workspace held."""
    t, rows, groups = _dtype(name), 40000, len(offsets) - 1
    gen = _gen(inner + out + groups)
    x, w = _rand(gen, rows, inner, dtype=t), _rand(gen, groups, out, inner, scale=0.2, dtype=t)
    dy, z = _rand(gen, rows, out, dtype=t), _rand(gen, rows, out, dtype=t)
    for act in ("none", "silu"):
        ws = _filled_workspace(gs, rows, inner, out, groups, t, act, 255)
        _linear_bwd_check(gs, x, w, dy, z if act != "none" else None, act, offsets, workspace=ws)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("groups", [0, 5])
@pytest.mark.parametrize("rows,inner,out", [(1, 4096, 4096), (60, 72, 59), (3000, 520, 40), (9000, 264, 520),
                                            (20000, 1024, 512), (40000, 512, 512), (70000, 64, 256), (70000, 256, 56),
                                            (33000, 251, 59)])
def test_linear_backward_reads_what_it_wrote(gs, name, groups, rows, inner, out):
    """The same bits from a workspace of zeros and from one of NaN, for every
    way the backward pass is cut."""
    t, act = _dtype(name), "gelu"
    gen = _gen(rows + inner + out + groups)
    lead = (groups,) if groups else ()
    x, w = _rand(gen, rows, inner, dtype=t), _rand(gen, *lead, out, inner, scale=0.2, dtype=t)
    dy, z = _rand(gen, rows, out, dtype=t), _rand(gen, rows, out, dtype=t)
    # one group long enough to be cut, one empty, a few rows of nobody
    cuts = [0, rows // 8, rows // 8, rows * 7 // 8, rows * 7 // 8 + 1, rows - rows // 100]
    off = torch.tensor([min(c, rows) for c in cuts], dtype=torch.int64, device="cuda")
    for a in (act, "none"):
        results = []
        for byte in (0, 255):
            ws = _filled_workspace(gs, rows, inner, out, groups, t, a, byte)
            zz = z if a != "none" else None
            dx = torch.zeros_like(x)
            results.append(gs.gs_grouped_linear_bwd(x, w, off, dy, zz, _act_id(gs, a), dx=dx, workspace=ws) if groups
                           else gs.gs_linear_bwd(x, w, dy, zz, _act_id(gs, a), dx=dx, workspace=ws))
        for zeros, nans in zip(*results):
            assert nans.isfinite().all() and torch.equal(zeros, nans)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,width", [(1, 7), (300, 515), (5000, 64), (40, 9001)])
def test_layer_norm_backward_reads_what_it_wrote(gs, name, rows, width):
    t, gen = _dtype(name), _gen(rows + width)
    x, dy = _rand(gen, rows, width, dtype=t), _rand(gen, rows, width, dtype=t)
    _, mean, rstd = gs.gs_layer_norm_fwd(x)
    results = []
    for byte in (0, 255):
        ws = torch.full((gs.gs_workspace_size(gs.GS_OP_LAYER_NORM_BWD, rows, width),), byte, dtype=torch.uint8,
                        device="cuda")
        results.append(gs.gs_layer_norm_bwd(x, dy, None, mean, rstd, workspace=ws))
    for zeros, nans in zip(*results):
        assert nans.isfinite().all() and torch.equal(zeros, nans)


@pytest.mark.parametrize("rows", [37, 3000, 40000])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_backward_of_frozen_weights(gs, rows, act):
    """want_dw false: dx alone, with the bits it has beside dw and db; what is
    passed in is written all the same."""
    gen, t = _gen(rows), torch.bfloat16
    x, w = _rand(gen, rows, 72, dtype=t), _rand(gen, 40, 72, scale=0.2, dtype=t)
    dy, z = _rand(gen, rows, 40, dtype=t), _rand(gen, rows, 40, dtype=t)
    off = torch.tensor([0, rows // 3, rows], dtype=torch.int64, device="cuda")
    w2 = torch.stack([w, -w])
    dx, dw, db = gs.gs_linear_bwd(x, w, dy, z, _act_id(gs, act))
    only = gs.gs_linear_bwd(x, w, dy, z, _act_id(gs, act), want_dw=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], dx)
    mine = gs.gs_linear_bwd(x, w, dy, z, _act_id(gs, act), dw=torch.empty_like(dw), want_dw=False)
    assert mine[2] is None and torch.equal(mine[1], dw)
    gx, gw, gb = gs.gs_grouped_linear_bwd(x, w2, off, dy, z, _act_id(gs, act))
    only = gs.gs_grouped_linear_bwd(x, w2, off, dy, z, _act_id(gs, act), want_dw=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], gx)
