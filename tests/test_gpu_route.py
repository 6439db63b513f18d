"""The gate and routed rows against their definitions in 64 bits, alone and
together with the sort and the grouped linear layer.

Tolerances (u: half a step of storage):
 - a weight e^(l - m) / sum: the difference is one fp32 rounding, 2^-24 of at
   most |l - m| <= D, so e^ of it is off by (D + 1) 2^-24 of itself beside the
   function's own 2^-23; the sum of n terms by (n + 4) 2^-24; the division by
   2^-24.  (D + n + 12) 2^-24 of the weight covers both ends of the quotient;
 - the logits' gradient: products of weights with (k + 6) 2^-24 of the
   absolute terms more, and u;
 - y: k products and sums in fp32, (k + 3) 2^-24 of the absolute terms, and u;
 - dweights: an fp32 sum of `width` products, (width + 4) 2^-24 of the absolute
   terms; dys: one product (2^-24) and u."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from net_helpers import EPS32, TYPES, close, gen, half_step, padding, rand, strided, tiny

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def gs():
    import differentiable_gaussian_splatting_dgs_amd as mod
    return mod


# --- the gate -----------------------------------------------------------------------

def _logits(seed, rows, groups, t):
    """Ties, masked logits, and rows that are masked altogether or but for one."""
    g = gen(seed)
    x = rand(g, rows, groups, scale=2.0).mul_(4).round_().div_(4)
    x.masked_fill_(torch.rand(rows, groups, generator=g, device="cuda") < 0.2, -INF)
    x[rows // 3] = -INF
    x[rows // 2] = -INF
    x[rows // 2, groups // 2] = 1.0
    x[-1] = torch.where(torch.arange(groups, device="cuda") % 2 == 0, 0.0, -0.0)
    return x.to(t)


def _gate_plain(x, k, renorm):
    x = x.double()
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    none = top == -INF
    m = top[:, :1].masked_fill(none[:, :1], 0.0)
    e = (top - m).exp()
    total = (e if renorm else (x - m).exp()).sum(1, keepdim=True)
    return ids.masked_fill(none, -1), torch.where(none, 0.0, e / total.masked_fill(none[:, :1], 1.0))


def _check_gate(gs, x, k, renorm, **kw):
    ids, w = gs.gs_gate_fwd(x, k, renorm, **kw)
    want_ids, want = _gate_plain(x, k, renorm)
    assert torch.equal(ids.long(), want_ids)
    spread = 40       # no listed logits are further apart
    close(w, want, (spread + x.shape[1] + 12) * EPS32 * want.nan_to_num(0.0), "weights")
    return ids, w


GROUPS = [1, 2, 5, 8, 31, 64, 65, 100, 128, 250, 256, 257, 512, 700, 1024]


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("groups", GROUPS)
def test_gate(gs, name, groups):
    t = TYPES[name]
    for rows, k in ((1, 1), (70, min(2, groups)), (131, min(8, groups)), (37, min(16, groups)), (9, min(3, groups))):
        x = _logits(rows + groups, rows, groups, t)
        for renorm in (True, False):
            ids, w = _check_gate(gs, x, k, renorm)
            assert _check_gate(gs, strided(x, 3, 1), k, renorm, ids=ids, weights=w)[0] is ids
            _check_gate_bwd(gs, x, ids, w, renorm)


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("groups,rows", [(20, 300_000), (32, 270_001), (33, 230_001), (40, 212_000), (64, 150_001), (65, 120_000),
                                         (128, 70_003), (250, 40_003), (256, 34_001), (500, 20_000), (512, 18_001),
                                         (700, 12_007), (1024, 9_001)])
def test_gate_of_many_rows(gs, name, groups, rows):
    """Rows enough for four waves for each SIMD: a row's lanes hold more of it then."""
    rows *= 1 if name == "fp32" else 2
    x = _logits(groups, rows, groups, TYPES[name])
    for k, renorm in ((1, True), (2, False), (4, True), (8, False), (8, True), (16, False), (13, True)):
        _check_gate(gs, x, k, renorm)
    _check_gate(gs, strided(x, 3, 1), 7, False)


def _check_gate_bwd(gs, x, ids, w, renorm, **kw):
    rows, k = ids.shape
    dw = rand(gen(rows), rows, k)
    got = gs.gs_gate_bwd(x, ids, w, dw, renorm, **kw)
    t = x.dtype
    xd, there = x.double(), ids >= 0
    at = torch.where(there, ids, 0).long()
    part = torch.where(there, w.double() * dw.double(), 0.0)
    s, size = part.sum(1, keepdim=True), part.abs().sum(1, keepdim=True)
    if renorm:
        p = torch.zeros_like(xd)
        mine = part - torch.where(there, w.double(), 0.0) * s
    else:
        p = torch.softmax(xd, 1).nan_to_num(0.0)
        mine = part
    want = (-p * s).scatter_add(1, at, mine)
    terms = (p * size).scatter_add(1, at, part.abs() + torch.where(there, w.double(), 0.0) * size)
    close(got, want, (half_step(t) + EPS32) * want.abs() + (40 + x.shape[1] + k + 20) * EPS32 * terms + tiny(t),
          "dlogits")
    return got, dw


def test_gate_backward_strided(gs):
    x = strided(_logits(1, 50, 70, torch.float16), 5, 1, fill=INF)
    for renorm in (True, False):
        ids, w = gs.gs_gate_fwd(x, 4, renorm)
        out = strided(torch.full((50, 70), 3.0, dtype=torch.float16, device="cuda"), 3, 1, fill=7.0)
        assert _check_gate_bwd(gs, x, ids, w, renorm, dlogits=out)[0] is out
        assert bool((padding(out) == 7.0).all())


def test_gate_infinities_and_nan(gs):
    for t in TYPES.values():
        x = torch.zeros(5, 20, dtype=t, device="cuda")
        x[0, 7], x[1, 3], x[1, 9], x[2, 4] = INF, float("nan"), INF, -float("nan")
        x[3] = -INF
        x[4, 11] = torch.finfo(t).min     # the lowest number is a logit like others
        x[4, :11], x[4, 12:] = -INF, -INF
        for renorm in (True, False):
            ids, w = gs.gs_gate_fwd(x, 3, renorm)
            assert ids[:, 0].tolist() == [7, 3, 4, -1, 11]
            assert ids[1, :2].tolist() == [3, 9] and ids[3].tolist() == [-1] * 3 and ids[4].tolist() == [11, -1, -1]
            assert bool(w[:3].isnan().any(1).all()) and w[3].tolist() == [0.0] * 3 and w[4].tolist() == [1.0, 0.0, 0.0]


@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_against_differences(gs, renorm):
    """fp32, steps of h = 2^-8 on logits whose choice no step changes: the central
    difference of sum(w dw) is off by h^2 / 6 times a third derivative (under 8 sum
    |dw|), and by the weights' roundings, (40 + 12 + 12) 2^-24 sum |dw|, over h."""
    groups, k, h = 12, 3, 2.0 ** -8
    x = torch.randperm(groups, generator=gen(1), device="cuda").float()[None] * 0.25
    ids, w = gs.gs_gate_fwd(x, k, renorm)
    dw = rand(gen(2), 1, k)
    got = gs.gs_gate_bwd(x, ids, w, dw, renorm)
    step = torch.eye(groups, device="cuda") * h
    d = dw.expand(groups, k).contiguous().double()
    up, down = (gs.gs_gate_fwd((x + s * step).contiguous(), k, renorm) for s in (1, -1))
    assert torch.equal(up[0], ids.expand(groups, k)) and torch.equal(down[0], up[0])
    want = ((up[1].double() - down[1].double()) * d).sum(1) / (2 * h)
    tol = (h * h * 8 / 6 + 64 * EPS32 / h) * float(dw.abs().sum())
    close(got[0], want, tol, "dlogits")


# --- routed rows ----------------------------------------------------------------------

def _picks(seed, rows, k, groups):
    g = gen(seed)
    ids = torch.rand(rows, groups, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    return ids.masked_fill_(torch.rand(rows, k, generator=g, device="cuda") < 0.1, -1)


def _check_routes(gs, x, place, w, residual, fill=0.0, shift=0):
    """All four calls; what no place names holds NaN before."""
    rows, k = place.shape
    width, t = x.shape[1], x.dtype
    lay = (lambda v, f: strided(v, 3, 1, fill=f)) if shift else (lambda v, f: v)
    there, at = place >= 0, place.clamp_min(0).long()
    named = torch.zeros(rows * k, dtype=torch.bool, device="cuda")
    named[place[there].long()] = True
    u, small = half_step(t), tiny(t)
    blank = torch.full((rows * k, width), 5.0, dtype=t, device="cuda")
    # dispatch
    xs = lay(blank.clone(), 7.0)
    assert gs.gs_dispatch_fwd(lay(x, INF), place, xs=xs) is xs
    assert bool((xs[~named] == 5.0).all())
    assert torch.equal(xs[place[there].long()], x[there.nonzero()[:, 0]])
    assert not shift or rows * k == 1 or bool((padding(xs) == 7.0).all())
    # combine
    g = gen(rows + width)
    ys = rand(g, rows * k, width, dtype=t)
    ys[~named] = float("nan")
    taken = torch.where(there[:, :, None], ys[at].double(), 0.0)
    wd = torch.where(there, torch.ones_like(w).double() if w is None else w.double(), 0.0)[:, :, None] \
        if w is not None else there.double()[:, :, None]
    want, size = (wd * taken).sum(1), (wd.abs() * taken.abs()).sum(1)
    if residual is not None:
        want, size = want + residual.double(), size + residual.double().abs()
    tol = u * want.abs() + (k + 3) * EPS32 * size + small
    y = gs.gs_combine_fwd(lay(ys, INF), place, w, residual=None if residual is None else lay(residual, INF))
    close(y, want, tol, "y")
    if residual is not None:      # in place
        y = lay(residual.clone(), 7.0)
        gs.gs_combine_fwd(ys, place, w, residual=y, y=y)
        close(y, want, tol, "y in place")
        dx = lay(residual.clone(), 7.0)
        gs.gs_dispatch_bwd(ys, place, dres=dx, dx=dx)
        plain = taken.sum(1) + residual.double()
        close(dx, plain, u * plain.abs() + (k + 3) * EPS32 * (taken.abs().sum(1) + residual.double().abs()) + small,
              "dx in place")
    dx = gs.gs_dispatch_bwd(ys, place)
    close(dx, taken.sum(1), u * taken.sum(1).abs() + (k + 3) * EPS32 * taken.abs().sum(1) + small, "dx")
    # combine's gradient
    dy = rand(g, rows, width, dtype=t)
    dys = lay(blank.clone(), 7.0)
    got, dw = gs.gs_combine_bwd(lay(dy, INF), lay(ys, INF), place, w, dys=dys)
    assert got is dys and bool((dys[~named] == 5.0).all())
    full = (wd * dy.double()[:, None, :]).reshape(-1, width)[there.reshape(-1)]
    close(dys[place.reshape(-1)[there.reshape(-1)].long()], full, (u + EPS32) * full.abs() + small, "dys")
    prod = dy.double()[:, None, :] * taken
    close(dw, prod.sum(2), (width + 4) * EPS32 * prod.abs().sum(2), "dweights")
    only, none = gs.gs_combine_bwd(dy, None, place, w, want_dw=False)
    assert none is None and torch.equal(only[named], dys[named])
    none, again = gs.gs_combine_bwd(dy, ys, place, w, want_dys=False)
    assert none is None and torch.equal(again, dw)


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("width", [1, 3, 4, 7, 8, 9, 64, 130, 255, 515, 1024, 2047, 4100])
def test_routed_rows(gs, name, width):
    t = TYPES[name]
    for rows, k, groups in ((1, 1, 4), (33, 2, 5), (65, 3, 300), (40, 5, 16), (21, 8, 64), (13, 16, 20)):
        g = gen(width + k)
        x, residual = rand(g, rows, width, dtype=t), rand(g, rows, width, dtype=t)
        w = torch.rand(rows, k, generator=g, device="cuda")
        place = gs.gs_group_sort(_picks(rows, rows, k, groups), groups)[2]
        _check_routes(gs, x, place, w, residual)
        _check_routes(gs, x, place, None, None, shift=1)


@pytest.mark.parametrize("rows,k,width,name", [
    (3001, 1, 258, "fp32"), (1500, 2, 261, "fp32"), (700, 2, 520, "bf16"), (2003, 1, 1000, "fp16"), (801, 2, 1025, "bf16"),
    (901, 4, 515, "fp32"), (5000, 2, 512, "bf16")])
def test_routed_rows_of_more_than_a_wave(gs, rows, k, width, name):
    g = gen(rows)
    x, residual = rand(g, rows, width, dtype=TYPES[name]), rand(g, rows, width, dtype=TYPES[name])
    w = torch.rand(rows, k, generator=g, device="cuda")
    place = gs.gs_group_sort(_picks(rows, rows, k, 24), 24)[2]
    _check_routes(gs, x, place, w, residual)
    _check_routes(gs, x, place, w, residual, shift=1)


def test_dispatch_beyond_the_caches(gs):
    """An output of over 2^28 bytes, whose stores go past the caches."""
    for rows, k, width, t in ((140_001, 2, 512, torch.bfloat16), (70_003, 3, 516, torch.float32)):
        x = rand(gen(k), rows, width, dtype=t)
        place = gs.gs_group_sort(_picks(1, rows, k, 16), 16)[2]
        there = place >= 0
        xs = torch.full((rows * k, width), 5.0, dtype=t, device="cuda")
        gs.gs_dispatch_fwd(x, place, xs=xs)
        want = torch.full_like(xs, 5.0)
        want[place[there].long()] = x[there.nonzero()[:, 0]]
        assert torch.equal(xs, want)


def test_routed_rows_all_dropped_and_no_rows(gs):
    x = rand(gen(1), 6, 40)
    place = torch.full((6, 2), -1, dtype=torch.int32, device="cuda")
    _check_routes(gs, x, place, torch.full((6, 2), float("nan"), device="cuda"), x)
    # places outside the rows count as left out
    bad = torch.tensor([[12, -2]] * 6, dtype=torch.int32, device="cuda")
    bad[0] = torch.tensor([2 ** 31 - 1, -2 ** 31])
    assert bool((gs.gs_dispatch_bwd(rand(gen(2), 12, 40), bad) == 0).all())
    xs = torch.full((12, 40), 3.0, device="cuda")
    gs.gs_dispatch_fwd(x, bad, xs=xs)
    assert bool((xs == 3.0).all())
    none = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 40, device="cuda")
    assert gs.gs_dispatch_fwd(e, none).shape == (0, 40) and gs.gs_combine_fwd(e, none).shape == (0, 40)
    assert [v.shape for v in gs.gs_combine_bwd(e, e, none)] == [(0, 40), (0, 2)]


def test_combine_infinities(gs):
    """An infinity or NaN reaches the rows that take it, a left out place none."""
    ys = torch.ones(6, 9, device="cuda")
    ys[1, 2], ys[4] = INF, float("nan")
    place = torch.tensor([[0, 1], [2, 4], [3, -1]], dtype=torch.int32, device="cuda")
    y = gs.gs_combine_fwd(ys, place, torch.tensor([[1.0, 1], [1, 1], [1, float("nan")]], device="cuda"))
    assert y[0, 2] == INF and bool(y[0, 3:].eq(2).all()) and bool(y[1].isnan().all()) and bool(y[2].eq(1).all())


def test_routed_rows_past_32_bits(gs):
    """Rows whose elements lie past 2^32."""
    rows, k, width = 40_000, 2, 60_000
    xs = torch.empty(rows * k, width, dtype=torch.bfloat16, device="cuda")
    place = torch.full((rows, k), -1, dtype=torch.int32, device="cuda")
    place[0], place[-1] = torch.tensor([79_999, 71_583]), torch.tensor([35_792, 0])
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    x[0], x[-1] = 3.0, 5.0
    gs.gs_dispatch_fwd(x, place, xs=xs)
    assert [float(xs[r].float().mean()) for r in (79_999, 71_583, 35_792, 0)] == [3.0, 3.0, 5.0, 5.0]
    y = gs.gs_combine_fwd(xs, place, torch.full((rows, k), 0.5, device="cuda"), y=x)
    assert float(y[0].float().mean()) == 3.0 and float(y[-1].float().mean()) == 5.0 and not bool(y[1:-1].any())
    dys, dw = gs.gs_combine_bwd(y, xs, place, dys=xs.clone())
    assert dw[0].tolist() == [9.0 * width] * 2 and dw[-1].tolist() == [25.0 * width] * 2


def test_combine_gradient_against_differences(gs):
    """combine is linear in ys and in the weights each, so that a difference over
    any step is the derivative, but for the roundings of y (fp32, (k + 3) 2^-24 of
    the absolute terms on either side) over twice the step."""
    rows, k, width = 30, 3, 50
    g = gen(11)
    place = gs.gs_group_sort(_picks(1, rows, k, 8), 8)[2]
    ys, w, dy = rand(g, rows * k, width), torch.rand(rows, k, generator=g, device="cuda"), rand(g, rows, width)
    dys = torch.zeros_like(ys)
    _, dw = gs.gs_combine_bwd(dy, ys, place, w, dys=dys)
    for d, h in ((rand(g, rows, k), 0.5), (rand(g, rows * k, width), 0.25)):
        if d.shape == w.shape:
            up, down, want = gs.gs_combine_fwd(ys, place, w + h * d), gs.gs_combine_fwd(ys, place, w - h * d), dw
        else:
            up, down, want = gs.gs_combine_fwd(ys + h * d, place, w), gs.gs_combine_fwd(ys - h * d, place, w), dys
        got = ((up.double() - down.double()) * dy.double()).sum() / (2 * h)
        want = (want.double() * d.double()).sum()
        there = place >= 0
        size = ((w.abs() + h * d.abs() if d.shape == w.shape else w)[:, :, None] *
                torch.where(there[:, :, None], ys.abs()[place.clamp_min(0).long()] + (0 if d.shape == w.shape else
                            h * d.abs()[place.clamp_min(0).long()]), 0.0)).sum(1)
        tol = 2 * ((k + 5) * EPS32 * size.double() * dy.double().abs()).sum() / (2 * h)
        # dw and dys themselves: sums of `width` products, and products
        tol += (width + 4) * EPS32 * float((size.double() * dy.double().abs()).sum()) * float(d.abs().max())
        assert abs(float(got - want)) <= float(tol)


def test_a_layer_of_routed_heads(gs):
    """Gate, sort, dispatch, grouped linear, combine, and the way back, as a
    user runs them, against autograd in 64 bits through the same choices;
    twice the same bits; and replayed from a graph.  Tolerance in 2-norms: at
    most 8 values between an input and a gradient are rounded into storage, and
    under 2^-16 for the sums in fp32."""
    rows, width, out, groups, k, t = 700, 72, 40, 9, 2, torch.bfloat16
    g = gen(5)
    s = dict(x=rand(g, rows, width, dtype=t), wr=rand(g, groups, width, scale=0.2, dtype=t),
             w=rand(g, groups, out, width, scale=0.1, dtype=t), b=rand(g, groups, out), dy=rand(g, rows, out, dtype=t))

    def layer():
        logits = gs.gs_linear_fwd(s["x"], s["wr"])
        ids, p = gs.gs_gate_fwd(logits, k)
        offsets, _, place = gs.gs_group_sort(ids, groups, want_order=False)
        xs = gs.gs_dispatch_fwd(s["x"], place)
        ys = gs.gs_grouped_linear_fwd(xs, s["w"], offsets, s["b"])
        y = gs.gs_combine_fwd(ys, place, p)
        dys, dp = gs.gs_combine_bwd(s["dy"], ys, place, p)
        dxs, dw, db = gs.gs_grouped_linear_bwd(xs, s["w"], offsets, dys)
        dl = gs.gs_gate_bwd(logits, ids, p, dp)
        dx, dwr, _ = gs.gs_linear_bwd(s["x"], s["wr"], dl)
        return ids, y, gs.gs_dispatch_bwd(dxs, place, dres=dx, dx=dx), dw, db, dwr

    def check(got):
        leaves = {n: s[n].double().requires_grad_() for n in ("x", "wr", "w", "b")}
        ids = got[0].long()
        logits = leaves["x"] @ leaves["wr"].t()
        p = torch.softmax(logits.gather(1, ids), 1)
        y = (p[:, :, None] * ((leaves["w"][ids] @ leaves["x"][:, None, :, None])[..., 0] + leaves["b"][ids])).sum(1)
        y.backward(s["dy"].double())
        tol = 8 * half_step(t) + 2.0 ** -16
        for a, want in zip(got[1:], (y.detach(), *(leaves[n].grad for n in ("x", "w", "b", "wr")))):
            assert float((a.double() - want).norm() / want.norm()) <= tol

    first = layer()
    check(first)
    assert all(torch.equal(a, b) for a, b in zip(layer(), first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out_ = layer()
    for n in range(4):
        s["x"].copy_(rand(gen(40 + n), rows, width))
        s["dy"].copy_(rand(gen(50 + n), rows, out))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out_, layer()))
        check(out_)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = layer()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, layer()))


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("groups", [3, 8, 12, 31, 64, 100, 250, 512, 700, 1024])
def test_gate_gradient_without_some_choices(gs, name, groups):
    """An id outside the groups is no choice, the first one or another: s is the
    sum over those that are left, and p stays the softmax of all logits, which
    may be far from 0 (fp16's largest is 65504, and what is left may be far
    below the row's largest).  Tolerances as above, with the sum over the row worked
    out again, which the n terms of the weight's bound hold as well."""
    t = TYPES[name]
    for shift, rows in ((0.0, 67), (300.0, 40), (-300.0, 41)):
        k = min(4, groups - 1)
        x = _logits(groups, rows, groups, torch.float32) + shift
        x = x.to(t)
        for renorm in (True, False):
            ids, w = gs.gs_gate_fwd(x, k, renorm)
            for drop in ([0], [0, 1], [k - 1], list(range(k)), [0, k - 1]):
                some, w_some = ids.clone(), w.clone()
                some[::2, drop] = -1
                w_some[::2, drop] = float("nan")      # of no choice: not read
                got, dw = _check_gate_bwd(gs, x, some, w_some, renorm)
                some[::4, drop] = groups + 5
                assert torch.equal(gs.gs_gate_bwd(x, some, w_some, dw, renorm), got)


def _check_weights(gs, x, k, renorm):
    """The weights within a bound that goes by how far each logit is from the
    largest.  (u = 2^-24, D the distance.)  The difference is off by u D, which
    makes e^ of it off by as much of itself, beside the function's 4 u; a sum's
    terms are off by 4 u and u times their distance, whose mean with the softmax's
    weights is at most ln n; at most 38 additions follow on each other (32 of a
    lane, 6 between lanes); the reciprocal's 2 u and the product's u.  Powers under
    2^-126 may become 0."""
    ids, w = gs.gs_gate_fwd(x, k, renorm)
    want_ids, want = _gate_plain(x, k, renorm)
    assert torch.equal(ids.long(), want_ids)
    xd = x.double()
    far = torch.where(want_ids >= 0, xd.amax(1, keepdim=True) - xd.gather(1, want_ids.clamp_min(0)), 0.0)
    n = k if renorm else x.shape[1]
    tol = (far + torch.tensor(float(n)).log() + 4 + 4 + 38 + 3) * EPS32 * want + 2.0 ** -126
    close(w, want, tol, "weights")
    return ids, w


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("spread", [0.1, 2.0, 20.0, 100.0, 1000.0])
@pytest.mark.parametrize("groups", [5, 16, 64, 100, 250, 256, 512, 1024])
def test_gate_of_far_logits(gs, name, spread, groups):
    """Logits up to thousands apart: powers of e that are subnormal, that are 0,
    and that still count; few rows, and rows that share lanes' registers."""
    t = TYPES[name]
    for rows in (201, 8 * 2 ** 20 // groups + 3):
        x = rand(gen(rows + groups), rows, groups, scale=spread).to(t)
        # next to where e^-D ends, 87.3 (the smallest normal) and 103.97 (0)
        x[3] = -torch.linspace(80.0, 110.0, groups, device="cuda").to(t)
        x[3, groups // 2] = 0.0
        for k, renorm in ((1, False), (min(2, groups), True), (min(5, groups), False), (min(8, groups), True)):
            ids, w = _check_weights(gs, x, k, renorm)
            if rows < 1000:
                _check_gate_bwd_far(gs, x, ids, w, renorm)


def _check_gate_bwd_far(gs, x, ids, w, renorm):
    """_check_gate_bwd with the distances counted: p = w0 e^(l - l0) is off by u
    times the distance and, with the weight's own bound, by under (110 + ln n + 60) u
    where it is above 2^-126."""
    rows, k = ids.shape
    dw = rand(gen(rows), rows, k)
    got = gs.gs_gate_bwd(x, ids, w, dw, renorm)
    xd, wd = x.double(), w.double()
    part = wd * dw.double()
    s, size = part.sum(1, keepdim=True), part.abs().sum(1, keepdim=True)
    p = torch.zeros_like(xd) if renorm else torch.softmax(xd, 1)
    mine = part - wd * s if renorm else part
    at = ids.long()
    want = (-p * s).scatter_add(1, at, mine)
    terms = (p * size).scatter_add(1, at, part.abs() + wd * size)
    tol = (half_step(x.dtype) + EPS32) * want.abs() + (110 + 7 + 60 + k + 6) * EPS32 * terms + tiny(x.dtype)
    # a power that became 0, and a weight that did
    close(got, want, tol + 2.0 ** -125 * (1 + size), "dlogits")


@pytest.mark.parametrize("name,rows,groups", [
    ("fp32", 20_003, 250), ("bf16", 20_003, 500), ("fp16", 20_003, 700), ("fp32", 20_003, 1024), ("bf16", 9_001, 1024),
    ("fp32", 40_003, 100), ("bf16", 70_001, 100), ("fp32", 140_003, 20), ("fp16", 140_001, 30), ("bf16", 300_001, 16), ("fp32", 300_001, 8),
    ("fp16", 600_001, 8), ("fp32", 600_001, 3), ("bf16", 600_001, 5)])
def test_gate_backward_of_many_rows(gs, name, rows, groups):
    """More rows than there are groups of lanes at a time, with a remainder: the
    rows that follow in the same lanes and the same part of LDS."""
    t = TYPES[name]
    x = _logits(rows, rows, groups, t)
    for k, renorm in ((min(2, groups), True), (min(8, groups), False), (min(16, groups), True), (1, False)):
        ids, w = gs.gs_gate_fwd(x, k, renorm)
        _check_gate_bwd(gs, x, ids, w, renorm)
    out = strided(torch.full((rows, groups), 3.0, dtype=t, device="cuda"), 3, 1, fill=7.0)
    ids, w = gs.gs_gate_fwd(x, min(3, groups), False)
    _check_gate_bwd(gs, strided(x, 5, 1, fill=INF), ids, w, False, dlogits=out)
    assert bool((padding(out) == 7.0).all())


def test_routing_of_the_most_rows(gs):
    """2^31 - 1 rows through the gate, and as many places."""
    n, step = 2 ** 31 - 1, 2 ** 28
    x = torch.zeros(n, 1, dtype=torch.bfloat16, device="cuda")
    x[0], x[2 ** 30], x[-1] = -INF, -INF, 3.0
    ids, w = gs.gs_gate_fwd(x, 1)
    assert [int(ids[i]) for i in (0, 1, 2 ** 30, n - 1)] == [-1, 0, -1, 0] and float(w[-1]) == 1
    assert sum(int((ids[a:a + step] == 0).sum()) for a in range(0, n, step)) == n - 2
    assert sum(int((w[a:a + step] == 1).sum()) for a in range(0, n, step)) == n - 2
    del w
    # every row one place on, the last one to the front
    place = ids
    for a in range(0, n, step):
        m = min(step, n - a)
        place[a:a + m, 0] = torch.arange(a + 1, a + m + 1, device="cuda", dtype=torch.int64).remainder_(n).int()
        x[a:a + m, 0] = (torch.arange(a, a + m, device="cuda") % 251).bfloat16()
    xs = gs.gs_dispatch_fwd(x, place)
    back = gs.gs_combine_fwd(xs, place)
    assert torch.equal(xs[1:2 ** 30], x[:2 ** 30 - 1]) and torch.equal(xs[2 ** 30:], x[2 ** 30 - 1:-1])
    assert torch.equal(xs[0], x[-1]) and torch.equal(back[:2 ** 30], x[:2 ** 30]) and torch.equal(back[2 ** 30:], x[2 ** 30:])
