"""The decoder with shared features and routed heads: the lookup, the gate,
the sort, routed rows and the optimiser's step as a program runs them."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _decoder(dtype, n=1200, rows=300, heads=7, seed=3, **kw):
    from differentiable_gaussian_splatting_dgs_amd.decoder import RoutedDecoder
    gen = torch.Generator()
    gen.manual_seed(seed)
    anchors = (torch.rand(n, generator=gen) ** 2 * rows).long()
    anchors[5] = -1
    return RoutedDecoder(anchors, rows, heads, width=48, hidden=136, dtype=dtype, seed=seed, **kw)


def _plain(dec, leaves, ids):
    """forward() in 64 bits on the stored values and the choices made, differentiable."""
    at = dec.anchors
    f = torch.where((at >= 0)[:, None], leaves["features"][at.clamp_min(0)], 0.0)
    c = f - f.mean(1, keepdim=True)
    n = c / ((c * c).mean(1, keepdim=True) + 1e-5).sqrt() * leaves["gamma"] + leaves["beta"]
    a = torch.nn.functional.gelu(n @ leaves["w1"].t() + leaves["b1"])
    h = f + a @ leaves["w2"].t() + leaves["b2"]
    p = torch.softmax((h @ leaves["gate"].t()).gather(1, ids), 1)
    ys = (leaves["heads"][ids] @ h[:, None, :, None])[..., 0] + leaves["hb"][ids]
    return (p[:, :, None] * ys).sum(1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("choices", [1, 2, 3])
def test_routed_decoder_gradients(dtype, choices):
    """Against autograd in 64 bits.  Tolerance, in 2-norms: 17 values between an
    input and a gradient are rounded into storage (8 on the way there, 9 on the
    way back), each by at most half a step; fp32 adds its sums, under 2^-16."""
    dec = _decoder(dtype, choices=choices)
    leaves = {k: dec.stored.get(k, v).double().requires_grad_() for k, v in dec.masters.items()}
    out = dec.forward()
    want = _plain(dec, leaves, dec._ids.long())
    tol = 17 * torch.finfo(dtype).eps / 2 + 2.0 ** -16
    assert float((out.double() - want.detach()).norm() / want.detach().norm()) <= tol
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    d = torch.randn(out.shape, generator=gen, device="cuda").to(dtype)
    want.backward(d.double())
    dec.backward(d)
    for k, v in dec.masters.items():
        ref = leaves[k].grad
        if k == "gate" and choices == 1:        # one choice's weight is 1 whatever its logit
            assert not bool(v.grad.any())
            continue
        err = float((v.grad.double() - ref).norm() / ref.norm())
        assert err <= tol, (k, err, tol)


@pytest.mark.parametrize("bits", [8, 32])
def test_optimizer_writes_what_kernels_read(bits):
    """A step moves every master against its gradient's sign and leaves the
    storage copies as sync() would."""
    dec = _decoder(torch.bfloat16)
    opt = dec.optimizer(lr=1e-3, weight_decay=0.0, bits=bits, min_8bit=1000)
    assert any(s[2] is not None for s in opt.state) == (bits == 8)
    before = {k: v.clone() for k, v in dec.masters.items()}
    dec.forward()
    dec.backward(torch.ones(1200, 64, device="cuda", dtype=torch.bfloat16))
    opt.step()
    for k, v in dec.masters.items():
        moved, g = v - before[k], v.grad
        assert bool((moved * g <= 0).all()) and bool((moved != 0).any()), k
        if k in dec.stored:
            assert torch.equal(dec.stored[k], v.to(torch.bfloat16)), k
    # zero_grad's way of leaving gradients, and a second pass
    for v in dec.masters.values():
        v.grad = None
    first = dec.forward()
    dec.backward(first)
    opt.step()
    assert opt.steps == 2 and bool(dec.forward().isfinite().all())


def test_routed_decoder_runs_through_the_rasteriser():
    from differentiable_gaussian_splatting_dgs_amd import decoder
    history = decoder.main(4, routed=True)
    assert len(history) == 4 and all(h == h for h in history)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_routed_gradients_through_the_rasteriser(dtype):
    """train_views' gradients are those of the network in 64 bits for the sum of
    the views' parameter gradients, as a TrainStep with the decoded parameters
    computes them.  Tolerance as in test_routed_decoder_gradients, with two
    roundings more (the attributes, the sum's storage); the atomic sums over
    pairs add fp32 roundings, under 2^-12 in a 2-norm."""
    import synth
    from differentiable_gaussian_splatting_dgs_amd import TrainStep
    from differentiable_gaussian_splatting_dgs_amd.decoder import RoutedDecoder, shared_rows
    work = synth.cut_down(synth.workload(2), 320, 180, n=20000)

    def fresh():
        return TrainStep(work.params, work.cameras, work.targets, work.w_l1, work.w_ssim, work.lr, work.beta1,
                         work.beta2, work.eps)

    step, check = fresh(), fresh()
    base = step.params.clone()
    dec = RoutedDecoder(shared_rows(work.params[:3], 5000), 5000, 6, width=32, hidden=64, dtype=dtype, seed=5)
    dec.masters["hb"][:, :3] += 0.05
    dec.masters["hb"][:, 11:14] += 0.3
    dec.train_views(step, base)
    assert torch.equal(step.params, base + dec.forward()[:, :59].t())
    check.params.copy_(step.params)
    for k in range(len(check.views)):
        check.forward_view(k)
        check.backward_view(k)
    leaves = {k: dec.stored.get(k, v).double().requires_grad_() for k, v in dec.masters.items()}
    d = torch.nn.functional.pad(check.grads.t().double(), (0, 64 - 59))
    _plain(dec, leaves, dec._ids.long()).backward(d)
    tol = 19 * torch.finfo(dtype).eps / 2 + 2.0 ** -12
    for k, v in dec.masters.items():
        ref = leaves[k].grad
        assert float(ref.norm()) > 0
        err = float((v.grad.double() - ref).norm() / ref.norm())
        assert err <= tol, (k, err, tol)


def test_shared_rows_and_refusals():
    from differentiable_gaussian_splatting_dgs_amd.decoder import RoutedDecoder, shared_rows
    at = shared_rows(torch.tensor([[3.0, -1.0, 5.0, 0.0, 4.0, 9.0]]), 3)
    assert at.tolist() == [1, 0, 2, 0, 1, 2]
    for bad in (dict(anchors=[0, 4]), dict(anchors=[-2]), dict(anchors=[[0]]), dict(choices=4), dict(choices=0)):
        with pytest.raises(ValueError):
            RoutedDecoder(**{**dict(anchors=[0, 1], rows=4, heads=3), **bad})
