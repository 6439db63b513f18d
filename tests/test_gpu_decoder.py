"""The attribute decoder (differentiable_gaussian_splatting_dgs_amd/decoder.py):
the network operators together, and trained through the rasteriser."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _plain(dec, leaves):
    """forward() in 64 bits on the stored values, differentiable."""
    x = leaves["features"]
    c = x - x.mean(1, keepdim=True)
    n = c / ((c * c).mean(1, keepdim=True) + 1e-5).sqrt() * leaves["gamma"] + leaves["beta"]
    a = torch.nn.functional.gelu(n @ leaves["w1"].t() + leaves["b1"])
    h = x + a @ leaves["w2"].t() + leaves["b2"]
    off = dec.offsets.tolist()
    return torch.cat([h[s:e] @ leaves["heads"][b].t() + leaves["hb"][b]
                      for b, (s, e) in enumerate(zip(off[:-1], off[1:]))])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_decoder_gradients(dtype):
    """Against autograd in 64 bits.  Tolerance, in 2-norms: on the way from
    an input to a gradient no value is rounded into storage more than 8 times
    (norm, z's slope, activation, h, and their gradients), each by at most
    half a step; fp32 adds its sums, under 2^-16."""
    from differentiable_gaussian_splatting_dgs_amd.decoder import AttributeDecoder
    dec = AttributeDecoder([0, 700, 700, 1500, 2003], width=48, hidden=136, dtype=dtype, seed=3)
    leaves = {k: dec.stored.get(k, v).double().requires_grad_() for k, v in dec.masters.items()}
    want = _plain(dec, leaves)
    out = dec.forward()
    tol = 8 * torch.finfo(dtype).eps / 2 + 2.0 ** -16
    assert float((out.double() - want.detach()).norm() / want.detach().norm()) <= tol
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    d = torch.randn(out.shape, generator=gen, device="cuda").to(dtype)
    want.backward(d.double())
    dec.backward(d)
    for k, v in dec.masters.items():
        ref = leaves[k].grad
        err = float((v.grad.double() - ref).norm() / ref.norm())
        assert err <= tol, (k, err, tol)


def test_decoder_trains_through_the_rasteriser():
    from differentiable_gaussian_splatting_dgs_amd import decoder
    history = decoder.main(12)
    assert all(h == h for h in history)
    assert min(history[-3:]) < history[0]


def test_block_offsets():
    from differentiable_gaussian_splatting_dgs_amd.decoder import block_offsets
    pos = torch.tensor([[0.0, 3.9, 1.0, 4.0, 0.5, 2.1], [0.0] * 6, [0.0] * 6])
    order, off = block_offsets(pos, 4)
    assert off.tolist() == [0, 2, 3, 4, 6] and order.tolist() == [0, 4, 2, 5, 1, 3]
