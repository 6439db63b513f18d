"""What the GPU tests of the row operators share: inputs, strided layouts and
element-by-element bounds."""
import torch

EPS32 = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(t):
    """What rounding into t is off by, relative to the value."""
    return torch.finfo(t).eps / 2


def tiny(t):
    """... and half the smallest number, which counts for fp16."""
    return 2.0 ** -25 if t == torch.float16 else 0.0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def strided(t, extra, shift=0, fill=float("nan")):
    """t's values with a leading dimension `extra` longer, the padding `fill`,
    the first element `shift` elements into its allocation."""
    rows, width = t.shape
    buf = torch.full((rows * (width + extra) + shift,), fill, dtype=t.dtype, device=t.device)
    v = buf[shift:].as_strided((rows, width), (width + extra, 1))
    v.copy_(t)
    return v


def padding(t):
    """The elements between the rows of strided()'s result."""
    rows, width = t.shape
    return t.as_strided((rows - 1, t.stride(0) - width), (t.stride(0), 1), t.storage_offset() + width)


def close(got, want, tol, what):
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= tol)
    # the same infinities and NaN are equal
    bad &= ~((got == want) | (got.isnan() & want.isnan()))
    n = int(bad.sum())
    if n:
        i = int(bad.flatten().nonzero()[0])
        at = torch.as_tensor(tol, device=want.device).expand_as(want).flatten()[i].item()
        raise AssertionError(f"{what}: {n} of {bad.numel()} off, first at {i}: {got.flatten()[i].item()} for "
                             f"{want.flatten()[i].item()}, tolerance {at}")
