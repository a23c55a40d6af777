"""Helpers of the tests of the operators around the routed experts: inputs,
64-bit references and the error bounds they are held to.

Bounds.  A rounding to a type is off by at most half a step, eps / 2 relative
to the value.  A product's terms are exact in fp32 (11-bit or 8-bit
significands); its n terms are added in fp32, each addition off by at most one
step of a partial sum, and no partial sum exceeds S = sum |a| |b| by more than
its own error: n 2^-23 S covers any order of the additions, also within a
matrix instruction.
"""
import math

import numpy as np
import torch

U32 = 2.0 ** -23  # one step of fp32, relative
SUBNORMAL = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def padded(t, pad, offset=0, fill=float("nan")):
    """t's values in a buffer with `pad` more elements a row and `offset` elements
    before the first, all of them `fill`: a strided, perhaps misaligned view."""
    ld = t.shape[-1] + pad
    rows = t.numel() // t.shape[-1] if t.shape[-1] else 0
    buf = torch.full((rows * ld + offset + 64,), fill, dtype=t.dtype, device=t.device)
    if t.dim() == 3:
        v = buf.as_strided(t.shape, (ld * t.shape[1], ld, 1), offset)
    else:
        v = buf.as_strided(t.shape, (ld, 1), offset)
    v.copy_(t)
    return v, buf


def bounded(got, want, bound, dtype, what=""):
    """|got - want| <= bound + the rounding of the result, element by element."""
    g = got.double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    if g.numel() == 0:
        return
    assert bool(torch.isfinite(g).all()), (what, "not finite")
    # the value before rounding lies within `bound` of `want`; 2% covers the
    # bound's own evaluation
    lim = 1.02 * (bound + half_step(dtype) * (want.abs() + bound)) + SUBNORMAL[dtype]
    over = ((g - want).abs() - lim).max().item()
    worst = ((g - want).abs() / lim).max().item()
    print(f"  {what}: largest error {worst:.3f} of its bound", flush=True)
    assert over <= 0, (what, worst)


def offsets_of(counts, device="cuda"):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=device)


def act64(z, name):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z * 1.0


def slope64(z, name):
    v = z.detach().clone().requires_grad_(True)
    with torch.enable_grad():
        (d,) = torch.autograd.grad(act64(v, name).sum(), v)
    return d
