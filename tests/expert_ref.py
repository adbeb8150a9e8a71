"""The experts' products in 64 bits, and how far the kernels may be from them.

The reference decodes the operands exactly and multiplies in fp64.  A kernel's fp32 sum of K products
is off by at most K steps of 2^-23 relative to the sum of their magnitudes (one rounding a product
and addition, each counted as a whole step, as the matrix units do not promise nearest); with block
scales each of the K/128 partial sums takes two more roundings (scale product, fused add), which
K + 8 covers.

The e4m3 matrix instruction adds something of its own: it brings each eight neighbouring products
to the exponent of their largest, 2^E, and drops what lies below 2^(E - 13) (measured: beside a
product of 2^16 one of 2^3 counts and one of 1.5 * 2^2 does not, in aligned groups of eight; its
accumulators are fp32).  The largest product itself has 8 significant bits and loses nothing, so a
group loses less than 7 * 2^-13 times its largest product, which is at most the product of the
largest values of its two operands.

Storing in bf16 adds 2^-8 of the value, in e4m3 2^-4 of it or, below e4m3's normal range, 2^-10 of the
block's scale (half its smallest step, 2^-9)."""
from __future__ import annotations

import torch

E4M3 = torch.float8_e4m3fn
STEP = 2.0 ** -23


def decode(v, scale, fp8):
    """float64 values of bf16 rows, or of e4m3 codes with a scale per 128."""
    if not fp8:
        return v.view(torch.bfloat16).double()
    return v.view(E4M3).double() * scale.double().repeat_interleave(128, -1)


def decode_weight(w, scale, fp8):
    """float64 values of one expert's matrix (C x K)."""
    if not fp8:
        return w.view(torch.bfloat16).double()
    s = scale.double().repeat_interleave(128, 0)[: w.shape[0]].repeat_interleave(128, 1)
    return w.view(E4M3).double() * s


def product(x, w, fp8):
    """(x . w^T, the bound on a kernel's sums) in float64."""
    bound = (x.shape[1] + 8) * STEP * (x.abs() @ w.abs().T)
    if fp8:
        x8, w8 = (v.abs().unflatten(1, (-1, 8)).amax(-1) for v in (x, w))
        bound = bound + 7 * 2.0 ** -13 * (x8 @ w8.T)
    return x @ w.T, bound


def gated(x, w, fp8):
    """(h, bound) in float64: h = g / (1 + exp(-g)) * u.  silu's slope is at most 1.1; the kernel's
    exp is off by a step for each unit of |g| (its argument's rounding) and a few more, the division
    and products by four."""
    v, e = product(x, w, fp8)
    n = w.shape[0] // 2
    g, u, eg, eu = v[:, :n], v[:, n:], e[:, :n], e[:, n:]
    silu = g * torch.sigmoid(g)
    h = silu * u
    return h, 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (8 + g.abs()) * STEP * h.abs()


def check_bf16(name, got, want, bound):
    """got: bf16 rows as int16/bf16; want, bound: float64."""
    got = got.view(torch.bfloat16).double()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - want).abs() - (2.0 ** -8 * (want.abs() + bound) + bound)
    assert over.numel() == 0 or over.max() <= 0, f"{name}: {over.max()} over the bound at {over.argmax()}"


def check_e4m3(name, codes, scale, want, bound):
    """codes u8 [rows][I], scale f32 [rows][I/128] against h in float64."""
    if want.numel() == 0:
        return
    blocks = want.abs().unflatten(-1, (-1, 128))
    amax, slack = blocks.amax(-1), bound.unflatten(-1, (-1, 128)).amax(-1)
    ref = torch.where(amax > 0, amax / 448, 1.0)
    over = (scale.double() - ref).abs() - (slack / 448 + 2 * STEP * ref)
    assert over.max() <= 0, f"{name}: a scale is {over.max()} over its bound"
    got = decode(codes, scale, True)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    s = scale.double().repeat_interleave(128, -1)
    # the division by the scale rounds once more
    over = (got - want).abs() - (2.0 ** -4 * (want.abs() + bound) + 2.0 ** -10 * s + bound + 2 * STEP * want.abs())
    assert over.max() <= 0, f"{name}: {over.max()} over the bound"
    # the largest of a block takes the largest code
    top = codes.view(E4M3).double().abs().unflatten(-1, (-1, 128)).amax(-1)
    assert torch.equal(top, torch.where(amax > 0, 448.0, 0.0).double()), f"{name}: a block's largest code"


def quantise(v):
    """(u8 codes, fp32 scales) of fp32 rows, a scale per 128 values: test inputs only."""
    b = v.float().unflatten(-1, (-1, 128))
    amax = b.abs().amax(-1)
    s = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    return (b / s.unsqueeze(-1)).clamp(-448, 448).to(E4M3).flatten(-2).view(torch.uint8), s


def make_weights(g, E, C, K, fp8):
    """Test weights on the host: bf16 as int16, or u8 codes and [E][ceil(C/128)][K/128] scales."""
    w = torch.randn((E, C, K), generator=g) * K ** -0.5
    if not fp8:
        return w.to(torch.bfloat16).view(torch.int16), None
    Cb = -(-C // 128)
    s = torch.rand((E, Cb, K // 128), generator=g) * 0.01 + 0.002
    full = s.repeat_interleave(128, 1)[:, :C].repeat_interleave(128, 2)
    return (w / full).clamp(-448, 448).to(E4M3).view(torch.uint8), s


def make_rows(g, shape, fp8):
    x = torch.randn(shape, generator=g)
    if not fp8:
        return x.to(torch.bfloat16).view(torch.int16), None
    return quantise(x)
