"""Plain 64-bit latent attention on the CPU, with the error bounds its GPU form has to keep.

Rounding to a type t is off by at most u = finfo(t).eps / 2, relative, and below its
smallest normal number by half the (constant) spacing there. The tensor cores
add 16 products at a time in fp32, so a sum over K terms is off by at most
(K / 16 + 8) * 2^-23 * sum |x||y| (truncating adds). From there:
  scores   e = (K / 16 + 8) * 2^-23 * scale * max_j sum |q||k|, the absolute error of a
           score and so the relative one of its weight
  output   the final rounding, and (u + 2 e + 2^-18) sum p |v|: the weights' rounding
           to t, the scores' error in numerator and denominator, and the fp32 sums,
           exponentials and rescalings
  lse      e + 2^-18 (1 + |lse|)
"""
import math

import torch


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(dtype, x):
    """Most that rounding the 64-bit values x to `dtype` moves them."""
    return half_step(dtype) * x.abs().clamp(min=torch.finfo(dtype).smallest_normal)


def attention(q, k, v, visible, scale, dtype):
    """q [R, D], k [S, D], v [S, V] (any type); row r sees keys j < visible[r].
    Returns (o, lse, o's bound, lse's bound), all 64-bit."""
    q, k, v = q.double(), k.double(), v.double()
    R, S = q.shape[0], k.shape[0]
    if S == 0:
        z = torch.zeros(R, v.shape[1], dtype=torch.float64)
        return z, torch.full((R,), -math.inf, dtype=torch.float64), z, torch.zeros(R, dtype=torch.float64)
    seen = torch.arange(S)[None] < torch.as_tensor(visible)[:, None]
    k = torch.where(seen.any(0)[:, None], k, 0.0)
    v = torch.where(seen.any(0)[:, None], v, 0.0)
    s = torch.where(seen, q @ k.T * scale, -math.inf)
    m = s.max(1, keepdim=True).values
    some = m > -math.inf
    p = torch.where(some, torch.exp(s - torch.where(some, m, 0.0)), 0.0)
    l = p.sum(1, keepdim=True)
    p = torch.where(some, p / torch.where(some, l, 1.0), 0.0)
    lse = torch.where(some, m + torch.log(torch.where(some, l, 1.0)), -math.inf)[:, 0]
    o = p @ v
    mag = torch.where(seen, q.abs() @ k.abs().T * scale, 0.0).max(1).values
    e = (q.shape[1] / 16 + 8) * 2.0 ** -23 * mag
    u = half_step(dtype)
    bound = rounding(dtype, o) + (u + 2 * e + 2.0 ** -18)[:, None] * (p @ v.abs())
    return o, lse, bound, torch.where(some[:, 0], e + 2.0 ** -18 * (1 + lse.abs()), 0.0)


def check(got, ref, bound, what):
    got, ref, bound = got.detach().double().cpu(), ref.double(), bound.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    bad = ~(same | ((got - ref).abs() <= bound))
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, first at {i}: "
                             f"{float(got[i])} for {float(ref[i])}, allowed {float(bound[i]):.3g}")


def rope_frequencies(dim, base, factor=1.0, original_ctx=4096, beta_fast=32.0, beta_slow=1.0):
    """Radians per position of each pair, 64-bit."""
    i = torch.arange(dim // 2, dtype=torch.float64)
    f = base ** (-2 * i / dim)
    if factor > 1:
        pair = lambda r: dim * math.log(original_ctx / (2 * math.pi * r)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), dim - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
    return f


def rotate(x, pos, freq, layout, amplitude=1.0):
    """x [T, ..., dim] rotated at positions pos [T]; returns (rotated, bound's magnitude |a| + |b|)."""
    x = x.double()
    ang = pos.double().reshape(-1, *[1] * (x.dim() - 1)) * freq
    c, s = amplitude * torch.cos(ang), amplitude * torch.sin(ang)
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if layout == "interleaved" else (x[..., :h], x[..., h:])
    y, z, mag = a * c - b * s, b * c + a * s, amplitude * (a.abs() + b.abs())
    if layout == "interleaved":
        return torch.stack((y, z), -1).flatten(-2), torch.stack((mag, mag), -1).flatten(-2)
    return torch.cat((y, z), -1), torch.cat((mag, mag), -1)
