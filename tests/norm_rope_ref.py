"""Norms and rotations in 64 bits, and how far a correct result may be from them."""
from __future__ import annotations

import torch

E4M3 = torch.float8_e4m3fn


def rounding(dtype) -> float:
    """Half a step, relative to the value."""
    return torch.finfo(dtype).eps / 2


def table(positions: int, rope: int, base: float = 10000.0):
    i = torch.arange(rope // 2, dtype=torch.float64)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-2 * i / max(rope, 1))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def normed(x, weight, eps):
    """x * weight / rms(x) over the last axis, and the relative error that float32 may make of it: each of the n
    squares and n - 1 sums of the mean is rounded once, which its root halves; then the division by n, eps, root,
    reciprocal and two products, each at most two units of 2^-24."""
    x, n = x.double(), x.shape[-1]
    y = x * weight.double() / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return y, (n / 2 + 1 + 12) * 2.0 ** -24


def rotated(x, angles, interleaved, rel):
    """x [T, .., R] float64 by angles [T, R], and the error of float32: values off by rel, two products and a sum."""
    half = x.shape[-1] // 2
    angles = angles.double().view(x.shape[0], *[1] * (x.dim() - 2), 2 * half)
    c, s = angles[..., :half], angles[..., half:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    ya, yb = a * c - b * s, b * c + a * s
    ea = ((a * c).abs() + (b * s).abs()) * (rel + 3 * 2.0 ** -24)
    eb = ((b * c).abs() + (a * s).abs()) * (rel + 3 * 2.0 ** -24)
    put = (lambda u, v: torch.stack([u, v], -1).flatten(-2)) if interleaved else (lambda u, v: torch.cat([u, v], -1))
    return put(ya, yb), put(ea, eb)


def queries(q, weight, nope, angles, interleaved, eps):
    """(nope, its error), (rope, its error) of heads q [T, H, P + R], before the last rounding."""
    x, rel = q.double(), 0.0
    if weight is not None:
        x, rel = normed(q, weight, eps)
    return (x[..., :nope], x[..., :nope].abs() * rel), rotated(x[..., nope:], angles, interleaved, rel)


def rows(kv, weight, angles, interleaved, eps):
    """Rows [c_kv | k_pe] of kv [T, L + R] and their error, before the last rounding."""
    latent = weight.shape[0]
    c, rel = normed(kv[:, :latent], weight, eps)
    pe, err = rotated(kv[:, latent:].double(), angles, interleaved, 0.0)
    return torch.cat([c, pe], 1), torch.cat([c.abs() * rel, err], 1)


def check(got, want, err, dtype, what):
    """got is want, off by err and one rounding to dtype (of a value that may be off by err)."""
    tol = err + rounding(dtype) * (want.abs() + err) + 2.0 ** -126
    off = (got.double().cpu() - want).abs() - tol
    assert not torch.isnan(off).any(), f"{what}: NaN"
    assert off.numel() == 0 or off.max() <= 0, f"{what}: {off.max():.3e} beyond its bound at {off.argmax()}"


def nearest(y):
    """The nearest e4m3 value: steps of 2^(exponent - 3), no exponent below -6, halves to even, saturating."""
    step = torch.exp2(y.abs().clamp_min(2.0 ** -20).log2().floor().clamp_min(-6) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def check_codes(got, want, err, what):
    """Rounding keeps order: a code lies between the codes of want - err and want + err."""
    v = got.cpu().view(E4M3).double()
    assert ((v >= nearest(want - err)) & (v <= nearest(want + err))).all(), what
