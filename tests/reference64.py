"""What the operators' tests share: seeded values, rotary positions in 64 bits, and the bound on an output that was computed in
fp32 and rounded once."""
import torch

U = 2.0 ** -24  # half a step of fp32


def half_step(t, value):
    """The largest error of rounding `value` (float64) to type t."""
    f = torch.finfo(t)
    return value.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def pairs(rotary, interleaved):
    r = torch.arange(rotary // 2)
    return (2 * r, 2 * r + 1) if interleaved else (r, r + rotary // 2)


def turned(y, pos, inv_freq, factor, interleaved, sign=1.0):
    """y [B, H, L, d] float64, pos [B, L]: the turned rows and, per element, the sum of its terms' magnitudes."""
    i, j = pairs(2 * inv_freq.numel(), interleaved)
    a = pos.double()[:, None, :, None] * inv_freq
    c, s = factor * a.cos(), sign * factor * a.sin()
    z, size = y.clone(), y.abs()
    z[..., i] = y[..., i] * c - y[..., j] * s
    z[..., j] = y[..., j] * c + y[..., i] * s
    size[..., i] = size[..., j] = factor * (y[..., i].abs() + y[..., j].abs())
    return z, size


def check(got, want, size, what, depth=64):
    got = got.cpu()
    assert torch.isfinite(got).all(), what
    err = (got.double() - want).abs()
    tol = half_step(got.dtype, want) + depth * U * size
    assert (err <= tol).all(), f"{what}: {(err / tol).max():.2f} times the tolerance"


def draw(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)
