"""Inverse frequencies of rotary positions, for contexts as long as the trained one and longer."""
from __future__ import annotations

import math

import torch


def attn_rope_frequencies(rotary: int, base: float = 10000.0, scaling: str | None = None, scale: float = 1.0,
                          trained_length: int | None = None, fast_turns: float = 32.0, slow_turns: float = 1.0,
                          device="cuda"):
    """(inv_freq, factor) for attn_rope: float64 [rotary / 2] on `device`, and the factor on cosine and sine.

    Unscaled, inv_freq[r] = base^(-2r / rotary).  For a context `scale` (>= 1) times the trained one:
      "linear": every frequency divided by `scale` (positions interpolated);
      "base":   base raised to base * scale^(rotary / (rotary - 2)), which slows the slowest pair by `scale`
                and leaves the fastest alone;
      "parts":  pairs that make at least `fast_turns` turns over `trained_length` positions keep their
                frequency, those that make at most `slow_turns` are divided by `scale`, those between are
                blended linearly over the pair's index; factor = 0.1 ln(scale) + 1 (the YaRN method)."""
    if rotary < 2 or rotary % 2:
        raise ValueError("gbattn: rotary must be even and at least 2")
    if not (math.isfinite(base) and base > 1.0) or not (math.isfinite(scale) and scale >= 1.0):
        raise ValueError("gbattn: base must be above 1 and scale at least 1")
    r = torch.arange(rotary // 2, dtype=torch.float64)
    factor = 1.0
    if scaling == "base":
        if rotary == 2:
            raise ValueError("gbattn: scaling 'base' needs rotary above 2")
        base = base * scale ** (rotary / (rotary - 2))
    inv_freq = torch.pow(torch.tensor(base, dtype=torch.float64), -2.0 * r / rotary)
    if scaling == "linear":
        inv_freq = inv_freq / scale
    elif scaling == "parts":
        if not trained_length or trained_length <= 0 or not 0 < slow_turns < fast_turns:
            raise ValueError("gbattn: scaling 'parts' needs trained_length and 0 < slow_turns < fast_turns")
        # Pair r turns trained_length base^(-2r / rotary) / 2 pi times: the index with a given number.
        low, high = (rotary * math.log(trained_length / (2.0 * math.pi * n)) / (2.0 * math.log(base))
                     for n in (fast_turns, slow_turns))
        low, high = max(math.floor(low), 0), min(math.ceil(high), rotary - 1)
        slowed = ((r - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        inv_freq = inv_freq * (1.0 - slowed) + inv_freq / scale * slowed
        factor = 0.1 * math.log(scale) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError("gbattn: scaling must be None, 'linear', 'base' or 'parts'")
    elif scaling is None and scale != 1.0:
        raise ValueError("gbattn: a scale needs a scaling")
    return inv_freq.to(device), factor
