"""attn_decode_tree on rows that take a CTA longer than a bounded wait lasts (2^32 cycles, about two seconds)."""
import math

import pytest
import torch

import scaled_dot_product_sdpa_gb300 as gb
from reference64 import U, draw, half_step
from test_tree_gpu import _lib  # noqa: F401 (a fixture)
from test_tree_sums_gpu import one_row_a_cta, rows_alike

pytestmark = pytest.mark.gpu


def test_a_unit_of_several_seconds_before_another():
    """One sequence more than CTAs, of 1.6 million tiles each: the first CTA has a whole one of them (about 3700 cycles a tile, 6e9 in all) and then
    a part of the second, whose queries wait for the first one's buffer (two row tiles of 128 leave room for one).  Tolerances as for other
    long rows, and 2^-24 a run of 64 tiles for sums that are rounded to nearest where a run's joins them."""
    T, d, page, tiles = 130, 128, 1 << 15, 1_600_000
    k, v = draw((2, page, d), torch.float16, 1), 1 + 0.1 * draw((2, page, d), torch.float16, 2)
    q = draw((1, T, d), torch.float16, 3, 0.5)
    got, o, lse, size, S, n = one_row_a_cta(k, v, q, torch.zeros(tiles * 128 // page, dtype=torch.long), 1 / math.sqrt(d), more=1)
    assert gb.attn_last_device_error() == 0
    logit, rounded = (d + 8) * U * S, tiles / 64 * U
    tol = half_step(torch.float16, o) + (2 * logit + 2.0 ** -11 + 2.0 ** -13 + rounded)[..., None] * size
    rows_alike(got, o, lse, tol, logit + 2.0 ** -20 * (1 + lse.abs()) + rounded, "seconds")
