"""attn_decode_paged where one CTA adds up many tiles of a row: a sum must not drift with the number of its terms.

Values near 1 make every error of a sum one of the result.  Keys and queries are multiples of 1/16, so that the products are exact and
a logit is off by its scaling alone.  Tolerance, besides half a step of the output's type, relative to sum p |v|: 4 x 2^-24 times the
largest logit (times 2: numerator and sum) plus 2^-20 (the exponential), 2^-17 (weights as two 16-bit parts), 2^-17 (8 tiles of 8
products added with a cut, each at most 2^-23 of a sum), 2^-18 (64 of those sums, rounded to nearest) and 2^-16 (a thread's sum of
512 weights, rounded to nearest)."""
import math

import pytest
import torch

import scaled_dot_product_sdpa_gb300 as gb
from reference64 import U, half_step

pytestmark = pytest.mark.gpu
B, KINDS = 304, 8  # sequences: as many as CTAs, of eight kinds


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from scaled_dot_product_sdpa_gb300 import build
    gb.load_library(build.build())
    assert gb.attn_last_device_error() == 0
    yield
    assert gb.attn_last_device_error() == 0


def quantised(shape, seed, most):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).double() / 16


def check_rows(dtype, d, G, k, v, q, table, lengths):
    """Rows of one key head: k, v [tokens, d] lie in pages of 128 in order, which `table` [entries] may name more than once."""
    kp, vp = (x.reshape(-1, 1, 128, d).cuda() for x in (k, v))
    kind = torch.arange(B) % KINDS
    o, lse = gb.attn_decode_paged(q[kind].cuda(), kp, vp, table[None].cuda().expand(B, -1), lengths[kind].cuda(), scale=0.25)
    s = (q.cuda().double() @ k.cuda().double().T) * 0.25  # [kinds, G, tokens]
    page = torch.arange(table.numel() * 128) // 128
    times = torch.zeros(KINDS, k.shape[0], dtype=torch.float64)  # how often each token occurs in a row
    for i, n in enumerate(lengths.tolist()):
        at = table[page[:n]].long() * 128 + torch.arange(n) % 128
        times[i].index_add_(0, at, torch.ones(n, dtype=torch.float64))
    s = s + times.log().cuda()[:, None]
    want, p = torch.logsumexp(s, -1), torch.softmax(s, -1)
    ow, size = p @ v.cuda().double(), p @ v.cuda().double().abs()
    off = 4 * U * float((s - times.log().cuda()[:, None]).abs().nan_to_num(0, 0, 0).max())
    tol = half_step(dtype, ow) + (2 * off + 2.0 ** -20 + 2 * 2.0 ** -17 + 2.0 ** -18 + 2.0 ** -16) * size
    err = (o.double() - ow[kind.cuda()]).abs() / tol[kind.cuda()]
    assert (err <= 1).all(), f"o {err.max():.2f} times the tolerance, {(err > 1).double().mean():.4f} of the values beyond it"
    err = (lse.double() - want[kind.cuda()]).abs() / (off + 2.0 ** -20 + 2.0 ** -16 + 2.0 ** -23 * want[kind.cuda()].abs())
    assert (err <= 1).all(), f"lse {err.max():.2f} times the tolerance"


SHAPES = [(64, 1), (64, 12), (64, 20), (128, 8), (128, 16), (128, 32), (256, 2), (256, 9), (256, 20), (512, 2), (512, 16)]


@pytest.mark.parametrize("d,G", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rows_of_many_tiles(dtype, d, G):
    """512 tiles to a row and CTA: 8192 tokens, eight times over."""
    tokens = 8192
    k = quantised((tokens, d), 1, 16).to(dtype)
    q = quantised((KINDS, G, d), 2, 16)
    q[..., 12:] = 0
    v = (1 + 0.1 * torch.randn(tokens, d, generator=torch.Generator().manual_seed(3))).to(dtype)
    lengths = torch.tensor([65536, 65000, 65535, 61441, 65409, 60000, 63999, 62000], dtype=torch.int32)
    check_rows(dtype, d, G, k, v, q.to(dtype), torch.arange(64, dtype=torch.int32).repeat(8), lengths)


@pytest.mark.parametrize("d,G", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rising_rows_of_many_tiles(dtype, d, G):
    """The maximum moves every fifth tile, by so little that all tiles count: between sums that are taken, and with them."""
    tiles = 45
    k = quantised((tiles * 128, d), 4, 8)
    k[:, 0] = torch.arange(tiles * 128) // 128 // 5
    q = quantised((KINDS, G, d), 5, 8)
    q[..., 8:] = 0
    q[..., 0] = 7
    v = (1 + 0.1 * torch.randn(tiles * 128, d, generator=torch.Generator().manual_seed(6))).to(dtype)
    lengths = torch.tensor([5760, 5759, 5633, 5400, 1025, 1024, 2049, 1153], dtype=torch.int32)
    check_rows(dtype, d, G, k.to(dtype), v, q.to(dtype), torch.arange(tiles, dtype=torch.int32), lengths)


def test_tables_with_room_for_more_than_lengths_can_say():
    """65536 sequences, each with a table of 2^30 pages of 2^24 tokens: the units of work that they have room for pass 2^63."""
    N, d, page, n = 65536, 64, 1 << 24, 300
    kp, vp = (torch.zeros(1, 1, page, d, dtype=torch.float16, device="cuda") for _ in range(2))
    kp[0, 0, :n], vp[0, 0, :n] = (quantised((2, n, d), 7, 8) + torch.tensor([0.0, 1.0])[:, None, None]).half().cuda()
    q = quantised((1, 1, d), 8, 8).half().cuda()
    table = torch.zeros(1, 1 << 30, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(N, dtype=torch.int32, device="cuda")
    lengths[[0, 777, N - 1]] = n
    o, lse = gb.attn_decode_paged(q.expand(N, 1, d), kp, vp, table.expand(N, -1), lengths)
    want = gb.attn_decode_paged(q, kp, vp, table[:, :1], lengths[:1])
    at = lengths > 0
    assert torch.isfinite(want[1]).all() and torch.equal(o[at], want[0].expand(3, 1, d)) and torch.equal(lse[at], want[1].expand(3, 1))
    assert (o[~at] == 0).all() and torch.isneginf(lse[~at]).all()
