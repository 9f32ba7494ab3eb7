"""attn_decode_tree's sums of weighted values: where they would leave fp32, and in rows of many tiles."""
import math

import pytest
import torch

import scaled_dot_product_sdpa_gb300 as gb
from reference64 import U, half_step
from test_tree_gpu import _lib, call, problem  # noqa: F401 (_lib is a fixture)
from tree_reference import attention, check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,d,Hq,T,old", [
    (2, 64, 2, 9, 3000), (2, 64, 8, 20, 3000), (2, 128, 8, 4, 3000), (2, 128, 4, 20, 3000), (2, 128, 4, 60, 3000), (2, 256, 2, 9, 3000), (2, 256, 4, 30, 3000),
    (2, 512, 2, 5, 3000), (2, 512, 1, 60, 3000), (160, 64, 1, 9, 700), (160, 64, 8, 20, 700), (160, 128, 1, 4, 700), (160, 128, 1, 40, 700), (160, 256, 1, 4, 700)])
@pytest.mark.parametrize("least,most", [(1e38, 3.3e38), (1e-20, 3e-20)])
def test_values_of_one_sign(B, d, Hq, T, old, least, most):
    """bf16 values whose sums do not cancel: the result lies within the type, and so has every sum on the way to within fp32."""
    q, store, view, table, lengths, counts, m, seen = problem(B, Hq, 1, T, d, 16, "heads", torch.bfloat16, "own", old, full=True)
    v = view(store)[1]
    v.copy_((torch.rand(v.shape, generator=torch.Generator().manual_seed(9)).double() * (most - least) + least).to(torch.bfloat16))
    got = call(q.cuda(), store.cuda(), view, table, lengths, counts, m)
    check_attention(got, attention(q, *view(store), table, lengths, counts, seen, 1 / math.sqrt(d)), max(lengths), d, "values of one sign", Hq * T)


def one_row_a_cta(k, v, q, older, scale, short=False, more=0):
    """attn_decode_tree's results for sequences of one key head, as many as CTAs (`short`: fewer, so that they are cut; and `more`), all alike: tokens
    `older` (numbers of pages of k, v [pages, page, d], one after the other) and then new ones, the last rows of k and v, as a
    chain; q [Hq, T, d].  Beside it 64 bits: o, lse, and per element sum p |v|."""
    Hq, T, d = q.shape
    P, page, _ = k.shape
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B = (sms * 2 // 3 if short else sms) + more
    last = -(-T // page)
    n = older.numel() * page + T
    table = torch.cat([older.int(), torch.arange(P - last, P, dtype=torch.int32)]).cuda()[None].expand(B, -1)
    got = gb.attn_decode_tree(q.cuda()[None].expand(B, -1, -1, -1).contiguous(), k.cuda()[:, None], v.cuda()[:, None], table, torch.full((B,), n, dtype=torch.int32, device="cuda"),
                              scale=scale)
    kd, vd, qd = (x.cuda().double() for x in (k, v, q))
    times = torch.zeros(P, dtype=torch.float64).index_add_(0, older, torch.ones(older.numel(), dtype=torch.float64)).cuda()
    x = scale * (qd @ kd.flatten(0, 1).T)  # [Hq, T, tokens of all pages]
    fresh = scale * (qd @ kd[P - last:].flatten(0, 1)[:T].T)
    S = scale * (qd.abs() @ kd.flatten(0, 1).abs().T).amax(-1)
    x = torch.cat([x + times.log().repeat_interleave(page), torch.where(torch.ones(T, T, dtype=torch.bool).tril().cuda(), fresh, -math.inf)], -1)
    p, values = torch.softmax(x, -1), torch.cat([vd.flatten(0, 1), vd[P - last:].flatten(0, 1)[:T]])
    return got, p @ values, torch.logsumexp(x, -1), p @ values.abs(), S, n


def rows_alike(got, o, lse, tol, lse_tol, what):
    err = (got[0].double() - o).abs() / tol
    assert (err <= 1).all(), f"{what}: o {err.max():.2f} times the tolerance, {(err > 1).double().mean():.4f} of the values beyond it"
    err = (got[1].double() - lse).abs() / lse_tol
    assert (err <= 1).all(), f"{what}: lse {err.max():.2f} times the tolerance"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,n", [(64, 1 << 22), (128, 1 << 22), (256, 1 << 21), (512, 1 << 20)])
@pytest.mark.parametrize("Hq,T", [(1, 2), (1, 40), (2, 90)])
def test_long_tails_behind_few_large_weights(dtype, d, n, Hq, T):
    """One token of each of the first two tiles has weight 1 and a value of zero, all others have weights of 2^-36.2, which fp16 cannot hold
    beside it (scaled by 2^11: half the smallest number is 2^-36), and values that they alone decide.  All of these tails' weights are
    alike, so that errors would not average out.
    Tolerance of o, beside half a step: of sum p |v|, twice a logit's error ((d + 8) 2^-24 S), 2^-20 (the exponential, the sums), 2^-17 or half
    a step of the type (weights), 2^-10 (sums that are cut off over up to 512 tiles); and in fp16, for the runs of up to 64 tiles that hold
    the large weights, 2^-36 a token, of which a run has 2^13 and each of the two large weights one: 2^-23 of the largest value."""
    page = 1 << 14
    k, v = torch.zeros(3, page, d), (torch.rand(3, page, d, generator=torch.Generator().manual_seed(1)) + 1) * 3e4
    k[0, [0, 128], 0] = 25.09
    v[0, [0, 128]] = 0
    q = torch.zeros(Hq, T, d)
    q[..., 0] = 8
    older = torch.cat([torch.zeros(1, dtype=torch.long), torch.ones(n // page - 1, dtype=torch.long)])
    got, o, lse, size, S, n = one_row_a_cta(k.to(dtype), v.to(dtype), q.to(dtype), older, 0.125)
    rows = Hq * T
    logit = (d + 8) * U * S
    share = 2 * logit + 2.0 ** -20 + (2.0 ** -17 if rows <= 32 else torch.finfo(dtype).eps / 2) + 2.0 ** -10
    tol = half_step(dtype, o) + share[..., None] * size + (2.0 ** -23 * 6e4 if dtype == torch.float16 else 0)
    rows_alike(got, o, lse, tol, logit + 2.0 ** -20 * (1 + lse.abs()), "tails")


# Up to 32 rows of a key head, 33 to 128, more (d <= 128: two row tiles that share each key tile).
ROWS = [(4, 6), (2, 30), (1, 140)]


def run_of(rows, dtype):
    """Tiles whose sums stay in an accumulator."""
    return 8 if rows <= 32 else 64 if dtype == torch.float16 else 128


def half_a_step(dtype, value, off):
    """The largest error of rounding a number within `off` of `value` (both normal): half the distance of its neighbours, not of a power of two's."""
    return torch.exp2(torch.floor(torch.log2(value.abs() + off))) * (torch.finfo(dtype).eps / 2)


def values(shape, g):
    """Values around a mean of each column's own, below 2 (so that the results lie anywhere between two numbers of their type)."""
    return (1.6 + 0.3 * torch.rand(shape[-1], generator=g)) * (1 + 0.05 * torch.randn(shape, generator=g))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("Hq,T", ROWS)
@pytest.mark.parametrize("short", [False, True])
def test_weights_of_powers_of_two_over_many_tiles(dtype, d, Hq, T, short):
    """Weights of 1, 1/2, ... 2^-14, drawn at random: each fits its type, so that o is off by what its sums lose, and products with 8 or 11 bits
    of a value reach below the sums' last bits.
    Tolerance beside half a step, of sum p |v| (v > 0): a run's 16 products a tile (8 where weights have one part) are cut off by up
    to 2^-23 of the sum at the time, whose mean is half of the run's; the sums of values and of weights are rounded to nearest where a run's
    joins them, 2^-24 of what there is, half of that in the mean; 2^-20 for the rest (an exponent is off by up to 14 2^-24)."""
    page, tiles = 1 << 10, 1104
    g = torch.Generator().manual_seed(d + T)
    k, v = torch.zeros(9, page, d), values((9, page, d), g)
    k[..., 0] = -torch.randint(0, 15, (9, page), generator=g)
    q = torch.zeros(Hq, T, d)
    q[..., 0] = 8
    older = torch.arange(8).repeat(tiles // 64)
    scale = float(torch.tensor(math.log(2) / 8, dtype=torch.float32))
    got, o, lse, size, S, n = one_row_a_cta(k.to(dtype), v.to(dtype), q.to(dtype), older, scale, short)
    rows, run = Hq * T, run_of(Hq * T, dtype)
    turns = tiles / 2 if d <= 128 and rows <= 128 else tiles
    off = (run * (16 if rows <= 32 else 8) * U + turns / run * U + 2.0 ** -20) * size
    rows_alike(got, o, lse, half_a_step(dtype, o, off) + off, 2.0 ** -20 * (1 + lse.abs()), "powers of two")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("Hq,T", ROWS)
@pytest.mark.parametrize("short", [False, True])
def test_maxima_that_rise_and_fall_over_many_tiles(dtype, d, Hq, T, short):
    """Logits of about +-12 that change from page to page, 64 pages in an order drawn at random: runs of tiles whose maxima lie far apart, in
    either order.  Tolerance, beside half a step: of sum p |v|, twice a logit's error, 2^-20 (the exponential), the weights' rounding, 16 products a
    tile of a run (8 where the weights have one part) cut off by 2^-23 of its sum each, and all sums' roundings to nearest (32 weights one after
    the other, moves of the maximum in a run, runs); in fp16 the floor of small weights, 2^-36 a token of a run: 2^-23 of the largest value."""
    page, tiles = 1 << 10, 400
    g = torch.Generator().manual_seed(d + T)
    k, v = 0.3 * torch.randn(65, page, d, generator=g), values((65, page, d), g)
    k[..., 0] = 24 * torch.rand(65, 1, generator=g) - 12
    q = torch.randn(Hq, T, d, generator=g)
    q[..., 0] = 8
    older = torch.randint(0, 64, (tiles // 8,), generator=g)
    got, o, lse, size, S, n = one_row_a_cta(k.to(dtype), v.to(dtype), q.to(dtype), older, 0.125, short)
    rows, run = Hq * T, run_of(Hq * T, dtype)
    logit, rounded = (d + 8) * U * S, 2 * (32 + run + tiles / run) * U
    share = 2 * logit + 2.0 ** -20 + (2.0 ** -17 if rows <= 32 else torch.finfo(dtype).eps / 2) + run * (16 if rows <= 32 else 8) * 2 * U + rounded
    off = share[..., None] * size + (2.0 ** -23 * 4 if dtype == torch.float16 else 0)
    rows_alike(got, o, lse, half_a_step(dtype, o, off) + off, logit + 2.0 ** -20 * (1 + lse.abs()) + rounded, "moving maxima")
