"""The paged cache on the GPU: attn_cache_append, attn_cache_copy and attn_decode_paged against their definitions in 64 bits, and a
run of them together.

Tolerances.  Values and copies are exact.  Rotated keys and queries: as for attn_rope (tests/test_rope_gpu.py).  Decoding: o is
rounded once (half a step of its type).  Before that, with S the largest sum of |q_i k_i| scale over a row's keys: a logit is off by at
most (d + 8) 2^-24 S (d fp32 additions of exact products, scaling), a weight, relatively, by twice that (numerator and sum) plus
2^-20 (the exponential's approximation, the sums) plus 2^-17 (weights enter the second product as two 16-bit parts); so o by that times
sum p |v|, and lse by (d + 8) 2^-24 S + 2^-20 (1 + |lse|)."""
import math

import pytest
import torch

import scaled_dot_product_sdpa_gb300 as gb
from reference64 import U, check, draw, half_step, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from scaled_dot_product_sdpa_gb300 import build
    gb.load_library(build.build())
    assert gb.attn_last_device_error() == 0
    yield
    assert gb.attn_last_device_error() == 0


LAYOUTS = ["heads", "slots", "joint", "side", "heads_joint"]


def cache(layout, P, H, page, d, dtype, seed, fill=None):
    """k and v pages [P, H, page, d] on the CPU in one of the layouts of memory, and a function that moves both to the GPU as they lie."""
    shape, view = {"heads": ((2, P, H, page, d), lambda t: (t[0], t[1])),
                   "slots": ((2, P, page, H, d), lambda t: (t[0].transpose(1, 2), t[1].transpose(1, 2))),
                   "joint": ((P, 2, H, page, d), lambda t: (t[:, 0], t[:, 1])),
                   "side": ((P, page, H, 2 * d), lambda t: (t[..., :d].transpose(1, 2), t[..., d:].transpose(1, 2))),
                   "heads_joint": ((P, H, 2, page, d), lambda t: (t[:, :, 0], t[:, :, 1]))}[layout]
    t = draw(shape, dtype, seed) if fill is None else torch.full(shape, fill, dtype=dtype)
    return t, view


def tables(lengths, page, P, seed, extra=0):
    """Tables over random distinct pages; entries behind a sequence's last page are out of the cache."""
    need = [-(-n // page) for n in lengths]
    assert sum(need) <= P
    deal = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).tolist()
    width = max(1, max(need)) + extra
    t = torch.full((len(lengths), width), 1 << 30, dtype=torch.int32)
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor([deal.pop() for _ in range(n)], dtype=torch.int32)
    return t


# ------------------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("B,Hq,Hkv,L,d,page,layout", [
    (1, 0, 1, 1, 64, 8, "heads"), (3, 4, 2, 5, 128, 16, "slots"), (4, 7, 1, 1, 256, 24, "joint"), (2, 3, 3, 40, 64, 32, "side"),
    (1, 8, 8, 333, 128, 128, "heads_joint"), (2, 2, 1, 9, 512, 8, "heads"), (300, 4, 2, 1, 64, 16, "slots")])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("mode", ["plain", "turn", "norm"])
def test_append(B, Hq, Hkv, L, d, page, layout, dtype, mode):
    g = torch.Generator().manual_seed(3)
    counts = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
    counts[0] = L
    lengths = counts + torch.randint(0, 50, (B,), generator=g, dtype=torch.int32)
    P = sum(-(-int(n) // page) for n in lengths) + 2
    table = tables(lengths.tolist(), page, P, 4, extra=1)
    store, view = cache(layout, P, Hkv, page, d, dtype, 5)
    joint = draw((B, L, Hq + 2 * Hkv, d), dtype, 6)
    q, k, v = joint.transpose(1, 2).split([Hq, Hkv, Hkv], dim=1)
    wq, wk = draw((d,), dtype, 7), draw((d,), dtype, 8)
    inv_freq, _ = gb.attn_rope_frequencies(d // 2, device="cpu")
    if mode == "plain":
        q, Hq, inv_freq = None, 0, inv_freq[:0]
    norm = mode == "norm"
    there = store.cuda()
    on_gpu = joint.cuda().transpose(1, 2).split([joint.shape[2] - 2 * Hkv, Hkv, Hkv], dim=1)  # slices of one projection
    out = gb.attn_cache_append(*on_gpu[1:], *view(there), table.cuda(), lengths.cuda(), counts=counts.cuda(), q=on_gpu[0] if Hq else None,
                               inv_freq=inv_freq.cuda() if mode != "plain" else None, interleaved=layout == "slots", q_weight=wq.cuda() if norm and Hq else None,
                               k_weight=wk.cuda() if norm else None)
    pos = (lengths - counts)[:, None] + torch.arange(L)[None]

    def want(x, w):
        y = x.double()
        if norm:
            y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
        return turned(y, pos, inv_freq, 1.0, layout == "slots")

    kw, ksize = want(k, wk)
    expect, size = store.double(), torch.zeros_like(store, dtype=torch.float64)
    (ke, ve), (ks, _) = view(expect), view(size)
    for b in range(B):
        for t in range(int(counts[b])):
            at = int(lengths[b] - counts[b]) + t
            p, slot = int(table[b, at // page]), at % page
            ke[p, :, slot], ks[p, :, slot], ve[p, :, slot] = kw[b, :, t], ksize[b, :, t], v[b, :, t].double()
    if mode == "plain":
        assert torch.equal(there.cpu().double(), expect)
        return
    kg, vg = view(there.cpu())
    assert torch.equal(vg.double(), ve)
    untouched = ks.sum(-1) == 0
    assert torch.equal(kg[untouched].double(), ke[untouched])
    check(kg, ke, ks, "keys")
    if not Hq:
        assert out is None
        return
    qw, qsize = want(q, wq)
    mask = (torch.arange(L)[None] < counts[:, None])[:, None, :, None]
    check(out, torch.where(mask, qw, 0), torch.where(mask, qsize, 0), "queries")
    assert (out.cpu()[~mask.expand_as(qw)] == 0).all()


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("weights", [False, True])
def test_append_without_rotation(d, weights):
    """Queries beside keys with nothing to compute are copied (zeros behind counts); with weights alone both are normalised."""
    B, Hq, Hkv, L, page = 3, 6, 2, 20, 8
    counts = torch.tensor([20, 0, 7], dtype=torch.int32)
    lengths = counts + 3
    store, view = cache("heads", 12, Hkv, page, d, torch.float16, 71)
    table = tables(lengths.tolist(), page, 12, 72)
    q, k, v = (draw((B, L, H, d), torch.float16, 73 + H).transpose(1, 2) for H in (Hq, Hkv, Hkv))
    wq, wk = (draw((d,), torch.float16, 74 + n).cuda() if weights else None for n in (0, 1))
    there = store.cuda()
    out = gb.attn_cache_append(k.cuda(), v.cuda(), *view(there), table.cuda(), lengths.cuda(), counts=counts.cuda(), q=q.cuda(), q_weight=wq, k_weight=wk)
    kg, vg = view(there.cpu())

    def normed(x, w):
        y = x.double()
        return y if w is None else y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.cpu().double()

    qn, kn = normed(q, wq), normed(k, wk)
    for b, c in enumerate(counts.tolist()):
        check(out[b, :, :c], qn[b, :, :c], qn[b, :, :c].abs() * weights, "queries")
        assert (out[b, :, c:] == 0).all()
        for t in range(c):
            at = int(table[b, (3 + t) // page]), slice(None), (3 + t) % page
            check(kg[at], kn[b, :, t], kn[b, :, t].abs() * weights, "keys")
            assert torch.equal(vg[at], v[b, :, t])


def test_append_leaves_bad_sequences_out():
    """A length beyond the table, a count above L or above the length, a negative count: the sequence is left out; a page outside the
    cache: the token is.  All others are written, and the status word says what was found first."""
    B, H, L, d, page, P = 6, 2, 4, 64, 8, 12
    store, view = cache("heads", P, H, page, d, torch.float16, 9, fill=0.0)
    table = torch.arange(12, dtype=torch.int32).reshape(6, 2)
    table[5] = torch.tensor([P, -1])
    lengths = torch.tensor([4, 17, 16, 2, 9, 4], dtype=torch.int32)
    counts = torch.tensor([4, 4, 5, 3, -1, 4], dtype=torch.int32)
    k, q = draw((B, H, L, d), torch.float16, 10), draw((B, H, L, d), torch.float16, 11)
    there = store.cuda()
    inv_freq, _ = gb.attn_rope_frequencies(d)
    out = gb.attn_cache_append(k.cuda(), k.cuda(), *view(there), table.cuda(), lengths.cuda(), counts=counts.cuda(), q=q.cuda(), inv_freq=inv_freq)
    assert gb.attn_last_device_error() in (8, 9)
    kg, vg = view(there.cpu())
    assert torch.equal(vg[0, :, :4], k[0]) and (vg[0, :, 4:] == 0).all() and (vg[1:] == 0).all() and (kg[1:] == 0).all()
    assert (out[1:5] == 0).all() and (out[0] != 0).any() and (out[5] != 0).any()
    gb.attn_cache_append(k.cuda(), k.cuda(), *view(there), table.cuda(), torch.full((B,), 4, dtype=torch.int32).cuda())
    assert gb.attn_last_device_error() == 8


# ------------------------------------------------------------------------------------------------- copy
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("H,page,d,P,n", [(1, 8, 64, 20, 1), (8, 16, 128, 150, 60), (5, 24, 256, 40, 19), (2, 16, 64, 9000, 4300), (1, 8, 512, 3, 0)])
def test_copy(layout, H, page, d, P, n):
    store, view = cache(layout, P, H, page, d, torch.bfloat16, 12)
    deal = torch.randperm(P, generator=torch.Generator().manual_seed(13), dtype=torch.int32)
    src, dst = deal[:n].contiguous(), deal[n:2 * n].contiguous()
    there = store.cuda()
    gb.attn_cache_copy(*view(there), src, dst)
    for pages in view(store):
        pages[dst.long()] = pages[src.long()]
    assert torch.equal(there.cpu(), store)


def test_copy_one_after_the_other():
    """Chains, cycles, repeated destinations and a page onto itself: as if the pages were copied one by one."""
    P = 40
    store, view = cache("heads", P, 2, 8, 64, torch.float16, 14)
    g = torch.Generator().manual_seed(15)
    lists = [([5, 7], [3, 5]), ([3, 5], [5, 7]), ([1, 2], [2, 1]), ([4, 6], [9, 9]), ([8], [8]), ([0, 10, 0], [10, 11, 12]),
             (torch.randint(0, P, (500,), generator=g).tolist(), torch.randint(0, P, (500,), generator=g).tolist())]
    there = store.cuda()
    for src, dst in lists:
        gb.attn_cache_copy(*view(there), src, dst)
        for a, b in zip(src, dst):
            for pages in view(store):
                pages[b] = pages[a].clone()
        assert torch.equal(there.cpu(), store), (src, dst)


def test_copy_refusals_touch_nothing():
    store, view = cache("heads", 6, 1, 8, 64, torch.float16, 16)
    there = store.cuda()
    for src, dst in (([0, 6], [1, 2]), ([0, 1], [2, -1]), ([0, 2 ** 31 - 1], [1, 2])):
        with pytest.raises(gb.GbattnError):
            gb.attn_cache_copy(*view(there), src, dst)
    for src, dst in (([0], [1, 2]), (torch.tensor([0]), torch.tensor([1])), (torch.tensor([0], dtype=torch.int32).cuda(), [1])):
        with pytest.raises(ValueError):
            gb.attn_cache_copy(*view(there), src, dst)
    with pytest.raises(TypeError):
        gb.attn_cache_copy(*view(there), [0.5], [1])
    with pytest.raises(gb.GbattnError):
        gb.attn_cache_copy(view(there)[0], view(there)[0], [0], [1])
    assert torch.equal(there.cpu(), store)


# ------------------------------------------------------------------------------------------------- decode
def decode_reference(q, kp, vp, table, lengths, scale):
    """o, lse, sum p |v| and the largest logit's sum of magnitudes, in 64 bits."""
    B, Hq, d = q.shape
    H, page = kp.shape[1], kp.shape[2]
    o, lse = torch.zeros(B, Hq, d, dtype=torch.float64), torch.full((B, Hq), -math.inf, dtype=torch.float64)
    size, big = torch.zeros_like(o), torch.zeros_like(lse)
    for b, n in enumerate(lengths.tolist()):
        if n == 0:
            continue
        at = table[b, :-(-n // page)].long()
        k, v = (x[at].transpose(0, 1).reshape(H, -1, d)[:, :n].double().repeat_interleave(Hq // H, 0) for x in (kp, vp))
        s = torch.einsum("hd,hnd->hn", q[b].double(), k) * scale
        p = torch.softmax(s, -1)
        o[b], lse[b] = torch.einsum("hn,hnd->hd", p, v), torch.logsumexp(s, -1)
        size[b] = torch.einsum("hn,hnd->hd", p, v.abs())
        big[b] = torch.einsum("hd,hnd->hn", q[b].double().abs(), k.abs()).amax(-1) * scale
    return o, lse, size, big


def check_decode(got, ref, what=""):
    (o, lse), (ow, lw, size, big) = [t.cpu() for t in got], ref
    d = o.shape[-1]
    off = (d + 8) * U * big
    tol = half_step(o.dtype, ow) + (2 * off[..., None] + 2.0 ** -20 + 2.0 ** -17) * size
    err = (o.double() - ow).abs()
    assert (err <= tol).all(), f"{what}: o {(err / tol).max():.2f} times the tolerance"
    empty = torch.isinf(lw)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all(), what
    err, tol = (lse.double() - lw).abs()[~empty], (off + 2.0 ** -20 * (1 + lw.abs()))[~empty]
    assert (err <= tol).all(), f"{what}: lse {(err / tol).max():.2f} times the tolerance"


DECODE = [  # lengths, Hq, Hkv, d, page, layout
    ([1], 1, 1, 64, 8, "heads"), ([0], 2, 1, 128, 16, "heads"), ([127, 128, 129], 4, 4, 128, 16, "slots"),
    ([0, 5, 1000, 0, 77, 256], 8, 2, 128, 16, "joint"), ([300], 7, 1, 64, 24, "side"), ([1, 513, 200], 16, 1, 256, 32, "heads_joint"),
    ([700, 3], 4, 2, 512, 8, "heads"), ([5000], 32, 2, 64, 64, "slots"), ([0, 0, 0], 4, 4, 128, 8, "heads"), ([2000, 1], 40, 1, 128, 40, "heads"),
    ([90, 91], 66, 2, 64, 16, "heads"), ([1200], 71, 1, 256, 128, "slots"), ([260, 7], 48, 1, 512, 16, "heads"), ([30000], 8, 8, 128, 256, "heads"),
    ([20000, 0, 1], 5, 5, 256, 136, "joint"), ([9000], 3, 3, 512, 16, "slots"), ([1 + i % 140 for i in range(400)], 4, 2, 64, 16, "heads"),
    ([64] * 1500, 1, 1, 64, 64, "heads")]


@pytest.mark.parametrize("lengths,Hq,Hkv,d,page,layout", DECODE, ids=[f"{len(c[0])}x{max(c[0])}-{c[1]}-{c[2]}-{c[3]}-{c[4]}" for c in DECODE])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_decode(lengths, Hq, Hkv, d, page, layout, dtype):
    P = sum(-(-n // page) for n in lengths) + 1
    store, view = cache(layout, P, Hkv, page, d, dtype, 21)
    table, n = tables(lengths, page, P, 22, extra=2), torch.tensor(lengths, dtype=torch.int32)
    q = draw((len(lengths), Hq, d), dtype, 23, scale=2.0)
    there = view(store.cuda())
    got = gb.attn_decode_paged(q.cuda(), *there, table.cuda(), n.cuda())
    again = gb.attn_decode_paged(q.cuda()[:, :, None], *there, table.cuda(), n.cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "not the same bits twice"
    check_decode(got, decode_reference(q, *view(store), table, n, 1.0 / math.sqrt(d)))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d,Hq", [(64, 1), (128, 8), (256, 3), (512, 2)])
def test_decode_ignores_what_lies_behind_the_last_token(value, d, Hq):
    """Every slot of the cache that no token of a sequence is in holds NaN or infinities."""
    lengths, page, H = [1, 130, 0, 255, 40], 16, 1
    P = 60
    store, view = cache("heads", P, H, page, d, torch.float16, 24, fill=value)
    kp, vp = view(store)
    table, n = tables(lengths, page, P, 25), torch.tensor(lengths, dtype=torch.int32)
    real = draw((2, P, H, page, d), torch.float16, 26)
    for b, m in enumerate(lengths):
        for j in range(m):
            at = (int(table[b, j // page]), slice(None), j % page)
            kp[at], vp[at] = real[0][at], real[1][at]
    q = draw((len(lengths), Hq, d), torch.float16, 27)
    ref = decode_reference(q, kp, vp, table, n, 0.125)
    check_decode(gb.attn_decode_paged(q.cuda(), *view(store.cuda()), table.cuda(), n.cuda(), scale=0.125), ref)


@pytest.mark.parametrize("d,G,page", [(64, 1, 8), (64, 12, 24), (64, 20, 16), (128, 2, 24), (128, 12, 8), (128, 20, 136), (256, 1, 8), (256, 20, 24),
                                      (512, 3, 24), (512, 16, 8)])
def test_decode_last_tiles_of_every_kind(d, G, page):
    """Sequences that end anywhere in a group of 16 keys, a page and a tile, with NaN in every slot behind their last token."""
    lengths, H = [*range(1, 19), 31, 32, 33, 95, 96, 97, 112, 113, *range(126, 131), 143, 144, 145, 255, 256, 257, 0, 400], 2
    P = sum(-(-m // page) for m in lengths)
    store, view = cache("slots", P, H, page, d, torch.bfloat16, 81)
    kp, vp = view(store)
    table, n = tables(lengths, page, P, 82), torch.tensor(lengths, dtype=torch.int32)
    for b, m in enumerate(lengths):
        if m % page:
            for x in (kp, vp):
                x[int(table[b, m // page]), :, m % page:] = math.nan
    q = draw((len(lengths), G * H, d), torch.bfloat16, 83)
    ref = decode_reference(q, kp, vp, table, n, 1.0 / math.sqrt(d))
    check_decode(gb.attn_decode_paged(q.cuda(), *view(store.cuda()), table.cuda(), n.cuda()), ref)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_decode_peaks_and_tails(dtype):
    """A rising row of logits (the maximum moves in every tile), a single key far above a long flat tail that still counts, and
    equal logits: the running maximum, the rescaling and the weights' 16-bit parts have to keep all of it."""
    L, d, page = 6000, 64, 16
    P = L // page
    kp = torch.zeros(P, 3, page, d, dtype=dtype)
    vp = draw((P, 3, page, d), dtype, 28) + 1
    ramp = torch.arange(L, dtype=torch.float64).reshape(P, page)
    kp[:, 0, :, 0] = (ramp * (60.0 / L)).to(dtype)
    kp[5, 1, 3, 0] = 13.0
    vp[5, 1, 3] = 0
    q = torch.zeros(1, 3, d, dtype=dtype)
    q[..., 0] = 1
    table, n = torch.arange(P, dtype=torch.int32)[None], torch.tensor([L], dtype=torch.int32)
    check_decode(gb.attn_decode_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), n.cuda(), scale=1.0), decode_reference(q, kp, vp, table, n, 1.0))


def test_decode_of_repeated_inputs():
    """One query row for all heads and sequences, one table row and one page for all: strides of 0."""
    H, d, page, B = 2, 128, 16, 3
    store, view = cache("heads", 2, H, page, d, torch.bfloat16, 75)
    kp, vp = view(store)
    q = draw((1, 1, d), torch.bfloat16, 76).expand(B, 4, d)
    table, n = torch.tensor([[1, 0]], dtype=torch.int32).expand(B, 2), torch.tensor([30, 5, 17], dtype=torch.int32)
    wide = q[:1, :1].cuda().expand(B, 4, d)
    assert wide.stride()[:2] == (0, 0)
    got = gb.attn_decode_paged(wide, kp.cuda(), vp.cuda(), table[:1].cuda().expand(B, 2), n.cuda())
    check_decode(got, decode_reference(q, kp, vp, table, n, 1.0 / math.sqrt(d)))


def test_decode_bad_pages_and_lengths():
    """A page outside the cache counts as zeros, a negative length as none, one beyond the table as its end; the status word tells,
    other sequences are not affected."""
    H, d, page, P = 2, 128, 16, 8
    store, view = cache("heads", P, H, page, d, torch.float16, 29)
    kp, vp = view(store)
    q = draw((4, 4, d), torch.float16, 30)
    table = torch.tensor([[0, 1], [2, 3], [4, 99], [6, -7]], dtype=torch.int32)
    n = torch.tensor([33, -1, 32, 20], dtype=torch.int32)
    got = gb.attn_decode_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), n.cuda(), scale=0.1)
    assert gb.attn_last_device_error() in (8, 9)
    kz, vz = (torch.cat([x, torch.zeros_like(x[:1])]) for x in (kp, vp))
    ref = decode_reference(q, kz, vz, torch.tensor([[0, 1], [2, 3], [4, P], [6, P]]), torch.tensor([32, 0, 32, 20]), 0.1)
    check_decode(got, ref)
    check_decode(gb.attn_decode_paged(q[:1].cuda(), kp.cuda(), vp.cuda(), table[:1].cuda(), torch.tensor([32], dtype=torch.int32).cuda(), scale=0.1),
                 [x[:1] for x in ref])


@pytest.mark.parametrize("d,page,Hkv,G", [(512, 16, 2, 1), (512, 128, 1, 8), (256, 8, 1, 20), (64, 8, 3, 2), (128, 24, 2, 16)])
def test_decode_many_times(d, page, Hkv, G):
    """The kernel's warps meet in many orders: a few thousand calls give the same bits, and no wait runs out."""
    lengths = [1000, 3, 0, 517, 128, 2000]
    P = sum(-(-m // page) for m in lengths)
    store, view = cache("heads", P, Hkv, page, d, torch.bfloat16, 77)
    there, table, n = view(store.cuda()), tables(lengths, page, P, 78).cuda(), torch.tensor(lengths, dtype=torch.int32).cuda()
    q = draw((len(lengths), Hkv * G, d), torch.bfloat16, 79).cuda()
    o, lse = gb.attn_decode_paged(q, *there, table, n)
    differ = torch.zeros((), dtype=torch.int32, device="cuda")
    for _ in range(3000):
        a, b = gb.attn_decode_paged(q, *there, table, n)
        differ += (a != o).any() | (b != lse).any()
    assert int(differ) == 0


def test_decode_agrees_with_the_contiguous_cache():
    """attn_decode's cache, one page to a sequence."""
    B, H, L, d = 2, 4, 1024, 128
    q, k, v = draw((B, H, d), torch.float16, 31).cuda(), draw((B, H, L, d), torch.float16, 32).cuda(), draw((B, H, L, d), torch.float16, 33).cuda()
    o, lse = gb.attn_decode(q, k, v)
    table, n = torch.arange(B, dtype=torch.int32)[:, None].cuda(), torch.full((B,), L, dtype=torch.int32).cuda()
    op, lp = gb.attn_decode_paged(q, k, v, table, n)
    assert (o.float() - op.float()).abs().max() <= 2e-3 and (lse - lp).abs().max() <= 1e-4


def test_decode_streams_graphs_and_two_at_once():
    """Captured calls read lengths, tables and queries anew at each replay; two calls on two streams do not disturb one another."""
    H, d, page, P, B = 4, 128, 16, 400, 3
    store, view = cache("heads", P, H, page, d, torch.bfloat16, 34)
    there = view(store.cuda())
    sets = []
    for seed, lengths in ((35, [900, 10, 2000]), (36, [1, 1500, 0])):
        sets.append((draw((B, 8, d), torch.bfloat16, seed).cuda(), tables([2048, 2048, 2048], page, P, seed).cuda(), torch.tensor(lengths, dtype=torch.int32).cuda()))
    want = [gb.attn_decode_paged(a, *there, t, n) for a, t, n in sets]
    q, table, n = (t.clone() for t in sets[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = gb.attn_decode_paged(q, *there, table, n)
    for i in (1, 0, 1):
        for a, b in zip((q, table, n), sets[i]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[gb.attn_decode_paged(sets[i][0], *there, *sets[i][1:], stream=streams[i]) for i in range(2)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for r in got for i in range(2) for x, y in zip(r[i], want[i]))


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 elements: pages at its end are written, copied and read where they are."""
    H, d, page = 8, 128, 128
    P = (1 << 32) // (H * d * page) + 40
    kp = torch.zeros(P, H, page, d, dtype=torch.float16, device="cuda")
    vp = torch.zeros_like(kp)
    L = 300
    k, v = draw((1, H, L, d), torch.float16, 37), draw((1, H, L, d), torch.float16, 38)
    table = torch.tensor([[P - 1, P - 7, P - 3]], dtype=torch.int32)
    n = torch.tensor([L], dtype=torch.int32).cuda()
    gb.attn_cache_append(k.cuda(), v.cuda(), kp, vp, table.cuda(), n)
    moved = torch.tensor([[P - 30, P - 31, P - 32]], dtype=torch.int32)
    gb.attn_cache_copy(kp, vp, table[0], moved[0])
    q = draw((1, 16, d), torch.float16, 39)
    got = gb.attn_decode_paged(q.cuda(), kp, vp, moved.cuda(), n)
    small = [torch.zeros(3, H, page, d, dtype=torch.float16) for _ in range(2)]
    for x, y in zip(small, (k, v)):
        flat = torch.zeros(H, 3 * page, d, dtype=torch.float16)
        flat[:, :L] = y[0]
        x.copy_(flat.reshape(H, 3, page, d).transpose(0, 1))
    check_decode(got, decode_reference(q, *small, torch.tensor([[0, 1, 2]]), torch.tensor([L]), 1.0 / math.sqrt(d)))
    del kp, vp
    torch.cuda.empty_cache()


def test_decode_refusals():
    H, d, page, P = 2, 64, 8, 4
    store, view = cache("heads", P, H, page, d, torch.float16, 41)
    kp, vp = view(store.cuda())
    good = dict(q=draw((2, 4, d), torch.float16, 42).cuda(), k_pages=kp, v_pages=vp, table=torch.zeros(2, 2, dtype=torch.int32).cuda(),
                lengths=torch.ones(2, dtype=torch.int32).cuda())
    for bad in (dict(q=good["q"].bfloat16()), dict(q=good["q"][..., :32]), dict(q=good["q"].cpu()), dict(k_pages=kp[:, :, :4]), dict(v_pages=vp.transpose(1, 2)),
                dict(table=good["table"].long()), dict(table=good["table"][:1]), dict(table=good["table"].cpu()), dict(lengths=good["lengths"].long()),
                dict(lengths=good["lengths"][:1]), dict(o=torch.empty(2, 4, d, device="cuda")), dict(lse=torch.empty(2, 5, device="cuda")),
                dict(workspace=torch.empty(0, device="cuda")), dict(q=good["q"].float(), k_pages=kp.float(), v_pages=vp.float())):
        with pytest.raises(ValueError):
            gb.attn_decode_paged(**{**good, **bad})
    for bad in (dict(q=torch.zeros(2, 3, d, dtype=torch.float16, device="cuda")), dict(scale=0.0), dict(scale=math.nan), dict(v_pages=kp), dict(o=good["q"]),
                dict(k_pages=kp.reshape(1, 2, 32, d)[:, :, :20], v_pages=vp.reshape(1, 2, 32, d)[:, :, :20])):
        with pytest.raises(gb.GbattnError):
            gb.attn_decode_paged(**{**good, **bad})


def test_append_refusals():
    H, d, page, P, B = 2, 64, 8, 4, 2
    store, view = cache("heads", P, H, page, d, torch.float16, 43)
    kp, vp = view(store.cuda())
    k = draw((B, H, 3, d), torch.float16, 44).cuda()
    good = dict(k=k, v=k.clone(), k_pages=kp, v_pages=vp, table=torch.zeros(2, 1, dtype=torch.int32).cuda(), lengths=torch.full((2,), 3, dtype=torch.int32).cuda())
    w = torch.ones(d, dtype=torch.float16, device="cuda")
    for bad in (dict(k=k[:, :1]), dict(v=k[:1]), dict(v=k.bfloat16()), dict(q=k[:, :, :2]), dict(counts=torch.ones(2).cuda()), dict(lengths=good["lengths"].cpu()),
                dict(q_weight=w), dict(q=k, k_weight=w), dict(inv_freq=torch.ones(16).cuda()), dict(table=good["table"][0])):
        with pytest.raises(ValueError):
            gb.attn_cache_append(**{**good, **bad})
    for bad in (dict(v_pages=kp), dict(k=kp[:2, :, :3]), dict(q=k.clone(), q_out=k), dict(inv_freq=torch.ones(33, dtype=torch.float64, device="cuda")), dict(factor=-1.0)):
        with pytest.raises(gb.GbattnError):
            gb.attn_cache_append(**{**good, **bad})
    assert torch.equal(kp.cpu(), view(store)[0])


# ------------------------------------------------------------------------------------------------- together
def test_a_run_of_them_together():
    """Prompts of a ragged batch, a fork, steps of single tokens, a sequence given up, a compaction, more steps: at every step the
    decoded rows against attention over each sequence's own tokens, kept apart on the CPU."""
    H, G, d, page, P = 2, 3, 64, 8, 40
    inv_freq, _ = gb.attn_rope_frequencies(d)
    f = inv_freq.cpu()
    pages = gb.CachePages(P, page)
    store, view = cache("heads", P, H, page, d, torch.float16, 51, fill=math.nan)
    kp, vp = view(store.cuda())
    seqs, lengths, kept = [], [], []  # kept: float64 keys (turned) and values of each sequence
    seed = [100]

    def step(counts):
        B, L = len(seqs), max(counts)
        seed[0] += 1
        q, k, v = draw((B, L, (G + 2) * H, d), torch.float16, seed[0]).transpose(1, 2).split([G * H, H, H], dim=1)
        for b, c in enumerate(counts):
            gb.attn_cache_copy(kp, vp, *pages.grow(seqs[b], lengths[b], lengths[b] + c))
            lengths[b] += c
        table, n = pages.table(seqs).cuda(), torch.tensor(lengths, dtype=torch.int32).cuda()
        qr = gb.attn_cache_append(k.cuda(), v.cuda(), kp, vp, table, n, counts=torch.tensor(counts, dtype=torch.int32).cuda(), q=q.cuda(), inv_freq=inv_freq)
        pos = torch.tensor([[m - c + t for t in range(L)] for m, c in zip(lengths, counts)])
        kw, qw = (turned(x.double(), pos, f, 1.0, False)[0] for x in (k, q))
        for b, c in enumerate(counts):
            kept[b] = [torch.cat([a, x[b, :, :c].double()], 1) for a, x in zip(kept[b], (kw, v))]
        last = torch.tensor([c - 1 for c in counts])
        rows = qr[torch.arange(B), :, last.cuda()]
        o, lse = gb.attn_decode_paged(rows, kp, vp, table, n)
        for b in range(B):
            ke, ve = (x.repeat_interleave(G, 0) for x in kept[b])
            s = torch.einsum("hd,hnd->hn", qw[b, :, last[b]], ke) / math.sqrt(d)
            want = torch.einsum("hn,hnd->hd", torch.softmax(s, -1), ve)
            # keys and queries are rounded to fp16: a logit moves by at most 2 x 2^-11 x sum |q k| scale (below 12 here)
            off = 2 * 2.0 ** -11 * 12
            assert (o[b].cpu().double() - want).abs().max() <= 2.0 ** -11 * want.abs().max() + 2 * off * ve.abs().max()
            assert (lse[b].cpu().double() - torch.logsumexp(s, -1)).abs().max() <= off

    def add(length=0):
        seqs.append(pages.new(length))
        lengths.append(0)
        kept.append([torch.zeros(H, 0, d, dtype=torch.float64) for _ in range(2)])

    for _ in range(3):
        add()
    step([20, 3, 33])
    mine, src, dst = pages.fork(seqs[0], 20)
    assert len(src) == len(dst) == 1
    gb.attn_cache_copy(kp, vp, src, dst)
    seqs.append(mine), lengths.append(20), kept.append([x.clone() for x in kept[0]])
    step([1, 1, 1, 1])
    step([1, 1, 1, 1])
    pages.free(seqs[1])
    del seqs[1], lengths[1], kept[1]
    src, dst = pages.compact(seqs)
    gb.attn_cache_copy(kp, vp, src, dst)
    assert max(max(s) for s in seqs) < P - pages.free_pages
    step([1, 1, 1])
    step([9, 1, 2])


def test_a_captured_step_of_both_serves_growing_sequences():
    """One graph of append and decode, replayed while lengths grow across a page's end."""
    H, G, d, page, P, B = 2, 2, 64, 8, 16, 2
    store, view = cache("heads", P, H, page, d, torch.float16, 61, fill=0.0)
    kp, vp = view(store.cuda())
    inv_freq, _ = gb.attn_rope_frequencies(d)
    table = torch.arange(P, dtype=torch.int32).reshape(B, P // B).cuda()
    n = torch.tensor([6, 0], dtype=torch.int32).cuda()
    rows = draw((12, B, 1, (G + 2) * H, d), torch.float16, 62).cuda()
    now = rows[0].clone()
    q, k, v = now.transpose(1, 2).split([G * H, H, H], dim=1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n.add_(1)
        qr = gb.attn_cache_append(k, v, kp, vp, table, n, q=q, inv_freq=inv_freq)
        o, lse = gb.attn_decode_paged(qr, kp, vp, table, n)
    got = []
    for r in rows:
        now.copy_(r)
        graph.replay()
        got.append((o.clone(), lse.clone()))
    torch.cuda.synchronize()
    kp2, vp2 = (torch.zeros_like(x) for x in (kp, vp))
    n2 = torch.tensor([6, 0], dtype=torch.int32).cuda()
    for r, (a, b) in zip(rows, got):
        q, k, v = r.transpose(1, 2).split([G * H, H, H], dim=1)
        n2 += 1
        qr = gb.attn_cache_append(k, v, kp2, vp2, table, n2, q=q, inv_freq=inv_freq)
        o2, lse2 = gb.attn_decode_paged(qr, kp2, vp2, table, n2)
        assert torch.equal(a, o2) and torch.equal(b, lse2)
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2)
