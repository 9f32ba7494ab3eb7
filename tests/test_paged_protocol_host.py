"""Host models of the paged decode kernel's bookkeeping (csrc/paged_decode.cu), which need no GPU: the shares of the CTAs cover
every tile once and name the partial results that belong together, and the ring's protocol never stalls and never lets a slot be
refilled or a buffer rewritten too early."""
import random

import pytest

TILE = 128


def shares(lengths, hvs, G):
    """Per CTA its segments (row, first tile, tiles, tiles of the row), as the kernel walks them, and its record."""
    tiles = [-(-n // TILE) for n in lengths]
    total = sum(tiles) * hvs
    out = []
    grid, G = G, min(G, max(total, 1))
    for c in range(grid):
        u0, u1 = total * min(c, G) // G, total * min(c + 1, G) // G
        segs, record = [], None
        if u0 < u1:
            off, b = u0, 0
            while off >= tiles[b] * hvs:
                off -= tiles[b] * hvs
                b += 1
            hv, tile, left = off // tiles[b], off % tiles[b], u1 - u0
            while left > 0:
                n = min(left, tiles[b] - tile)
                segs.append(((b, hv), tile, n, tiles[b]))
                left -= n
                tile += n
                if tile == tiles[b]:
                    tile, hv = 0, hv + 1
                    if hv == hvs:
                        hv, b = 0, b + 1
                        while left > 0 and b < len(tiles) and tiles[b] == 0:
                            b += 1
            row, first, n, whole = segs[-1]
            if first == 0 and n < whole:
                end = u1 + (whole - n) - 1
                record = ((end + 1) * G - 1) // total - c + 1
        out.append((segs, record))
    return out


@pytest.mark.parametrize("seed", range(60))
def test_shares(seed):
    rng = random.Random(seed)
    B, hvs, G = rng.choice([1, 2, 7, 200]), rng.choice([1, 2, 8, 30]), rng.choice([1, 2, 13, 152])
    lengths = [rng.choice([0, 1, 128, 129, rng.randint(0, 3000), rng.randint(0, 50000)]) for _ in range(B)]
    got = shares(lengths, hvs, G)
    seen = {}
    for c, (segs, record) in enumerate(got):
        for k, (row, first, n, whole) in enumerate(segs):
            assert n > 0 and first + n <= whole
            assert first == 0 or k == 0, "a later part of a row opens its CTA's share"
            assert first + n == whole or k == len(segs) - 1, "a row that goes on ends it"
            for t in range(first, first + n):
                assert seen.setdefault((row, t), c) == c
        parts = record or 0
        if parts:  # this CTA's last segment and the first ones of the next parts - 1 CTAs make the row
            row, first, n, whole = segs[-1]
            at = n
            for d in range(c + 1, c + parts):
                r, f, m, w = got[d][0][0]
                assert r == row and f == at
                at += m
            assert at == whole
        elif segs:
            assert segs[-1][1] != 0 or segs[-1][2] == segs[-1][3]
    assert len(seen) == sum(-(-n // TILE) for n in lengths) * hvs


def v_pos(t, T, nc):
    return (min(t + 2, T) + t) * nc


@pytest.mark.parametrize("nc,nslot,nqb", [(1, 12, 2), (1, 11, 2), (1, 6, 2), (1, 5, 2), (2, 6, 2), (2, 5, 2), (2, 5, 1), (2, 4, 1), (2, 4, 2), (4, 6, 2), (4, 5, 2)])
@pytest.mark.parametrize("seed", range(40))
def test_ring_protocol(nc, nslot, nqb, seed):
    """The three roles step by step in a random interleaving, each blocked exactly where the kernel waits.  Loads, products and
    arrivals complete at once or later, at random."""
    rng = random.Random(seed)
    segs = [rng.randint(1, 5) for _ in range(rng.randint(1, 9))]
    T = sum(segs)
    first = [i == 0 for n in segs for i in range(n)]
    last = [i == n - 1 for n in segs for i in range(n)]
    seg = [s for s, n in enumerate(segs) for _ in range(n)]
    tail = [l or rng.random() < 0.2 for l in last]
    done = {}  # barrier -> completed phases

    def ready(bar, phase):
        """A parity wait for `phase`: it must be the last phase that completed, or the one that is next."""
        n = done.get(bar, 0)
        assert phase <= n <= phase + 1, (bar, phase, n)
        return n > phase

    def arrive(bar):
        done[bar] = done.get(bar, 0) + 1

    slots, s_buf, p_buf, q_buf = [None] * nslot, [None] * 2, [None] * 2, [None] * nqb
    order, read, o_buf = [], set(), [None] * 2

    def producer():
        at = 0
        for t in range(T + 1):
            for what, u in (("K", t), ("V", t - 1)):
                if not 0 <= u < T:
                    continue
                if what == "K" and first[u]:
                    s = seg[u]
                    while s >= nqb and not ready(("qempty", s % nqb), s // nqb - 1):
                        yield
                    q_buf[s % nqb] = s
                    arrive(("qfull", s % nqb))
                if what == "V":
                    assert at == v_pos(u, T, nc)
                for c in range(nc):
                    while at >= nslot and not ready(("empty", at % nslot), at // nslot - 1):
                        yield
                    assert slots[at % nslot] is None
                    slots[at % nslot] = (what, u, c)
                    arrive(("full", at % nslot))
                    at += 1
                    yield

    def mma():
        at = 0

        def take(what, t, finish):
            nonlocal at
            for c in range(nc):
                while not ready(("full", at % nslot), at // nslot):
                    yield
                assert slots[at % nslot] == (what, t, c)
                slots[at % nslot] = None
                if c == nc - 1:
                    finish()
                arrive(("empty", at % nslot))
                at += 1
                yield

        def qk(t):
            while first[t] and not ready(("qfull", seg[t] % nqb), seg[t] // nqb):
                yield
            assert t < 2 or t - 2 in read, "S is rewritten before it was read"
            assert q_buf[seg[t] % nqb] == seg[t]
            yield from take("K", t, lambda: s_buf.__setitem__(t & 1, t))
            if nc > 1:
                arrive(("sfull", t & 1))
            if last[t]:
                arrive(("qempty", seg[t] % nqb))

        yield from qk(0)
        for t in range(T):
            if t + 1 < T:
                yield from qk(t + 1)
            while not ready(("pfull", t & 1), t >> 1):
                yield
            assert p_buf[t & 1] == t
            assert not first[t] or o_buf[seg[t] & 1] is None, "O is overwritten before its results were taken"
            o_buf[seg[t] & 1] = seg[t]
            yield from take("V", t, lambda: order.append(t))
            if nc > 1:
                arrive(("pdone", t & 1))

    def s_there(t):
        x = 0 if t == 0 else 2 * t - 1
        return ready(("empty", x % nslot), x // nslot) if nc == 1 else ready(("sfull", t & 1), t >> 1)

    def pv_done(t):
        x = v_pos(t, T, 1)
        return ready(("empty", x % nslot), x // nslot) if nc == 1 else ready(("pdone", t & 1), t >> 1)

    def results(t):
        """Of the segment that ends with tile t, taken a tile later."""
        while not pv_done(t):
            yield
        assert order[:t + 1] == list(range(t + 1)) and o_buf[seg[t] & 1] == seg[t]
        o_buf[seg[t] & 1] = None

    def softmax():
        due = None
        for t in range(T):
            while not s_there(t):
                yield
            assert s_buf[t & 1] == t
            yield
            read.add(t)
            while t >= 2 and not pv_done(t - 2):
                yield
            p_buf[t & 1] = t
            if not first[t] and rng.random() < 0.5:  # the maximum moved
                while not pv_done(t - 1):
                    yield
                assert order == list(range(t))
            if tail[t]:
                while nslot < 3 * nc and t >= 1 and not pv_done(t - 1):
                    yield
                while nslot < 3 * nc and t + 1 < T and not s_there(t + 1):
                    yield
                for c in range(nc):
                    x = v_pos(t, T, nc) + c
                    while not ready(("full", x % nslot), x // nslot):
                        yield
                    assert slots[x % nslot] == ("V", t, c)
                    yield
            arrive(("pfull", t & 1))
            if due is not None:
                yield from results(due)
            due = t if last[t] else None
            yield
        yield from results(due)

    roles = [producer(), mma(), softmax()]
    idle = 0
    while roles:
        r = rng.choice(roles)
        before = (dict(done), list(order))
        try:
            next(r)
        except StopIteration:
            roles.remove(r)
            continue
        idle = idle + 1 if before == (dict(done), list(order)) else 0
        assert idle < 5000, "the protocol stalled"
    assert order == list(range(T)) and slots == [None] * nslot
