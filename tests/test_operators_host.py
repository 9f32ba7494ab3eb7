"""Host-side checks of the operators beside the attention kernels that need no GPU: their C entry points refuse bad arguments before any
CUDA call, the page bookkeeping against a plain model, the frequencies of scaled contexts, and the kernels' reduction of angles."""
import ctypes
import math
import os
import random
import re
from fractions import Fraction

import pytest
import torch

import scaled_dot_product_sdpa_gb300 as gb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# Fake device addresses, 4 GiB apart: every call below is refused before anything is read.
A = [(i + 1) << 32 for i in range(24)]


@pytest.fixture(scope="module")
def lib():
    from scaled_dot_product_sdpa_gb300 import build as b
    return gb.load_library(b.build())


def code(name):
    text = open(os.path.join(ROOT, "include", "gbattn.h")).read()
    return int(re.search(r"#define GBATTN_ERR_%s \((-?\d+)\)" % name, text).group(1))


def rows(p, H, L, d):
    return [p, H * L * d, L * d, d]


def rope(lib, q=A[0], k=A[1], qo=A[2], ko=A[3], freq=A[4], rotary=64, factor=1.0, pos=A[5], ps=0, wq=A[6], wk=A[7], eps=1e-6, dtype=0, B=2, Hq=4, Hkv=2,
         L=8, d=64, qs=None):
    return lib.attn_rope(*(qs or rows(q, Hq, L, d)), *rows(k, Hkv, L, d), qo, ko, freq, rotary, 0, factor, pos, ps, wq, wk, eps, dtype, B, Hq, Hkv, L, d, None)


def rope_bwd(lib, dq=A[0], dk=A[1], q=A[2], k=A[3], dqo=A[4], dko=A[5], gq=A[6], gk=A[7], freq=A[8], rotary=64, factor=1.0, wq=A[9], wk=A[10], eps=1e-6,
             ws=A[11], dtype=1, B=2, Hq=4, Hkv=2, L=8, d=64):
    return lib.attn_rope_bwd(*rows(dq, Hq, L, d), *rows(dk, Hkv, L, d), *rows(q, Hq, L, d), *rows(k, Hkv, L, d), dqo, dko, gq, gk, freq, rotary, 0, factor,
                             None, 0, wq, wk, eps, ws, dtype, B, Hq, Hkv, L, d, None)


def append(lib, k=A[0], v=A[1], q=A[2], qo=A[3], kp=A[4], vp=A[5], strides=None, pages=10, page=16, table=A[6], ts=4, tw=4, lengths=A[7], counts=A[8], freq=A[9],
           rotary=64, factor=1.0, wq=A[10], wk=A[11], eps=1e-6, dtype=0, B=2, Hq=4, Hkv=2, L=8, d=64):
    return lib.attn_cache_append(*rows(k, Hkv, L, d), *rows(v, Hkv, L, d), *rows(q, Hq, L, d), qo, kp, vp, *(strides or (Hkv * page * d, page * d, d)), pages,
                                 page, table, ts, tw, lengths, counts, freq, rotary, 0, factor, wq, wk, eps, dtype, B, Hq, Hkv, L, d, None)


def copy(lib, kp=A[0], vp=A[1], strides=None, pages=10, page=16, Hkv=2, d=64, src=(0,), dst=(1,), n=None):
    a, b = (ctypes.c_int * max(1, len(src)))(*src), (ctypes.c_int * max(1, len(dst)))(*dst)
    return lib.attn_cache_copy(kp, vp, *(strides or (Hkv * page * d, page * d, d)), pages, page, Hkv, d, ctypes.addressof(a), ctypes.addressof(b),
                               len(src) if n is None else n, None)


def decode(lib, q=A[0], kp=A[1], vp=A[2], strides=None, pages=10, page=16, table=A[3], ts=4, tw=4, lengths=A[4], o=A[5], lse=A[6], ws=A[7], dtype=0, B=2, Hq=4,
           Hkv=2, d=64, scale=0.125, qs=None):
    return lib.attn_decode_paged(q, *(qs or (Hq * d, d)), kp, vp, *(strides or (Hkv * page * d, page * d, d)), pages, page, table, ts, tw, lengths, o, lse, ws,
                                 dtype, B, Hq, Hkv, d, scale, None)


CALLS = {"rope": rope, "rope_bwd": rope_bwd, "append": append, "copy": copy, "decode": decode}
REFUSED = {
    "NULL": [("rope", dict(q=None)), ("rope", dict(k=None)), ("rope", dict(ko=None)), ("rope_bwd", dict(q=None)), ("rope_bwd", dict(ws=None)),
             ("rope_bwd", dict(gk=None)), ("append", dict(v=None)), ("append", dict(q=None)), ("append", dict(qo=None)), ("append", dict(table=None)),
             ("append", dict(lengths=None)), ("copy", dict(kp=None)), ("decode", dict(ws=None)), ("decode", dict(lse=None)), ("decode", dict(table=None))],
    "DTYPE": [("rope", dict(dtype=2)), ("rope_bwd", dict(dtype=-1)), ("append", dict(dtype=7)), ("decode", dict(dtype=2))],
    "DIMS": [(c, {x: v}) for c in ("rope", "rope_bwd", "append") for x in ("B", "L") for v in (0, -3)] + [("rope", dict(B=1 << 20, L=1 << 20)),
             ("rope", dict(Hq=1 << 30)), ("append", dict(tw=0)), ("append", dict(pages=0)), ("copy", dict(n=-1)), ("decode", dict(B=0)), ("decode", dict(tw=-1)),
             ("decode", dict(Hq=0)), ("decode", dict(B=1 << 16, Hq=1 << 16))],
    "HEAD_DIM": [(c, dict(d=v)) for c in CALLS for v in (0, 32, 96, 1024)],
    "ROTARY": [("rope", dict(rotary=v)) for v in (-16, 8, 40, 80)] + [("rope", dict(freq=None)), ("rope", dict(wq=None)), ("rope", dict(wk=None)),
               ("rope_bwd", dict(rotary=24)), ("append", dict(rotary=128)), ("append", dict(wk=None))],
    "SCALE": [("rope", dict(factor=v)) for v in (0.0, -1.0, math.inf, math.nan)] + [("rope", dict(eps=-1e-6)), ("rope", dict(eps=math.nan)),
              ("rope_bwd", dict(factor=0.0)), ("append", dict(eps=math.inf)), ("decode", dict(scale=0.0)), ("decode", dict(scale=math.nan))],
    "ALIGN": [("rope", {x: A[12] + 8}) for x in ("q", "k", "qo", "ko", "wq", "wk")] + [("rope", dict(freq=A[12] + 4)), ("rope", dict(pos=A[12] + 2)),
              ("rope_bwd", dict(ws=A[12] + 8)), ("rope_bwd", dict(gq=A[12] + 4)), ("append", dict(kp=A[12] + 2)), ("append", dict(table=A[12] + 1)),
              ("copy", dict(vp=A[12] + 8)), ("decode", dict(q=A[12] + 2)), ("decode", dict(lengths=A[12] + 1))],
    "STRIDE": [("rope", dict(qs=[A[0], 2048, 512, 68])), ("rope", dict(qs=[A[0], -2048, 512, 64])), ("rope", dict(ps=-1)), ("append", dict(ts=-1)),
               ("append", dict(strides=(2048, 1024, 60))), ("copy", dict(strides=(2040, 1024, 64))), ("decode", dict(strides=(0, 1024, 64))),
               ("decode", dict(strides=(2048, 1024, 0))), ("decode", dict(strides=(2048, 512, 64))), ("decode", dict(qs=(256, 4))),
               # offsets that would pass 2^40 elements, and 2^63 with them
               ("rope", dict(B=1 << 28, L=1, qs=[A[0], 1 << 38, 64, 64])), ("rope", dict(B=1 << 20, ps=1 << 50)), ("append", dict(B=1 << 20, ts=1 << 60)),
               ("append", dict(page=1 << 30, strides=(1 << 38, 64, 1 << 38))), ("copy", dict(page=1 << 30, Hkv=1 << 30, strides=(1 << 38, 1 << 31, 64))),
               ("copy", dict(pages=1 << 30, strides=(1 << 38, 1024, 64))), ("decode", dict(ts=1 << 62)), ("decode", dict(B=1 << 27, qs=(1 << 38, 64)))],
    "PAGES": [("append", dict(page=v)) for v in (0, -8, 4, 20)] + [("decode", dict(page=12)), ("copy", dict(page=1)), ("copy", dict(src=(0, 10), dst=(1, 2))),
              ("copy", dict(src=(0,), dst=(-1,)))],
    "HEADS": [("decode", dict(Hq=3)), ("decode", dict(Hq=1))],
    "ALIAS": [("rope", dict(qo=A[0])), ("rope", dict(ko=A[0] + 64)), ("rope", dict(ko=A[2])), ("rope", dict(qo=A[4])), ("rope", dict(ko=A[7])),
              ("rope_bwd", dict(dqo=A[0])), ("rope_bwd", dict(ws=A[3])), ("rope_bwd", dict(gq=A[7])), ("rope_bwd", dict(dko=A[9])), ("append", dict(kp=A[0])),
              ("append", dict(vp=A[4])), ("append", dict(vp=A[4] + 128)), ("append", dict(qo=A[5])), ("append", dict(vp=A[6])), ("copy", dict(vp=A[0])),
              ("copy", dict(vp=A[0] + 2048 * 2 * 3)), ("copy", dict(vp=A[0] + 16)), ("decode", dict(o=A[0])), ("decode", dict(ws=A[1] + 4096)),
              ("decode", dict(lse=A[5] + 16)), ("decode", dict(o=A[3])), ("decode", dict(vp=A[1]))],
}


@pytest.mark.parametrize("name,call,bad", [(n, c, b) for n, l in REFUSED.items() for c, b in l], ids=lambda x: x if isinstance(x, str) else "-".join(x))
def test_refusals(lib, name, call, bad):
    assert CALLS[call](lib, **bad) == code(name)


def test_good_calls_pass_every_check(lib):
    """Without a GPU they end at the device; the strides of interleaved caches are no aliases."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    ended = (code("LAUNCH"), code("DEVICE"))
    for c in CALLS.values():
        assert c(lib) in ended
    H, page, d = 2, 16, 64
    block = H * page * d
    for strides, gap in (((2 * block, page * d, d), block), ((2 * block, 2 * page * d, d), page * d), ((2 * block, 2 * page * d, 2 * d), d),
                         ((2 * block, 2 * d, 2 * H * d), d), ((block, d, H * d), 10 * block), ((2 * block, 2 * d, 2 * H * d), 21 * d)):
        for x, y in ((A[0], A[0] + 2 * gap), (A[0] + 2 * gap, A[0])):
            assert copy(lib, kp=x, vp=y, strides=strides) in ended, (strides, gap)
    for strides, gap in (((2 * block, page * d, d), block - 8), ((2 * block, 2 * page * d, d), page * d + 8), ((2 * block, 2 * d, 2 * H * d), 2 * d),
                         ((2 * block, 2 * d, 2 * H * d), 22 * d + 8)):
        assert copy(lib, vp=A[0] + 2 * gap, strides=strides) == code("ALIAS"), (strides, gap)
    assert rope(lib, k=None, ko=None, Hkv=0, wk=None) in ended
    assert rope(lib, rotary=0, freq=None) in ended
    assert append(lib, q=None, qo=None, Hq=0, wq=None) in ended
    assert copy(lib, src=(), dst=()) in ended


def test_workspaces(lib):
    assert lib.attn_rope_bwd_workspace_bytes(96) == code("HEAD_DIM") and lib.attn_rope_bwd_workspace_bytes(128) > 0
    assert lib.attn_decode_paged_workspace_bytes(8, 3, 64) == code("HEADS")
    assert lib.attn_decode_paged_workspace_bytes(8, 0, 64) == code("DIMS")
    assert lib.attn_decode_paged_workspace_bytes(8, 2, 65) == code("HEAD_DIM")
    assert lib.attn_decode_paged_workspace_bytes(8, 2, 64) >= 16


def test_cpu_tensors_are_refused(lib):
    q, f = torch.zeros(1, 2, 3, 64, dtype=torch.float16), torch.ones(32, dtype=torch.float64)
    pages = torch.zeros(4, 2, 8, 64, dtype=torch.float16)
    table, n = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for call in (lambda: gb.attn_rope(q, q, f), lambda: gb.attn_rope_bwd(q, q, f), lambda: gb.attn_cache_append(q, q, pages, pages, table, n),
                 lambda: gb.attn_cache_copy(pages, pages, [0], [1]), lambda: gb.attn_decode_paged(q[:, :, 0], pages, pages, table, n)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


# ------------------------------------------------------------------------------------------------- page bookkeeping
def test_pages_against_a_plain_model():
    """Random forks, growth, releases and compactions; contents are kept beside as (page -> tokens) and moved by the copies that the
    methods return, and must always spell each sequence's own tokens."""
    rng = random.Random(1)
    P, page = 30, 4
    pages = gb.CachePages(P, page)
    memory = [[None] * page for _ in range(P)]
    seqs, texts = [], []
    fresh = iter(range(10 ** 9))

    def copied(src, dst):
        for a, b in zip(src, dst):
            memory[b] = list(memory[a])

    for _ in range(3000):
        act = rng.choice(["new", "grow", "grow", "grow", "fork", "free", "compact"])
        before = ([list(s) for s in seqs], pages.free_pages)
        try:
            if act == "new":
                seqs.append(pages.new(0))
                texts.append([])
            elif act == "grow" and seqs:
                i, n = rng.randrange(len(seqs)), rng.randint(0, 9)
                copied(*pages.grow(seqs[i], len(texts[i]), len(texts[i]) + n))
                for t in range(len(texts[i]), len(texts[i]) + n):
                    assert pages.users(seqs[i][t // page]) == 1
                    texts[i].append(next(fresh))
                    memory[seqs[i][t // page]][t % page] = texts[i][t]
            elif act == "fork" and seqs:
                i = rng.randrange(len(seqs))
                n = rng.randint(0, len(texts[i]))
                mine, src, dst = pages.fork(seqs[i], n)
                copied(src, dst)
                seqs.append(mine)
                texts.append(texts[i][:n])
            elif act == "free" and seqs:
                i = rng.randrange(len(seqs))
                pages.free(seqs[i])
                assert seqs[i] == []
                del seqs[i], texts[i]
            elif act == "compact":
                src, dst = pages.compact(seqs)
                assert not src or min(src) > max(dst)
                copied(src, dst)
                assert max((max(s, default=-1) for s in seqs), default=-1) < P - pages.free_pages
        except gb.CacheFull:
            assert before == ([list(s) for s in seqs], pages.free_pages), "a refused request changed something"
        for s, text in zip(seqs, texts):
            assert [memory[s[t // page]][t % page] for t in range(len(text))] == text
        assert pages.free_pages == P - len({p for s in seqs for p in s})
    t = pages.table(seqs)
    assert t.dtype == torch.int32 and t.shape[0] == len(seqs) and all(t[i, :len(s)].tolist() == s for i, s in enumerate(seqs))


def test_pages_refusals():
    pages = gb.CachePages(4, 8)
    a = pages.new(20)
    with pytest.raises(gb.CacheFull):
        pages.new(9)
    for bad in (lambda: pages.free([3]), lambda: pages.fork(a, 25), lambda: pages.grow(a, 9, 8), lambda: pages.compact([]), lambda: pages.free([7]),
                lambda: pages.new(-1), lambda: pages.free([a[0], a[0]]), lambda: pages.table([a], 2), lambda: gb.CachePages(0, 8)):
        with pytest.raises(ValueError):
            bad()
    assert pages.free_pages == 1 and pages.table([a]).tolist() == [a] and pages.table([]).shape == (0, 1)


# ------------------------------------------------------------------------------------------------- frequencies and angles
def test_frequencies():
    f, one = gb.attn_rope_frequencies(8, base=16.0, device="cpu")
    assert f.dtype == torch.float64 and one == 1.0 and torch.allclose(f, torch.tensor([1.0, 0.5, 0.25, 0.125], dtype=torch.float64), rtol=1e-15)
    g, one = gb.attn_rope_frequencies(8, base=16.0, scaling="linear", scale=4.0, device="cpu")
    assert torch.equal(g, f / 4) and one == 1.0
    g, _ = gb.attn_rope_frequencies(8, base=16.0, scaling="base", scale=4.0, device="cpu")
    assert g[0] == 1.0 and math.isclose(g[3], f[3] / 4, rel_tol=1e-14)
    f, _ = gb.attn_rope_frequencies(128, device="cpu")
    g, factor = gb.attn_rope_frequencies(128, scaling="parts", scale=8.0, trained_length=4096, device="cpu")
    ratio, turns = f / g, 4096 * f / (2 * math.pi)
    # the blend's ends are whole indices: one pair beyond each end already counts as fast or slow
    step = 10000.0 ** (-2 / 128)
    assert torch.equal(g[turns * step >= 32], f[turns * step >= 32]) and torch.allclose(ratio[turns <= step], torch.tensor(8.0, dtype=torch.float64))
    assert (ratio.diff() >= 0).all() and math.isclose(factor, 0.1 * math.log(8.0) + 1.0)
    for bad in (dict(rotary=7), dict(rotary=0), dict(rotary=8, base=1.0), dict(rotary=8, scaling="linear", scale=0.5), dict(rotary=8, scaling="other"),
                dict(rotary=8, scale=2.0), dict(rotary=8, scaling="parts", scale=2.0), dict(rotary=2, scaling="base", scale=2.0)):
        with pytest.raises(ValueError):
            gb.attn_rope_frequencies(device="cpu", **bad)


def test_reduction_of_angles():
    """The kernels' integer arithmetic, restated: m C 2^(e - 2) modulo 2^64 for inv_freq = m 2^e, with C = floor(2^65 / pi), is
    inv_freq / 2 pi turns as a 64-bit fraction; times a position modulo 2^64 it is the angle.  C is below 2^65 / pi by less than 1, and
    m 2^(e - 2) = inv_freq / 4 multiplies that; cutting the product to an integer loses less than 1 more: off by less than 1 + inv_freq / 4."""
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286, 10 ** 75)
    C = 0xA2F9836E4E441529
    assert C == (2 << 64) * pi.denominator // pi.numerator
    rng = random.Random(2)
    for x in [1.0, 0.5, 1e-4 / 32, 2.0 ** -60, 511.9, 2.0 ** -126, 1e-300] + [math.exp(rng.uniform(-25, 6)) for _ in range(200)]:
        m, e = math.frexp(x)
        m, e = int(m * 2 ** 53), e - 53
        P, s = m * C, 2 - e
        fixed = (P >> s) % 2 ** 64 if s > 0 else (P << -s) % 2 ** 64
        exact = Fraction(x) / (2 * pi)
        off = (Fraction(fixed) - exact * 2 ** 64) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        most = 1 + Fraction(x) / 4
        assert off <= most
        for pos in (1, -1, 8191, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
            turn = (pos * fixed) % 2 ** 64
            gap = (Fraction(turn, 2 ** 64) - exact * pos) % 1
            assert min(gap, 1 - gap) <= most * abs(pos) / 2 ** 64
