"""The device status after calls of the tree operators that hold one kind of bad number each, so that no other error hides it."""
import math

import pytest
import torch

import scaled_dot_product_sdpa_gb300 as gb
import test_tree_long_gpu
from test_paged_cache_gpu import cache
from test_tree_gpu import BAD_LENGTH, BAD_PAGE, _lib, call, ints, problem  # noqa: F401 (_lib is a fixture)
from tree_reference import attention, check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("T,Hq", [(9, 4), (70, 4)])
def test_tree_bad_page(d, T, Hq):
    """Sound lengths, and a page outside the cache within one of them: reported, and taken for zeros.  Behind the last token it is not looked at."""
    q, store, view, table, _, _, m, seen = problem(3, Hq, 2, T, d, 16, "heads", torch.float16, "own", 300, full=True)
    lengths, counts = [T + 31, 0, T], [T, 0, T]
    P = store.shape[1]
    table[:] = torch.randint(0, P, table.shape, generator=torch.Generator().manual_seed(9)).int()
    with_zeros = torch.cat([store, torch.zeros_like(store[:, :1])], 1)
    for bad in (-1, P, 2 ** 31 - 1, -2 ** 31):
        for at, status in ((1, BAD_PAGE), ((T + 30) // 16, BAD_PAGE), ((T + 30) // 16 + 1, 0)):
            here, good = table.clone(), table.clone()
            here[0, at], good[0, at] = bad, P
            got = call(q.cuda(), store.cuda(), view, here, lengths, counts, m)
            assert gb.attn_last_device_error() == status
            check_attention(got, attention(q, *view(with_zeros), good, lengths, counts, seen, 1 / math.sqrt(d)), max(lengths), d, "bad page", T * Hq // 2)


def test_keep_bad_lists_and_bad_pages():
    """Bad lengths, counts and lists alone, and pages outside the cache alone, as source and as place."""
    page, Hkv, d = 8, 2, 64
    store, view = cache("heads", 9, Hkv, page, d, torch.float16, 1)
    table = torch.arange(9, dtype=torch.int32).view(3, 3)

    def keep(expect, status, table=table, lengths=(20, 20, 20), counts=(10, 10, 10), kept=((1, 3), (0, 1), (4, 9)), kept_counts=None):
        there = store.cuda()
        gb.attn_cache_keep(*view(there), table.cuda(), ints(lengths), ints(counts), ints(kept), None if kept_counts is None else ints(kept_counts))
        assert gb.attn_last_device_error() == status
        want = store.clone()
        for b, a, z in expect:
            for pages in view(want):
                pages[int(table[b, z // page]), :, z % page] = pages[int(table[b, a // page]), :, a % page]
        assert torch.equal(there.cpu(), want)

    all_moves = ((0, 11, 10), (0, 13, 11), (2, 14, 10), (2, 19, 11))
    keep(all_moves, 0)
    keep(all_moves[2:], BAD_LENGTH, lengths=(25, 20, 20))
    keep(all_moves[2:], BAD_LENGTH, lengths=(-1, 20, 20))
    keep(all_moves[2:], BAD_LENGTH, counts=(21, 10, 10))
    keep(all_moves[2:], BAD_LENGTH, counts=(-1, 10, 10))
    for kept in ((3, 3), (5, 10), (-1, 2), (3, 1), (2 ** 31 - 1, 0)):
        keep(all_moves[2:], BAD_LENGTH, kept=(kept, (0, 1), (4, 9)))
    keep(all_moves[2:], BAD_LENGTH, kept_counts=(3, 2, 2))
    keep(all_moves[2:], BAD_LENGTH, kept_counts=(-1, 2, 2))
    for bad in (-1, 9, 2 ** 31 - 1, -2 ** 31):
        source, place, unused = table.clone(), table.clone(), table.clone()
        source[2, 2] = bad   # tokens 16 .. of sequence 2: kept token 9 (position 19), not 4 (position 14)
        place[0, 1] = bad    # tokens 8 .. 15 of sequence 0: places 10 and 11, and what moves there
        unused[:, 0] = bad   # tokens 0 .. 7
        keep(all_moves[:3], BAD_PAGE, table=source)
        keep(all_moves[2:], BAD_PAGE, table=place)
        keep(all_moves, 0, table=unused)


def test_calls_between_refusals_leave_no_error(monkeypatch):
    """The sound calls of the refusals' test, whose status it reads and drops."""
    real, got = gb.attn_last_device_error, []
    monkeypatch.setattr(gb, "attn_last_device_error", lambda: got.append(real()) or got[-1])
    test_tree_long_gpu.test_refusals_of_tensors()
    assert got == [0]
