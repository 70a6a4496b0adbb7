"""Forks and releases of rows that contradict the page counts: status bit 2, and table, lengths and counts as they were."""
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import Book, Cache
from test_gpu_kv_pages import Ops, both

pytestmark = pytest.mark.gpu


def filled(seqs, cols, held, page=16):
    """Sequences 0..held-1 with (cols - 1) full pages and a begun one each; the others empty."""
    pages = held * cols + 5
    c = Cache([], page, 1, 16, seqs=seqs, spare_pages=pages, poison=False)
    c.table = torch.full((seqs, cols), -1, dtype=torch.int32, device="cuda")
    c.handle = fmad.KvCache(c.k, c.v, c.table, c.lens, c.refs)
    ops = Ops(c, 1024)
    for at in range(0, held, 1024):
        some = list(range(at, min(held, at + 1024)))
        assert ops.reserve(some, [(cols - 1) * page + 3] * len(some))[0] == 0
    return c, ops


def refused(c, call):
    before = [x.clone() for x in (c.table, c.lens, c.refs)]
    assert call() == (2, 0)
    assert all(torch.equal(a, b) for a, b in zip(before, (c.table, c.lens, c.refs)))


# one small CTA; a large one; a cluster; several parts of a row a warp, once and in rounds
SIZES = [(12, 6, 5), (60, 20, 30), (60, 40, 30), (20, 700, 6), (2000, 9, 1000), (80, 1500, 30), (130, 1500, 60)]


@pytest.mark.parametrize("seqs,cols,held", SIZES)
@pytest.mark.parametrize("what", ["none", "behind the pool", "uncounted"])
def test_a_page_that_is_not_one(seqs, cols, held, what):
    """A place below the length names no page, one outside the pool, or one that nobody has counted."""
    require_gpu()
    for row, place in ((0, 0), (held - 1, cols - 1), (held // 2, cols // 2)):
        c, ops = filled(seqs, cols, held)
        page = int(c.table[row, place])
        if what == "uncounted":
            c.refs[page] = 0
        else:
            c.table[row, place] = -1 if what == "none" else c.refs.numel()
        everyone = list(range(held))
        targets = list(range(held, min(seqs, 2 * held)))
        refused(c, lambda: ops.fork(([row] + everyone)[:len(targets)], targets))
        refused(c, lambda: ops.fork([row], [held]))
        refused(c, lambda: ops.release(everyone))
        refused(c, lambda: ops.release([row]))
        # the places that a cut leaves alone are not looked at
        others = [s for s in everyone if s != row]
        keep = [c.lens[0].item()] * held
        assert ops.release(everyone, keep) == (0, 0)
        assert ops.release(others) == (0, 0)
        # mended by hand, the row is as good as any other
        c.table[row, place] = page
        c.refs[page] = 1
        assert ops.fork([row], [held]) == (0, 0)
        assert ops.release([row, held]) == (0, 0)
        assert int(c.refs.abs().sum()) == 0 and bool((c.table == -1).all())


@pytest.mark.parametrize("seqs,cols,held", SIZES)
def test_more_releases_than_a_page_has_users(seqs, cols, held):
    """Two rows name pages that are counted once: the first release frees them, so both in one call are refused."""
    require_gpu()
    c, ops = filled(seqs, cols, held)
    spare = held
    c.table[spare], c.lens[spare] = c.table[1], c.lens[1]
    refused(c, lambda: ops.release(list(range(held)) + [spare]))
    refused(c, lambda: ops.release([spare, 1], [5, 5]))
    assert ops.release([spare, 1], [10 ** 6, (cols - 1) * 16 + 1]) == (0, 0)   # no page becomes free: nothing contradicts
    assert ops.release(list(range(held))) == (0, 0)
    refused(c, lambda: ops.release([spare]))


def test_long_rows_against_the_model():
    """Rows of many places, few and many entries, cuts inside: as the sequential model has them."""
    require_gpu()
    c = Cache([], 16, 1, 16, seqs=50, spare_pages=9000, poison=False)
    c.table = torch.full((50, 1500), -1, dtype=torch.int32, device="cuda")
    c.handle = fmad.KvCache(c.k, c.v, c.table, c.lens, c.refs)
    ops, book = Ops(c, 64), Book(c)
    both(ops, book, "reserve", [0, 7, 9], [1500 * 16, 129 * 16 + 1, 1027 * 16])
    both(ops, book, "fork", [0, 7, 0, 9, 9], [1, 2, 3, 4, 5])
    both(ops, book, "fork", [9] * 30, list(range(20, 50)))
    both(ops, book, "release", [0, 1, 9], [700 * 16, 33, 1026 * 16 + 1])
    both(ops, book, "release", list(range(20, 50)), [16 * j for j in range(30)])
    both(ops, book, "compact")
    both(ops, book, "release", [0, 1, 2, 3, 4, 5, 7, 9] + list(range(20, 50)))
    assert int(c.refs.abs().sum()) == 0
