"""Page bookkeeping of the paged cache against a sequential model: bit for bit, K, V, table, lengths and counts."""
import numpy as np
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import Book, Cache

pytestmark = pytest.mark.gpu


class Ops:
    """The library's calls on a cache, returning the two status words."""

    def __init__(self, cache, n=64):
        self.c = cache
        self.ws = torch.empty(fmad.kv_workspace_size(cache.handle, n), dtype=torch.uint8, device="cuda")
        self.status = torch.full((2,), -9, dtype=torch.int32, device="cuda")

    def _i(self, x):
        return torch.tensor(list(x), dtype=torch.int32, device="cuda")

    def _done(self):
        torch.cuda.synchronize()
        out = tuple(int(x) for x in self.status.cpu())
        self.status.fill_(-9)
        return out

    def reserve(self, seq, count):
        fmad.kv_reserve(self.c.handle, self._i(seq), self._i(count), self.status, self.ws)
        return self._done()

    def fork(self, src, dst):
        fmad.kv_fork(self.c.handle, self._i(src), self._i(dst), self.status)
        return self._done()

    def release(self, seq, keep=None):
        fmad.kv_release(self.c.handle, self._i(seq), self.status, None if keep is None else self._i(keep))
        return self._done()

    def compact(self):
        fmad.kv_compact(self.c.handle, self.status, self.ws)
        return self._done()


def both(ops, book, name, *a):
    got, want = getattr(ops, name)(*a), getattr(book, name)(*a)
    assert got == want, (name, a, got, want)
    book.check(ops.c)
    return got


def empty(page=16, pages=40, seqs=9, cols=12, **kw):
    c = Cache([], page, 2, 64, layers=kw.pop("layers", 2), seqs=seqs, spare_pages=pages, poison=False, **kw)
    c.table = torch.full((seqs, cols), -1, dtype=torch.int32, device="cuda")
    c.handle = fmad.KvCache(c.k, c.v, c.table, c.lens, c.refs, c.k_scale, c.v_scale)
    return c


@pytest.mark.parametrize("fp8,heads_first", [(False, False), (True, True), (False, True)])
def test_a_life_of_sequences(fp8, heads_first):
    require_gpu()
    c = empty(fp8=fp8, heads_first=heads_first)
    ops, book = Ops(c), Book(c)
    assert both(ops, book, "reserve", [3, 0, 5], [20, 16, 1]) == (0, 4)
    assert both(ops, book, "fork", [3, 3, 0], [1, 2, 4]) == (0, 0)
    # 3, 1 and 2 share a begun page: the first two writers copy it, the last keeps it; 0's page is full
    assert both(ops, book, "reserve", [1, 0, 3, 2], [5, 3, 40, 1]) == (0, 1 + 1 + 1 + 2)
    both(ops, book, "reserve", [1], [0])
    both(ops, book, "release", [3, 5], [17, 0])
    both(ops, book, "release", [0])
    both(ops, book, "release", [1], [99])   # more than its length: unchanged
    assert both(ops, book, "compact")[0] == 0
    both(ops, book, "compact")              # nothing left to move
    both(ops, book, "fork", [2], [0])
    both(ops, book, "release", [2, 0, 1, 3, 4])
    assert int(c.refs.abs().sum()) == 0 and int(c.lens.abs().sum()) == 0 and bool((c.table == -1).all())


def test_refused_calls_change_nothing():
    require_gpu()
    c = empty(pages=10)
    ops, book = Ops(c), Book(c)
    both(ops, book, "reserve", [0, 1], [40, 24])    # 3 + 2 pages of 10
    for name, args, want in [
        ("reserve", ([0, 0], [1, 1]), (2, 0)), ("reserve", ([9], [1]), (2, 0)), ("reserve", ([-1], [1]), (2, 0)),
        ("reserve", ([2], [-1]), (2, 0)), ("reserve", ([2], [12 * 16 + 1]), (4, 0)),
        ("reserve", ([2, 3], [16, 5 * 16]), (1, 1)), ("reserve", ([2, 0], [4 * 16, 9]), (0, 5)),
        ("fork", ([0, 1], [5, 5]), (2, 0)), ("fork", ([0], [1]), (2, 0)), ("fork", ([0], [0]), (2, 0)),
        ("fork", ([0, 5], [5, 6]), (2, 0)), ("fork", ([0], [9]), (2, 0)), ("fork", ([-1], [5]), (2, 0)),
        ("release", ([0, 0],), (2, 0)), ("release", ([77],), (2, 0)), ("release", ([0], [-1]), (2, 0)),
    ]:
        assert both(ops, book, name, *args) == want, (name, args)
    # a full pool with a shared begun page: its copy is what is missing
    both(ops, book, "fork", [1], [6])
    assert both(ops, book, "reserve", [1], [1]) == (1, 1)
    assert both(ops, book, "reserve", [], []) == (0, 0)
    assert both(ops, book, "fork", [], []) == (0, 0)
    assert both(ops, book, "release", []) == (0, 0)


def test_contradictory_bookkeeping_is_reported():
    require_gpu()
    c = empty()
    ops = Ops(c)
    assert ops.reserve([0], [20]) == (0, 2)
    c.table[0, 1] = -1
    assert ops.reserve([0], [1]) == (2, 0)
    c.table[0, 1] = 10 ** 6
    assert ops.reserve([0], [1]) == (2, 0)
    c.lens[0] = -4
    assert ops.reserve([0], [1]) == (2, 0) and ops.fork([0], [1]) == (2, 0) and ops.release([0]) == (2, 0)
    c.lens[0] = 10 ** 9
    assert ops.reserve([0], [1]) == (2, 0) and ops.fork([0], [1]) == (2, 0) and ops.release([0]) == (2, 0)


def test_random_histories():
    require_gpu()
    for seed in range(3):
        rng = np.random.default_rng(seed)
        c = empty(page=int(rng.choice([16, 32])), pages=150, seqs=40, cols=20, layers=1, seed=seed)
        ops, book = Ops(c), Book(c)
        for _ in range(25):
            kind = rng.choice(["reserve", "reserve", "fork", "release", "compact"])
            n = int(rng.integers(1, 20))
            if kind == "reserve":
                both(ops, book, kind, list(rng.permutation(40)[:n]), list(rng.integers(0, 60, n)))
            elif kind == "fork":
                order = rng.permutation(40)
                free = [s for s in order if book.lens[s] == 0][:n]
                held = [s for s in range(40) if s not in free]
                both(ops, book, kind, list(rng.choice(held, len(free))) if held else [], free if held else [])
            elif kind == "release":
                both(ops, book, kind, list(rng.permutation(40)[:n]), list(rng.integers(0, 200, n)))
            else:
                both(ops, book, kind)


def test_most_sequences_and_many_pages():
    require_gpu()
    c = Cache([], 16, 1, 16, seqs=1500, spare_pages=70001, poison=False)
    c.table = torch.full((1500, 70), -1, dtype=torch.int32, device="cuda")
    c.handle = fmad.KvCache(c.k, c.v, c.table, c.lens, c.refs)
    ops, book = Ops(c, 1024), Book(c)
    rng = np.random.default_rng(0)
    seq = list(rng.permutation(1500)[:1024])
    both(ops, book, "reserve", seq, list(rng.integers(1, 1000, 1024)))
    both(ops, book, "release", seq[:500])
    both(ops, book, "fork", [seq[1000]] * 470, [s for s in range(1500) if s not in seq][:470])
    both(ops, book, "reserve", [s for s in range(1500) if s not in seq][:470], [1] * 470)
    both(ops, book, "compact")


def test_graph_of_a_serving_step():
    """fork -> reserve -> release captured once, replayed as the bookkeeping changes under it."""
    require_gpu()
    c = empty()
    ops, book = Ops(c), Book(c)
    both(ops, book, "reserve", [0], [20])
    src, dst, cnt = ops._i([0, 0]), ops._i([1, 2]), ops._i([3, 30])
    fmad.kv_fork(c.handle, src, dst, ops.status)    # warm
    fmad.kv_reserve(c.handle, dst, cnt, ops.status, ops.ws)
    fmad.kv_release(c.handle, dst, ops.status)
    torch.cuda.synchronize()
    book.fork([0, 0], [1, 2]), book.reserve([1, 2], [3, 30]), book.release([1, 2])
    book.check(c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fmad.kv_fork(c.handle, src, dst, ops.status)
        fmad.kv_reserve(c.handle, dst, cnt, ops.status, ops.ws)
        fmad.kv_release(c.handle, dst, ops.status)
    for add in (0, 5, 30):
        both(ops, book, "reserve", [0], [add])
        g.replay()
        torch.cuda.synchronize()
        book.fork([0, 0], [1, 2]), book.reserve([1, 2], [3, 30]), book.release([1, 2])
        book.check(c)


def test_a_page_with_more_users_than_its_count():
    """Two rows name a begun page that is counted once: writing to both would mix them, so nothing is done."""
    require_gpu()
    c = empty()
    ops = Ops(c)
    assert ops.reserve([0], [20]) == (0, 2)
    c.table[1], c.lens[1] = c.table[0], 20
    before = [x.clone() for x in (c.table, c.lens, c.refs)]
    assert ops.reserve([0, 1], [1, 1]) == (2, 0)
    assert all(torch.equal(a, b) for a, b in zip(before, (c.table, c.lens, c.refs)))


def test_histories_of_hundreds_of_sequences():
    """Sequence and page numbers far apart and alike modulo powers of two; groups of forks that write in any order."""
    require_gpu()
    rng = np.random.default_rng(11)
    seqs = 4096
    c = Cache([], 16, 1, 16, seqs=seqs, spare_pages=9000, poison=False)
    c.table = torch.full((seqs, 9), -1, dtype=torch.int32, device="cuda")
    c.handle = fmad.KvCache(c.k, c.v, c.table, c.lens, c.refs)
    ops, book = Ops(c, 1024), Book(c)
    roots = [int(x) for x in range(0, seqs, 64)]
    both(ops, book, "reserve", roots, list(rng.integers(1, 60, len(roots))))
    kids = [r + 1 + j for r in roots for j in range(15)]
    both(ops, book, "fork", [k // 64 * 64 for k in kids], kids)
    everyone = roots + kids
    for step in range(3):
        some = [int(x) for x in rng.permutation(everyone)[:1000 if step else 700]]
        both(ops, book, "reserve", some, list(rng.integers(0, 20, len(some))))
    assert both(ops, book, "reserve", everyone[:1000] + [everyone[500]], [1] * 1001) == (2, 0)
    idle = list(range(32, 64)) + [r + 16 + j for r in roots for j in range(15)]
    assert both(ops, book, "fork", [0] * (len(idle) + 1), idle + [33]) == (2, 0)
    assert both(ops, book, "fork", [0, 96], [96, 97]) == (2, 0)
    both(ops, book, "release", [int(x) for x in rng.permutation(everyone)[:900]], list(rng.integers(0, 70, 900)))
    both(ops, book, "compact")
