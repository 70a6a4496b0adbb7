"""Attention of a batch in groups of forks, against the definition of plain attention in 64 bits.

Tolerance: the plain attention's (its tests derive it): 2^-8 |o| for the output's rounding, (2^-8 or, with an E4M3 cache,
2^-11, + 2^-9) sum_j p_j |v_j| for probabilities and scores. The join of the prefix with an entry's own keys is in fp32:
its weights and sums are off by 2^-20 of sum_j p_j |v_j| at most, far inside of the second term's slack."""
import numpy as np
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import attention_ref, batch, up

pytestmark = pytest.mark.gpu


class Forks:
    """Sequences in groups: (shared tokens, [tokens behind them, one number an entry]). Whole shared pages are the first
    entry's, a begun one is a copy; what lies behind a length and on free pages is NaN."""

    def __init__(self, groups, page, Hkv, Dh, fp8=False, heads_first=False, layers=1, seed=0, lone=(), in_order=False):
        g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed + 1)
        self.page, self.fp8, self.first, self.shared, self.lens_host = page, fp8, [0], [], []
        lead = []
        for shared, own in groups:
            lead += [(len(lead), shared)] * len(own) if own else []
            self.shared.append(shared)
            self.lens_host += [shared + x for x in own]
            self.first.append(len(self.lens_host))
        for x in lone:   # entries behind the last group
            lead.append((len(lead), 0))
            self.lens_host.append(x)
        n = len(self.lens_host)
        pages = sum(up(x, page) - (s // page if i != j else 0) for i, (x, (j, s)) in enumerate(zip(self.lens_host, lead))) + 3
        self.rows = list(range(n)) if in_order else list(rng.permutation(n + 2)[:n])
        order = list(rng.permutation(pages))
        table = np.full((n + 2, max(up(x, page) for x in self.lens_host) + 2), -1, np.int32)
        lens, keep, begun = np.zeros(n + 2, np.int32), torch.zeros((pages, page), dtype=torch.bool), []
        for i, (x, (j, s)) in enumerate(zip(self.lens_host, lead)):
            lens[self.rows[i]] = x
            for p in range(up(x, page)):
                if i != j and p < s // page:
                    table[self.rows[i], p] = table[self.rows[j], p]
                    continue
                pg = table[self.rows[i], p] = order.pop()
                keep[pg, :min(page, x - p * page)] = True
                if i != j and p == s // page and s % page:
                    begun.append((int(table[self.rows[j], p]), int(pg), s % page))
        shape = (layers, pages, Hkv, page, Dh) if heads_first else (layers, pages, page, Hkv, Dh)
        data = []
        for _ in range(2):
            t = torch.randn(shape, generator=g)
            t = (t * 16).clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else t.to(torch.bfloat16)
            t = t.transpose(2, 3) if heads_first else t
            bits = t.view(torch.uint8) if fp8 else t.view(torch.int16)
            for a, b, rows in begun:
                bits[:, b, :rows] = bits[:, a, :rows]
            bits.masked_fill_(~keep[None, :, :, None, None], 0x7F if fp8 else 0x7FC0)
            data.append(t)
        self.k, self.v = (t.to("cuda") for t in data)
        self.table, self.lens = (torch.from_numpy(x).cuda() for x in (table, lens))
        r = torch.rand(2, layers, generator=g) * 0.05 + 0.05
        self.k_scale, self.v_scale = (x.cuda() for x in r) if fp8 else (None, None)
        self.handle = fmad.KvCache(self.k, self.v, self.table, self.lens, None, self.k_scale, self.v_scale)

    def dense(self, i, layer=0):
        n, row = self.lens_host[i], self.rows[i]
        at = torch.arange(n, device="cuda")
        pg = self.table[row][at // self.page].long()
        out = []
        for t, s in ((self.k, self.k_scale), (self.v, self.v_scale)):
            x = t[layer].to(torch.float64)[pg, at % self.page]
            out.append(x * s[layer].double() if self.fp8 else x)
        return out

    def groups(self, max_entries=None, max_shared=None, first=None, shared=None):
        first, shared = first or self.first, self.shared if shared is None else shared
        most = max([b - a for a, b in zip(self.first, self.first[1:])] + [0])
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
        return fmad.KvGroups(i32(first), i32(shared), most if max_entries is None else max_entries,
                             max(list(self.shared) + [0]) if max_shared is None else max_shared)


def attend(c, new, H, causal=True, scale=None, lead=0, trail=0, layer=0, seed=5, groups=None, b=None, shares=True, status=0,
           pad=0, q=None):
    b, groups, Dh = b or batch(c, new, True, lead, trail), groups or c.groups(), c.k.shape[-1]
    if q is None:
        q = torch.randn((b.tokens, H + pad, Dh), generator=torch.Generator().manual_seed(seed)).mul_(1.5).to(torch.bfloat16).cuda()
        q = q[:, :H]
    out = torch.full((b.tokens, H + pad, Dh), 7.0, dtype=torch.bfloat16, device="cuda")
    need = fmad.shared_attention_workspace_size(c.handle, b, groups, H)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN, and a border
    if shares is not None and not status:   # groups are read, and bad ones reported, only where the plan is to share
        bad = fmad.KvGroups(groups.first, torch.full_like(groups.shared, -1), groups.struct.max_entries, groups.struct.max_shared)
        fmad.shared_attention(c.handle, layer, b, bad, q, out[:, :H], ws[:need], scale, causal)
        assert fmad.standalone_status() == (2 if shares else 0)
        out.fill_(7.0)
    fmad.shared_attention(c.handle, layer, b, groups, q, out[:, :H], ws[:need], scale, causal)
    torch.cuda.synchronize()
    assert fmad.standalone_status() == status
    assert (out[:, H:] == 7).all() and (ws[need:] == 0xFF).all()
    return q, out[:, :H], b


def check(c, new, q, out, b, causal=True, scale=None, layer=0, skip=()):
    scale = c.k.shape[-1] ** -0.5 if scale is None else scale
    start = b.start.cpu().numpy()
    assert (out[:start[0]] == 7).all() and (out[start[-1]:] == 7).all()
    for i, n in enumerate(new):
        if i in skip:
            continue
        rows = slice(int(start[i]), int(start[i + 1]))
        ref, size = attention_ref(c, i, q[rows], scale, causal, 0, layer)
        tol = ref.abs() * 2.0 ** -8 + size * ((2.0 ** -11 if c.fp8 else 2.0 ** -8) + 2.0 ** -9)
        err = (out[rows].double() - ref).abs()
        assert bool((err <= tol).all()), (i, n, c.lens_host[i], float((err - tol).max()), float(err.max()))


def spread(n, lo, hi, seed=0):
    return [int(x) for x in np.random.default_rng(seed).integers(lo, hi + 1, n)]


# enough entries and shared tokens to be divided: (H, Hkv, Dh)
HEADS = [(16, 2, 128), (8, 1, 64), (5, 5, 64), (6, 2, 128)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,Hkv,Dh", HEADS)
@pytest.mark.parametrize("shared,page", [(8192, 64), (8195, 16), (8223, 256)])
def test_single_tokens(shared, page, H, Hkv, Dh, fp8):
    """The prefix ends at a page's border, at a tile's, inside of both; one token behind it, or a few hundred."""
    require_gpu()
    own = [1, 2, 64, 65, 128, 300] + spread(120, 1, 40)
    c = Forks([(shared, own)], page, Hkv, Dh, fp8, heads_first=page == 64, seed=shared)
    new = [1] * len(own)
    q, out, b = attend(c, new, H, lead=1, trail=2)
    check(c, new, q, out, b)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,Hkv,Dh,most", [(16, 2, 128, 2), (10, 2, 64, 5), (4, 4, 64, 16), (14, 2, 64, 9), (12, 3, 128, 31)])
def test_several_tokens_and_groups(H, Hkv, Dh, most, causal, fp8):
    """Up to 16 and up to 128 rows an entry, groups of different lengths and counts, one of them of a single entry."""
    require_gpu()
    groups = [(20003, spread(55, most, 90, 1)), (700, [most + 3]), (8960, spread(35, most, 50, 2))]
    c = Forks(groups, 32, Hkv, Dh, fp8, seed=most)
    n = len(c.lens_host)
    new = [most] + [1 + x % most for x in spread(n - 1, 0, 100, 3)]
    q, out, b = attend(c, new, H, causal, scale=0.11, lead=3, shares=True if most < 31 else None)
    check(c, new, q, out, b, causal, 0.11)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefixes_that_are_not_for_all(fp8):
    """Tokens inside of the shared part (which then belong to no prefix), entries without tokens, an empty group, groups that
    share nothing, entries outside of all groups, empty sequences."""
    require_gpu()
    groups = [(6000, [1] * 60 + [0, 0, 2, 0]), (900, []), (0, [50, 0, 700]), (5500, [3] * 40 + [0])]
    c = Forks(groups, 16, 2, 128, fp8, seed=3, lone=[300, 0, 1])
    n = len(c.lens_host)
    new = [1] * n
    new[3], new[60], new[61], new[62], new[70] = 2, 2, 1, 0, 0   # entry 3 has one token of the prefix among its new ones
    for causal in (True, False):
        q, out, b = attend(c, new, 8, causal)
        check(c, new, q, out, b, causal)
        empty = [i for i in range(n) if c.lens_host[i] == 0 and new[i]]
        assert len(empty) == 2 and all((out[int(b.start[i])] == 0).all() for i in empty)


def test_entries_before_the_first_group():
    require_gpu()
    c = Forks([(2000, [5] * 4), (8000, [9] * 100)], 32, 2, 64, seed=4)
    new = [1] * 104
    q, out, b = attend(c, new, 8, groups=c.groups(first=[4, 104], shared=[8000]))
    check(c, new, q, out, b)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_groups_and_entries_in_order(fp8):
    """More groups than a warp has lanes, most of them empty; sequences without a list of them."""
    require_gpu()
    c = Forks([(8195, [3] * 130)] + [(100, [])] * 33 + [(6000, [2, 70] * 55), (50, [])] + [(0, [x]) for x in (90, 5, 1)] + [(7, [])],
              64, 1, 128, fp8, seed=15, in_order=True)
    new = [1] * len(c.lens_host)
    q, out, b = attend(c, new, 8, b=batch(c, new, False))
    check(c, new, q, out, b)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [dict(max_entries=70), dict(max_entries=33), dict(max_shared=3900), dict(max_shared=9000),
                                dict(max_entries=500, max_shared=4500)])
def test_other_bounds_than_the_counts(kw, fp8):
    require_gpu()
    c = Forks([(4100, spread(80, 1, 60))], 64, 2, 128, fp8, seed=5)
    new = [1 + i % 2 for i in range(80)]
    q, out, b = attend(c, new, 16, groups=c.groups(**kw))
    check(c, new, q, out, b)


def test_a_bound_on_the_lengths_that_is_too_small():
    require_gpu()
    c = Forks([(4100, [1, 1, 900] + [3] * 70)], 64, 2, 128, seed=6)
    new = [1] * 73
    q, out, b = attend(c, new, 16, b=batch(c, new, max_len=4120))
    check(c, new, q, out, b)


@pytest.mark.parametrize("H,Hkv,Dh,most", [(16, 2, 128, 1), (14, 2, 64, 4)])
def test_long_own_parts_are_split(H, Hkv, Dh, most):
    """Clusters over an entry's own keys."""
    require_gpu()
    c = Forks([(16000, [3000] + spread(9, most, 2500))], 128, Hkv, Dh, seed=7)
    new = [1 + i % most for i in range(10)]
    q, out, b = attend(c, new, H)
    check(c, new, q, out, b)
    c = Forks([(16000, [1500] + spread(23, 4, 1500))], 128, Hkv, Dh, True, seed=7)
    new = [1 + i % most for i in range(24)]
    q, out, b = attend(c, new, H)
    check(c, new, q, out, b)


@pytest.mark.parametrize("groups,new", [([(788, [5] * 8)], 1), ([(4000, [60] * 16)], 50), ([(40, [3] * 50)], 2)])
def test_where_sharing_costs_more_it_is_paged_attention(groups, new):
    require_gpu()
    c = Forks(groups, 16, 2, 128, seed=8)
    new = [new] * len(c.lens_host)
    q, out, b = attend(c, new, 16, shares=False)
    check(c, new, q, out, b)
    other = torch.full_like(out, 7.0)
    ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, 16), dtype=torch.uint8, device="cuda")
    fmad.paged_attention(c.handle, 0, b, q, other, ws)
    assert torch.equal(out, other)
    none = fmad.KvGroups(torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"), 0, 0)
    q, out, b = attend(c, new, 16, groups=none, shares=False)
    assert torch.equal(out, other)
    empty = fmad.KvBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), 0, 0, 0)
    fmad.shared_attention(c.handle, 0, empty, none, q[:0], out[:0])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("most", [1, 6])
def test_nan_in_one_query_or_one_entry_stays_there(most, fp8):
    require_gpu()
    c = Forks([(8100, [20] * 110)], 16, 2, 64, fp8, seed=9)
    new = [most] * 110
    q, clean, b = attend(c, new, 8, False)
    token, head = 110 * most - 1, 3
    q[token, head, 5] = float("nan")
    _, out, _ = attend(c, new, 8, False, q=q)
    assert out[token, head].isnan().all()
    out[token, head] = clean[token, head]
    assert torch.equal(out, clean)
    q[token, head, 5] = 1.0
    _, clean, _ = attend(c, new, 8, False, q=q)
    page = c.table[c.rows[11], 8110 // 16].long()   # one key and value of entry 11
    for t in (c.k, c.v):
        (t.view(torch.uint8) if fp8 else t.view(torch.int16))[:, page, 8110 % 16] = 0x7F if fp8 else 0x7FC0
    _, out, _ = attend(c, new, 8, False, q=q)
    rows = slice(11 * most, 12 * most)
    assert out[rows].isnan().all()
    out[rows] = clean[rows]
    assert torch.equal(out, clean)


def test_infinite_scores_far_apart():
    """The prefix's and the own part's maxima differ by more than exp can hold, either way."""
    require_gpu()
    c = Forks([(4096, [40] * 64)], 64, 2, 128, seed=10)
    new = [1] * 64
    for big, where in ((c.table[c.rows[0], 3].long(), "prefix"), (c.table[c.rows[5], 64].long(), "own")):
        saved = c.k.clone()
        c.k[:, big] *= 200
        q, out, b = attend(c, new, 16)
        check(c, new, q, out, b)
        c.k.copy_(saved)


def test_layers_strides_and_order():
    require_gpu()
    c = Forks([(6000, [30] * 104)], 32, 2, 64, layers=3, seed=11)
    new = [1] * 104
    for layer in (0, 2):
        q, out, b = attend(c, new, 14, layer=layer, pad=2)
        check(c, new, q, out, b, layer=layer)


@pytest.mark.parametrize("fp8", [False, True])
def test_repeats_graphs_streams_and_lengths(fp8):
    """The same bits every time; a captured call works on the lengths and groups that it finds."""
    require_gpu()
    c = Forks([(6500, [30] * 60), (5000, [9] * 40)], 64, 2, 128, fp8, seed=12)
    new = [1 + i % 2 for i in range(100)]
    q, eager, b = attend(c, new, 16)
    groups = c.groups()
    ws = torch.empty(fmad.shared_attention_workspace_size(c.handle, b, groups, 16), dtype=torch.uint8, device="cuda")
    s, g, replay = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.zeros_like(eager)
    with torch.cuda.graph(g, stream=s):
        for _ in range(3):   # one after the other in one workspace
            fmad.shared_attention(c.handle, 0, b, groups, q, replay, ws)
    for _ in range(3):
        replay.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, replay)
    other = torch.empty_like(q)
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        fmad.shared_attention(c.handle, 0, b, groups, q, other, ws, stream=s)
    s.synchronize()
    assert torch.equal(eager, other)
    c.lens[c.rows[3]] -= 5
    c.lens_host[3] -= 5
    groups.shared[0] = 6444   # a prefix may be shorter than what is shared
    g.replay()
    torch.cuda.synchronize()
    check(c, new, q, replay, b)
    assert fmad.standalone_status() == 0


@pytest.mark.parametrize("most", [1, 5])
def test_right_behind_the_kernel_that_writes_the_keys(most):
    """Appended keys, then attention, many times over without a wait: the second kernel starts beside the first."""
    require_gpu()
    c = Forks([(8100, [40] * 100)], 16, 2, 64, seed=13)
    new = [most] * 100
    b, groups, T = batch(c, new), c.groups(), 100 * most
    ws = torch.empty(fmad.shared_attention_workspace_size(c.handle, b, groups, 8), dtype=torch.uint8, device="cuda")
    rope, q, out = fmad.Rope(64), torch.empty((T, 8, 64), dtype=torch.bfloat16, device="cuda"), []
    assert ws.numel() > 0
    kv = [torch.randn((T, 12, 64), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in range(6)]
    for x in kv:
        o = torch.empty_like(q)
        fmad.norm_rope_append(c.handle, 0, b, rope, x[:, :8], x[:, 8:10], x[:, 10:], q, eps=1e-6)
        fmad.shared_attention(c.handle, 0, b, groups, q, o, ws)
        out.append(o)
    for x, o in zip(kv, out):
        fmad.norm_rope_append(c.handle, 0, b, rope, x[:, :8], x[:, 8:10], x[:, 10:], q, eps=1e-6)
        torch.cuda.synchronize()
        check(c, new, q, o, b)
    assert fmad.standalone_status() == 0


def test_two_streams_with_workspaces_of_their_own():
    require_gpu()
    c = Forks([(8100, [30] * 110)], 64, 2, 128, seed=16)
    new = [1] * 110
    q, want, b = attend(c, new, 16)
    groups = c.groups()
    need = fmad.shared_attention_workspace_size(c.handle, b, groups, 16)
    streams = [torch.cuda.Stream() for _ in range(3)]
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [[torch.empty_like(want) for _ in range(6)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(6):
        for s, w, o in zip(streams, ws, outs):
            fmad.shared_attention(c.handle, 0, b, groups, q, o[i], w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(want, x) for o in outs for x in o) and fmad.standalone_status() == 0


def test_device_side_faults_are_reported():
    require_gpu()
    c = Forks([(8100, [20] * 100)], 16, 2, 64, seed=14)
    new = [1] * 100
    q, clean, b = attend(c, new, 8)
    # groups out of range share nothing; all results stay right
    for first, shared in (([0, 101], [8100]), ([-1, 100], [8100]), ([0, 100], [8121]), ([0, 100], [-1]), ([0, 100], [10 ** 9]),
                          ([0, 50, 30, 100], [8100] * 3), ([100, 0], [8100])):
        q, out, _ = attend(c, new, 8, groups=c.groups(first=first, shared=shared), status=2)
        check(c, new, q, out, b)
    assert attend(c, new, 8)[1].equal(clean)
    # pages
    for place in (0, 100, 507):
        saved = int(c.table[c.rows[0], place])
        for page in (-1, 10 ** 6):
            c.table[c.rows[0], place] = page
            attend(c, new, 8, status=2)
        c.table[c.rows[0], place] = saved
    # entries
    ids = torch.tensor(np.asarray(c.rows), dtype=torch.int32, device="cuda")
    good = list(range(101))
    for at, value in ((100, 101), (0, -1), (50, 30)):
        start = list(good)
        start[at] = value
        bad = fmad.KvBatch(torch.tensor(start, dtype=torch.int32, device="cuda"), 100, 1, 8200, ids)
        attend(c, new, 8, b=bad, status=2)
    for row in (0, 7):
        ids[row] += 10 ** 6
        attend(c, new, 8, b=fmad.KvBatch(b.start, 100, 1, 8200, ids), status=2)
        ids[row] -= 10 ** 6
    assert attend(c, new, 8)[1].equal(clean)


def test_the_binding_refuses():
    require_gpu()
    c = Forks([(20, [4, 3])], 16, 2, 64, seed=1)
    b, groups = batch(c, [2, 2]), c.groups()
    q = torch.zeros((4, 4, 64), device="cuda", dtype=torch.bfloat16)
    good = dict(q=q, out=torch.empty_like(q))
    fmad.shared_attention(c.handle, 0, b, groups, **good)
    for bad in (dict(q=q[0]), dict(q=q[:3]), dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :, ::2]), dict(q=q[:, :3]),
                dict(out=q[:, :2]), dict(workspace=torch.empty(64)), dict(scale=0.0), dict(layer=1)):
        with pytest.raises(fmad.FmError):
            fmad.shared_attention(c.handle, bad.pop("layer", 0), b, groups, **{**good, **bad})
    first, shared = groups.first, groups.shared
    for args in ((first.cpu(), shared, 2, 20), (first.long(), shared, 2, 20), (first, shared[:0], 2, 20), (first[:0], shared, 2, 20),
                 (first, shared.float(), 2, 20)):
        with pytest.raises(fmad.FmError):
            fmad.KvGroups(*args)
    for args in ((first, shared, -1, 20), (first, shared, 2, -1)):
        with pytest.raises(fmad.FmError):
            fmad.shared_attention(c.handle, 0, b, fmad.KvGroups(*args), **good)
    cpu = fmad.KvGroups(first.cpu(), shared.cpu(), 2, 20)
    with pytest.raises(fmad.FmError):
        fmad.shared_attention(c.handle, 0, b, cpu, **good)
