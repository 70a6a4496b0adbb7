"""Shared by the tests of the paged prefix cache: caches with poisoned free space, plain 64-bit definitions of the
operators, and a sequential model of the page bookkeeping."""
import math

import numpy as np
import torch

import flow_matching_action_denoise_gb300 as fmad


def up(a, b):
    return -(-a // b)


class Cache:
    """A cache whose sequences `rows` hold lens tokens on scattered pages. What lies behind a length and on free pages
    is NaN (E4M3: its NaN code), so that a read out of place shows."""

    def __init__(self, lens, page, Hkv, Dh, fp8=False, layers=1, seqs=None, spare_pages=3, heads_first=False, seed=0,
                 rows=None, extra_cols=2, device="cuda", poison=True):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed + 1)
        held = [up(x, page) for x in lens]
        self.page, self.fp8, self.lens_host = page, fp8, list(lens)
        seqs = seqs or len(lens) + 2
        pages = max(1, sum(held) + spare_pages)
        self.rows = list(rng.permutation(seqs)[:len(lens)]) if rows is None else rows
        order = list(rng.permutation(pages))
        table = np.full((seqs, max(held + [1]) + extra_cols), -1, np.int32)
        ln, refs = np.zeros(seqs, np.int32), np.zeros(pages, np.int32)
        shape = (layers, pages, Hkv, page, Dh) if heads_first else (layers, pages, page, Hkv, Dh)
        data = []
        for _ in range(2):
            t = torch.randn(shape, generator=g)
            t = (t * 16).clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else t.to(torch.bfloat16)
            data.append(t.transpose(2, 3) if heads_first else t)
        bits = [t.view(torch.uint8) if fp8 else t.view(torch.int16) for t in data]
        nan = 0x7F if fp8 else 0x7FC0
        keep = torch.zeros((pages, page), dtype=torch.bool)
        for i, row in enumerate(self.rows):
            ln[row] = lens[i]
            for j in range(held[i]):
                pg = order.pop()
                table[row, j] = pg
                refs[pg] = 1
                keep[pg, :max(0, min(page, lens[i] - j * page))] = True
        if poison:
            for b in bits:
                b.masked_fill_(~keep[None, :, :, None, None], nan)
        self.k, self.v = (t.to(device) for t in data)
        if heads_first:   # .to keeps the strides of a dense permuted tensor
            assert self.k.stride() == data[0].stride()
        self.table, self.lens, self.refs = (torch.from_numpy(x).to(device) for x in (table, ln, refs))
        r = torch.rand(2, layers, generator=g) * 0.05 + 0.05
        self.k_scale, self.v_scale = (x.to(device) for x in r) if fp8 else (None, None)
        self.handle = fmad.KvCache(self.k, self.v, self.table, self.lens, self.refs, self.k_scale, self.v_scale)

    def dense(self, i, layer=0):
        """(K, V) of entry i in float64, [len][Hkv][Dh]."""
        n, row = self.lens_host[i], self.rows[i]
        at = torch.arange(n, device=self.k.device)
        pg = self.table[row][at // self.page].long()
        out = []
        for t, s in ((self.k, self.k_scale), (self.v, self.v_scale)):
            x = t[layer].to(torch.float64)[pg, at % self.page]
            out.append(x * s[layer].double() if self.fp8 else x)
        return out


def batch(cache, new, seq=True, lead=0, trail=0, max_tokens=None, max_len=None):
    """KvBatch of entries with `new` tokens each; lead/trail: packed rows before the first and behind the last."""
    start = lead + np.concatenate([[0], np.cumsum(new)])
    dev = cache.k.device
    start = torch.tensor(start, dtype=torch.int32, device=dev)
    ids = torch.tensor(np.asarray(cache.rows), dtype=torch.int32, device=dev) if seq else None
    tokens = lead + int(sum(new)) + trail
    return fmad.KvBatch(start, tokens, max(list(new) + [0]) if max_tokens is None else max_tokens,
                        max(cache.lens_host + [0]) if max_len is None else max_len, ids)


def attention_ref(cache, i, q, scale, causal, window, layer=0):
    """(out, sum_j p_j |v_j|) of entry i's q [new][H][Dh] in float64."""
    k, v = cache.dense(i, layer)
    n, H, Dh = q.shape
    ln = cache.lens_host[i]
    q = q.double()
    G = H // k.shape[1]
    pos = torch.arange(ln - n, ln, device=q.device)[:, None]
    key = torch.arange(ln, device=q.device)[None]
    ok = (pos >= 0) & (key >= 0)
    if causal:
        ok = ok & (key <= pos)
    if window:
        ok = ok & (key > pos - window)
    out, size = torch.zeros_like(q), torch.zeros_like(q)
    for h in range(H):
        s = (q[:, h] @ k[:, h // G].T) * scale
        s = s.masked_fill(~ok, -math.inf)
        top = s.amax(-1, keepdim=True) if ln else s.new_zeros((n, 1))
        p = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
        p = p / torch.where(p.sum(-1, keepdim=True) > 0, p.sum(-1, keepdim=True), torch.ones_like(top))
        out[:, h], size[:, h] = p @ v[:, h // G], p @ v[:, h // G].abs()
    return out, size


class Book:
    """The page bookkeeping, one entry after the other on the host."""

    def __init__(self, cache):
        self.page = cache.page
        self.table, self.lens, self.refs = (x.cpu().numpy().copy() for x in (cache.table, cache.lens, cache.refs))
        self.k, self.v = cache.k.clone(), cache.v.clone()

    def _bits(self, t):
        return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int16)

    def copy(self, src, dst, rows):
        for t in (self.k, self.v):
            b = self._bits(t)
            b[:, dst, :rows] = b[:, src, :rows]

    def reserve(self, seq, count):
        table, lens, refs = self.table.copy(), self.lens.copy(), self.refs.copy()
        copies, taken, missing = [], 0, 0
        held = set()
        if len(set(seq)) < len(seq):
            return 2, 0
        free = [int(x) for x in np.flatnonzero(refs == 0)]
        for s, c in zip(seq, count):
            if s < 0 or s >= len(lens) or c < 0:
                return 2, 0
            if lens[s] + c > table.shape[1] * self.page:
                return 4, 0
            want = []
            at = lens[s] // self.page
            if c and lens[s] % self.page and refs[table[s, at]] > 1:
                want.append(("copy", at))
            want += [("new", j) for j in range(up(lens[s], self.page), up(lens[s] + c, self.page))]
            for kind, j in want:
                if not free:
                    missing += 1
                    if kind == "copy":
                        refs[table[s, j]] -= 1
                    continue
                pg = free.pop(0)
                held.add(pg)
                taken += 1
                if kind == "copy":
                    copies.append((int(table[s, j]), pg, int(lens[s] % self.page)))
                    refs[table[s, j]] -= 1
                table[s, j] = pg
                refs[pg] = 1
            lens[s] += c
        if missing:
            return 1, missing
        self.table, self.lens, self.refs = table, lens, refs
        for c in copies:
            self.copy(*c)
        return 0, taken

    def fork(self, src, dst):
        if len(set(dst)) < len(dst) or set(src) & set(dst):
            return 2, 0
        if any(x < 0 or x >= len(self.lens) for x in list(src) + list(dst)) or any(self.lens[d] for d in dst):
            return 2, 0
        for s, d in zip(src, dst):
            self.table[d], self.lens[d] = self.table[s], self.lens[s]
            for pg in self.table[s][self.table[s] >= 0]:
                self.refs[pg] += 1
        return 0, 0

    def release(self, seq, keep=None):
        keep = [0] * len(seq) if keep is None else keep
        if len(set(seq)) < len(seq) or any(s < 0 or s >= len(self.lens) for s in seq) or any(k < 0 for k in keep):
            return 2, 0
        for s, k in zip(seq, keep):
            k = min(k, self.lens[s])
            for j in range(up(k, self.page), self.table.shape[1]):
                if self.table[s, j] >= 0:
                    self.refs[self.table[s, j]] -= 1
                    self.table[s, j] = -1
            self.lens[s] = k
        return 0, 0

    def compact(self):
        live = int((self.refs > 0).sum())
        src = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] == 0]
        for a, b in zip(src, dst):
            self.copy(a, b, self.page)
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.table[self.table == a] = b
        return 0, len(src)

    def check(self, cache):
        assert np.array_equal(self.table, cache.table.cpu().numpy())
        assert np.array_equal(self.lens, cache.lens.cpu().numpy())
        assert np.array_equal(self.refs, cache.refs.cpu().numpy())
        for a, b in ((self.k, cache.k), (self.v, cache.v)):
            assert torch.equal(self._bits(a), self._bits(b))
