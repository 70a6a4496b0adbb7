"""The paged prefix cache's entry points refuse bad arguments on the host with their status codes, and the rotary table
is what its formulas say (no GPU: nothing here launches a kernel)."""
import ctypes
import math
import os

import numpy as np
import pytest

import flow_matching_action_denoise_gb300 as fmad

P = 1 << 20   # a well-aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fmad.LIB_PATH):
        from flow_matching_action_denoise_gb300 import build
        build.build()
    return fmad.load()


def cache(**kw):
    c = fmad.FmKvCache(k=P, v=P, fmt=fmad.FMT_BF16, layers=2, pages=10, page_tokens=16, Hkv=2, Dh=64,
                       layer_stride=10 * 16 * 128, page_stride=16 * 128, token_stride=128, head_stride=64, table=P,
                       lens=P, refs=P, seqs=4, table_stride=8)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def batch(**kw):
    b = fmad.FmKvBatch(start=P, seq=P, n=2, tokens=5, max_tokens=3, max_len=100)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def at(x):
    return ctypes.addressof(x)


BAD_CACHES = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(fmt=2), 1), (dict(fmt=1), 1),
    (dict(layers=0), 2), (dict(pages=0), 2), (dict(Hkv=0), 2), (dict(seqs=0), 2), (dict(table_stride=0), 2),
    (dict(page_tokens=8), 2), (dict(page_tokens=48), 2), (dict(page_tokens=512), 2), (dict(Dh=72), 2), (dict(Dh=272), 2),
    (dict(k=P + 8), 3), (dict(v=P + 2), 3), (dict(token_stride=120), 2), (dict(head_stride=60), 2),
    (dict(page_stride=128), 2), (dict(page_stride=4096), 2), (dict(layer_stride=16), 2), (dict(token_stride=132), 2), (dict(head_stride=-64), 2),
    (dict(page_stride=1 << 50), 2), (dict(table_stride=1 << 28), 2),
    (dict(table_stride=(1 << 26) + 1), 2), (dict(table_stride=1 << 26, seqs=32), 2),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(lib, kw, status):
    c, b, n = cache(**kw), batch(), ctypes.c_size_t()
    assert lib.fm_kv_workspace_size(at(c), 1, ctypes.byref(n)) == status
    assert lib.fm_kv_compact(at(c), P, P, 1 << 20, None) == status
    assert lib.fm_kv_reserve(at(c), P, P, 1, P, P, 1 << 20, None) == status
    assert lib.fm_kv_fork(at(c), P, P, 1, P, None) == status
    assert lib.fm_kv_release(at(c), P, None, 1, P, None) == status
    assert lib.fm_paged_attention(at(c), 0, at(b), P, 128, 2, 1.0, 1, 0, P, 128, P, 1 << 30, None) == status
    assert lib.fm_paged_attention_workspace_size(at(c), at(b), 2, ctypes.byref(n)) == status
    r = fmad.FmRope(P, 16, 0, 1.0)
    assert lib.fm_rope_append(at(c), 0, at(b), at(r), P, 128, 2, P, 128, P, 128, P, 128, None, None) == status


@pytest.mark.parametrize("kw", [
    dict(token_stride=64, head_stride=16 * 64), dict(layer_stride=16 * 128, page_stride=2 * 16 * 128),
    dict(layer_stride=10 * 4096, page_stride=4096),
    dict(Hkv=1, head_stride=7, token_stride=64), dict(layers=1, layer_stride=3), dict(pages=1, page_stride=1),
])
def test_stride_orders_that_do_not_overlap(lib, kw):
    n = ctypes.c_size_t()
    assert lib.fm_kv_workspace_size(at(cache(**kw)), 3, ctypes.byref(n)) == 0


def test_page_calls(lib):
    c, n = cache(), ctypes.c_size_t()
    assert lib.fm_kv_workspace_size(at(c), 5, None) == 1
    assert lib.fm_kv_workspace_size(at(c), -1, ctypes.byref(n)) == 2
    assert lib.fm_kv_workspace_size(at(c), 1025, ctypes.byref(n)) == 2
    assert lib.fm_kv_workspace_size(at(c), 5, ctypes.byref(n)) == 0
    need = n.value
    assert lib.fm_kv_reserve(at(c), P, P, 5, P, P, need - 1, None) == 4
    assert lib.fm_kv_reserve(at(c), P, P, 5, P, None, need, None) == 1
    assert lib.fm_kv_reserve(at(c), P, P, 5, P, P + 4, need, None) == 3
    assert lib.fm_kv_reserve(at(c), None, P, 5, P, P, need, None) == 1
    assert lib.fm_kv_reserve(at(c), P, None, 5, P, P, need, None) == 1
    assert lib.fm_kv_reserve(at(c), P, P, 5, None, P, need, None) == 1
    assert lib.fm_kv_reserve(at(c), P, P, 1025, P, P, 1 << 30, None) == 2
    assert lib.fm_kv_compact(at(c), None, P, need, None) == 1
    assert lib.fm_kv_compact(at(c), P, P, 8, None) == 4
    assert lib.fm_kv_fork(at(c), P, None, 2, P, None) == 1 and lib.fm_kv_fork(at(c), P, P, -1, P, None) == 2
    assert lib.fm_kv_release(at(c), None, None, 2, P, None) == 1
    bare = cache(refs=None)
    assert lib.fm_kv_release(at(bare), P, None, 2, P, None) == 1 and lib.fm_kv_fork(at(bare), P, P, 2, P, None) == 1
    assert lib.fm_kv_release(None, P, None, 2, P, None) == 1


def test_attention(lib):
    c, b = cache(), batch()

    def call(c=c, b=b, layer=0, q=P, qs=256, H=4, scale=0.1, window=0, out=P, os_=256, ws=P, nb=1 << 40):
        return lib.fm_paged_attention(at(c), layer, at(b) if b else None, q, qs, H, scale, 1, window, out, os_, ws, nb, None)

    assert call(b=None) == 1 and call(layer=2) == 1 and call(layer=-1) == 1
    assert call(q=None) == 1 and call(out=None) == 1
    assert call(H=3) == 2 and call(H=0) == 2 and call(H=-2) == 2
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(scale=s) == 1
    assert call(window=-1) == 1
    assert call(qs=248) == 2 and call(os_=248) == 2 and call(qs=260) == 2
    assert call(q=P + 8) == 3 and call(out=P + 2) == 3
    assert call(c=cache(Dh=32, token_stride=64, head_stride=32), qs=128, os_=128) == 2
    for kw in (dict(n=-1), dict(tokens=-1), dict(max_tokens=-1), dict(max_len=-1), dict(n=70000), dict(seq=None, n=5),
               dict(max_tokens=1 << 30)):
        assert call(b=batch(**kw)) == 2
    assert call(b=batch(start=None)) == 1
    # a long key axis needs its workspace
    long = cache(table_stride=4000)
    n = ctypes.c_size_t()
    bl = batch(n=1, tokens=1, max_tokens=1, max_len=60000)
    assert lib.fm_paged_attention_workspace_size(at(long), at(bl), 4, ctypes.byref(n)) == 0 and n.value > 0
    assert call(c=long, b=bl, ws=None) == 1 and call(c=long, b=bl, nb=n.value - 1) == 4 and call(c=long, b=bl, ws=P + 8) == 3
    assert lib.fm_paged_attention_workspace_size(at(long), at(bl), 4, None) == 1
    # nothing to do
    assert call(b=batch(n=0)) == 0 and call(b=batch(tokens=0)) == 0 and call(b=batch(max_tokens=0)) == 0


def test_a_loose_bound_on_the_new_tokens(lib):
    """max_tokens above the packed rows changes neither the variant nor the workspace."""
    c, a, b = cache(table_stride=4000), ctypes.c_size_t(), ctypes.c_size_t()
    for tokens, H in ((1, 4), (5, 4), (40, 64)):
        tight, loose = (batch(n=1, tokens=tokens, max_tokens=m, max_len=60000) for m in (tokens, 1 << 20))
        assert lib.fm_paged_attention_workspace_size(at(c), at(tight), H, ctypes.byref(a)) == 0
        assert lib.fm_paged_attention_workspace_size(at(c), at(loose), H, ctypes.byref(b)) == 0
        assert a.value == b.value > 0


def test_rope_append(lib):
    def call(c=cache(), b=batch(), layer=0, r=fmad.FmRope(P, 64, 0, 1.0), q=P, qs=256, H=4, k=P, ks=128, v=P, vs=128,
             out=P, os_=256):
        return lib.fm_rope_append(at(c), layer, at(b), at(r) if r else None, q, qs, H, k, ks, v, vs, out, os_, None, None)

    assert call(r=None) == 1 and call(layer=2) == 1
    for dim in (-16, 8, 72, 80, 128):
        assert call(r=fmad.FmRope(P, dim, 0, 1.0)) == 2
    assert call(r=fmad.FmRope(None, 16, 0, 1.0)) == 1
    assert call(r=fmad.FmRope(P, 16, 2, 1.0)) == 1 and call(r=fmad.FmRope(P, 16, 0, math.nan)) == 1
    assert call(q=None) == 1 and call(out=None) == 1 and call(k=None) == 1 and call(v=None) == 1
    assert call(qs=252) == 2 and call(ks=120) == 2 and call(vs=132) == 2 and call(os_=128) == 2 and call(H=-1) == 2
    assert call(q=P + 2) == 3 and call(k=P + 8) == 3 and call(v=P + 8) == 3 and call(out=P + 4) == 3
    assert call(b=batch(n=0)) == 0


def test_norm_quant(lib):
    def call(x=P, xs=256, f32=1, r=P, rs=256, gamma=P, T=4, d=256, eps=1e-6, out=P, os_=256, codes=P, scales=P, block=0):
        return lib.fm_norm_quant(x, xs, f32, r, rs, gamma, T, d, eps, out, os_, codes, scales, block, None)

    for d in (0, 8, 24, 16400, -16):
        assert call(d=d) == 2
    assert call(T=-1) == 2 and call(T=0) == 0
    assert call(block=64) == 1 and call(eps=-1.0) == 1 and call(eps=math.nan) == 1
    assert call(x=None) == 1 and call(codes=None) == 1 and call(scales=None) == 1
    assert call(xs=248) == 2 and call(rs=260) == 2 and call(os_=128) == 2
    assert call(x=P + 4) == 3 and call(r=P + 2) == 3 and call(gamma=P + 4) == 3 and call(out=P + 8) == 3 and call(codes=P + 8) == 3


def test_refresh_prefix_pages_needs_a_policy(lib):
    assert lib.refresh_prefix_pages(None, 0, 1, at(cache()), 0, 0, None) == 1


def test_rope_table_values():
    for d, theta in ((16, 10000.0), (128, 500000.0), (64, 2.0)):
        f, mag = fmad.rope_table(d, theta)
        want = [theta ** (-2.0 * i / d) / (2 * math.pi) for i in range(d // 2)]
        # powers and the division in double: a few units in the 53rd bit; then rounded to whole 2^-64 turns
        assert mag == 1.0 and all(abs(int(a) / 2.0 ** 64 - b) <= b * 2.0 ** -50 + 2.0 ** -65 for a, b in zip(f, want))
    base = fmad.rope_table(64, 10000.0)[0].astype(np.float64)
    assert np.allclose(fmad.rope_table(64, 10000.0, fmad.ROPE_LINEAR, 8.0)[0] * 8.0, base, rtol=2.0 ** -48, atol=4.5)   # each whole number is half a unit off
    grown = fmad.rope_table(64, 10000.0, fmad.ROPE_BASE, 8.0)[0].astype(np.float64)
    # the fastest pair is unchanged, the slowest turns exactly `factor` times slower
    assert grown[0] == base[0] and abs(base[-1] / grown[-1] / 8.0 - 1) < 2.0 ** -44
    parts, mag = fmad.rope_table(64, 10000.0, fmad.ROPE_BY_PARTS, 8.0, 4096.0, 32.0, 1.0)
    ratio = base / parts.astype(np.float64)
    turns = base / 2.0 ** 64 * 4096.0
    assert abs(mag - (0.1 * math.log(8) + 1)) < 1e-6
    assert np.allclose(ratio[turns > 32 * 1.4], 1) and np.allclose(ratio[turns < 1 / 1.4], 8) and (np.diff(ratio) > -1e-9).all()
    # factor 1 mixes equal frequencies: three roundings of doubles, then whole numbers
    same = fmad.rope_table(64, 10000.0, fmad.ROPE_BY_PARTS, 1.0, 4096.0)[0].astype(np.float64)
    assert np.allclose(same, base, rtol=2.0 ** -51, atol=1.0)


@pytest.mark.parametrize("args,status", [
    ((8,), 2), ((24,), 2), ((272,), 2), ((64, 1.0), 1), ((64, math.nan), 1), ((64, math.inf), 1), ((64, 1e4, 4), 1),
    ((64, 1e4, -1), 1), ((64, 1e4, 1, 0.5), 1), ((64, 1e4, 2, math.inf), 1), ((64, 1e4, 3, 8.0, 0.0), 1),
    ((64, 1e4, 3, 8.0, 4096.0, 1.0, 1.0), 1), ((64, 1e4, 3, 8.0, 4096.0, 32.0, 0.0), 1),
])
def test_rope_table_refuses(args, status):
    with pytest.raises(fmad.FmError) as e:
        fmad.rope_table(*args)
    assert e.value.status == status
