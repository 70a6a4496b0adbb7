"""Attention with a window and first tokens that stay visible, against its definition in 64 bits.

Tolerance: the plain attention's (its tests derive it); the mask is the only difference: 2^-8 |o| for the output's rounding,
(2^-8 or, with an E4M3 cache, 2^-11, + 2^-9) sum_j p_j |v_j| for probabilities and scores."""
import math

import numpy as np
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import Cache, batch

pytestmark = pytest.mark.gpu


def reference(c, i, q, scale, causal, window, sinks, layer=0):
    """(out, sum_j p_j |v_j|) of entry i's q [new][H][Dh] in float64."""
    k, v = c.dense(i, layer)
    n, H, Dh = q.shape
    ln, G = c.lens_host[i], H // k.shape[1]
    pos = torch.arange(ln - n, ln, device=q.device)[:, None]
    key = torch.arange(ln, device=q.device)[None]
    ok = (pos >= 0) & (key >= 0)
    if causal:
        ok = ok & (key <= pos)
    if window:
        ok = ok & ((key > pos - window) | (key < sinks))
    out, size = torch.zeros(q.shape, dtype=torch.float64, device=q.device), torch.zeros_like(q, dtype=torch.float64)
    for h in range(H):
        s = ((q[:, h].double() @ k[:, h // G].T) * scale).masked_fill(~ok, -math.inf)
        p = torch.nan_to_num(torch.softmax(s, -1))
        out[:, h], size[:, h] = p @ v[:, h // G], p @ v[:, h // G].abs()
    return out, size


def attend(c, new, H, window, sinks, causal=True, scale=None, lead=0, trail=0, layer=0, seed=5, max_len=None, q_pad=0, ws=None):
    b = batch(c, new, True, lead, trail, max_len=max_len)
    Dh = c.k.shape[-1]
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn((b.tokens, H + q_pad, Dh), generator=g).mul_(1.5).to(torch.bfloat16).cuda()
    q = wide[:, :H]
    out = torch.full((b.tokens, H + q_pad, Dh), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, H), dtype=torch.uint8, device="cuda")
    fmad.sink_attention(c.handle, layer, b, q, out[:, :H], ws, scale, causal, window, sinks)
    torch.cuda.synchronize()
    assert fmad.standalone_status() == 0
    assert (out[:, H:] == 7).all()
    return q, out[:, :H], b


def check(c, new, q, out, b, window, sinks, causal=True, scale=None, layer=0):
    scale = c.k.shape[-1] ** -0.5 if scale is None else scale
    start = b.start.cpu().numpy()
    assert (out[:start[0]] == 7).all() and (out[start[-1]:] == 7).all()
    for i, n in enumerate(new):
        rows = slice(int(start[i]), int(start[i + 1]))
        ref, size = reference(c, i, q[rows], scale, causal, window, sinks, layer)
        tol = ref.abs() * 2.0 ** -8 + size * ((2.0 ** -11 if c.fp8 else 2.0 ** -8) + 2.0 ** -9)
        err = (out[rows].double() - ref).abs()
        assert bool((err <= tol).all()), (i, n, c.lens_host[i], float((err - tol).max()), float(err.max()))


# windows and first tokens that meet, touch, end inside of tiles and pages, or lie far apart
MASKS = [(1, 1), (64, 64), (100, 4), (128, 128), (129, 127), (200, 300), (37, 1000), (5000, 5)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("window,sinks", MASKS)
def test_single_tokens(window, sinks, Dh, fp8):
    require_gpu()
    lens = [1, 17, 64, 65, 127, 128, 129, 260, 400, 789, 1500]
    c = Cache(lens, 16, 2, Dh, fp8, seed=window + sinks)
    new = [1] * len(lens)
    q, out, b = attend(c, new, 8, window, sinks)
    check(c, new, q, out, b, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("window,sinks", MASKS)
def test_few_rows_and_chunks(window, sinks, Dh, fp8):
    """Up to 16 stacked rows, up to 128, row blocks of 256 of several entries, windows that begin inside of a chunk."""
    require_gpu()
    c = Cache([900, 40, 300, 3], 32, 2, Dh, fp8, heads_first=True, seed=window)
    for new, H in (([4, 2, 1, 3], 6), ([30, 17, 1, 2], 6), ([333, 40, 300, 1], 10)):
        q, out, b = attend(c, new, H, window, sinks, lead=2, trail=1)
        check(c, new, q, out, b, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(50, 7), (128, 200), (1, 64)])
def test_without_causality_and_with_other_scales(window, sinks, fp8):
    require_gpu()
    c = Cache([777, 140, 2, 1300], 16, 2, 64, fp8, seed=window)
    for new in ([300, 140, 1, 5], [1, 1, 1, 1]):
        q, out, b = attend(c, new, 6, window, sinks, causal=False, scale=0.2)
        check(c, new, q, out, b, window, sinks, False, 0.2)


def test_empty_sequences_and_rows():
    require_gpu()
    c = Cache([0, 50, 20, 0], 16, 2, 128, seed=9)
    new = [3, 0, 30, 0]
    for causal in (True, False):
        q, out, b = attend(c, new, 4, 5, 3, causal, trail=1)
        assert (out[:3] == 0).all() and (out[3:13] == 0).all() and (out[33:] == 7).all()
        check(c, new, q, out, b, 5, 3, causal)
    none = fmad.KvBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), 0, 0, 0)
    fmad.sink_attention(c.handle, 0, none, q[:0], out[:0], window=4, sinks=2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,H", [([1, 16, 1], 8), ([2, 1, 1], 8), ([60, 3, 1], 8), ([300, 9, 1], 8)])
def test_long_windows_are_split(new, H, fp8):
    """Clusters and workspaces that divide both stretches; a bound on the lengths that is too small."""
    require_gpu()
    c = Cache([20011, 4000, 1], 64, 1, 128, fp8, heads_first=True, seed=2)
    for window, sinks in ((9000, 700), (300, 9000), (17, 20000)):
        q, out, b = attend(c, new, H, window, sinks, lead=1, trail=1)
        check(c, new, q, out, b, window, sinks)
    q, out, b = attend(c, new, H, 9000, 700, max_len=700)
    check(c, new, q, out, b, 9000, 700)


@pytest.mark.parametrize("new", [[1, 2], [60, 2], [700, 30]])
def test_without_a_window_or_first_tokens_it_is_paged_attention(new):
    require_gpu()
    c = Cache([2000, 40], 16, 2, 64, seed=4)
    b = batch(c, new)
    q = torch.randn((b.tokens, 8, 64), device="cuda").to(torch.bfloat16)
    ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, 8), dtype=torch.uint8, device="cuda")
    for window, sinks in ((0, 0), (0, 9), (300, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)):
        a, e = torch.empty_like(q), torch.empty_like(q)
        fmad.sink_attention(c.handle, 0, b, q, a, ws, window=window, sinks=sinks)
        fmad.paged_attention(c.handle, 0, b, q, e, ws, window=window if sinks == 0 else 0)
        if window == 2 ** 31 - 1 or sinks == 2 ** 31 - 1:   # everything is visible, by another kernel
            assert bool(((a.float() - e.float()).abs() <= 2.0 ** -6 * e.float().abs().max()).all())
        else:
            assert torch.equal(a, e)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,H", [([1, 1], 8), ([9, 5], 8), ([260, 40], 8)])
def test_hidden_pages_are_not_read(new, H, fp8):
    """Pages between the two stretches may be gone or hold NaN, at no cost to the result."""
    require_gpu()
    c = Cache([3000, 2500], 16, 1, 128, fp8, seed=7)
    window, sinks = 200, 40
    q, clean, b = attend(c, new, H, window, sinks)
    for i, n in enumerate(new):
        first = (c.lens_host[i] - n - window + 1) // 128 * 8   # the page where the window's first tile begins
        row = c.rows[i]
        gone = c.table[row, 8:first].clone()
        for t in (c.k, c.v):
            (t.view(torch.uint8) if fp8 else t.view(torch.int16))[:, gone.long()] = 0x7F if fp8 else 0x7FC0
        c.table[row, 8:first] = -1
    _, out, _ = attend(c, new, H, window, sinks)
    assert torch.equal(clean, out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,new,H", [([1500, 90], [1, 2], 8), ([12000, 700], [50, 3], 8), ([4000, 300], [400, 300], 8)])
def test_a_nan_query_row_stays_alone(lens, new, H, fp8):
    require_gpu()
    c = Cache(lens, 16, 1, 64, fp8, seed=H)
    b = batch(c, new)
    ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, H), dtype=torch.uint8, device="cuda")
    q = torch.randn((b.tokens, H, 64), device="cuda").to(torch.bfloat16)
    clean, out = torch.empty_like(q), torch.empty_like(q)
    fmad.sink_attention(c.handle, 0, b, q, clean, ws, window=333, sinks=70)
    token, head = b.tokens - 1, H - 1
    q[token, head, 5] = float("nan")
    fmad.sink_attention(c.handle, 0, b, q, out, ws, window=333, sinks=70)
    assert fmad.standalone_status() == 0 and out[token, head].isnan().all()
    out[token, head] = clean[token, head]
    assert torch.equal(out, clean)


def test_layers_strides_and_order():
    require_gpu()
    c = Cache([260, 370], 32, 2, 64, layers=3, seed=8)
    for layer in (0, 2):
        q, out, b = attend(c, [5, 6], 4, 50, 20, layer=layer, q_pad=1)
        check(c, [5, 6], q, out, b, 50, 20, layer=layer)


def test_graph_replay_other_stream_and_lengths():
    require_gpu()
    c = Cache([5000, 300], 64, 2, 128, True, seed=11)
    b = batch(c, [2, 9])
    q = torch.randn((11, 8, 128), device="cuda").to(torch.bfloat16)
    ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, 8), dtype=torch.uint8, device="cuda")
    eager, replay = torch.empty_like(q), torch.zeros_like(q)
    kw = dict(window=900, sinks=130)
    fmad.sink_attention(c.handle, 0, b, q, eager, ws, **kw)
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fmad.sink_attention(c.handle, 0, b, q, replay, ws, **kw)
    for _ in range(3):
        replay.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, replay)
    other = torch.empty_like(q)
    fmad.sink_attention(c.handle, 0, b, q, other, ws, stream=s, **kw)
    s.synchronize()
    assert torch.equal(eager, other)
    c.lens[c.rows[0]] = 4000
    c.lens_host[0] = 4000
    g.replay()
    torch.cuda.synchronize()
    check(c, [2, 9], q, replay, b, 900, 130)


def test_device_side_faults_are_reported():
    require_gpu()
    c = Cache([1000, 400], 16, 1, 64, seed=12, poison=False)
    q = torch.randn((6, 2, 64), device="cuda").to(torch.bfloat16)
    out, ws = torch.empty_like(q), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def run(b):
        fmad.sink_attention(c.handle, 0, b, q, out, ws, window=100, sinks=20)
        return fmad.standalone_status()

    assert run(batch(c, [3, 3])) == 0
    assert run(batch(c, [3, 3], max_tokens=2)) == 2
    for place in (0, 1, 60):   # a page of the first tokens, of the window
        for page in (-1, 10 ** 6):
            saved = int(c.table[c.rows[0], place])
            c.table[c.rows[0], place] = page
            assert run(batch(c, [3, 3])) == 2
            c.table[c.rows[0], place] = saved
    for start in ([0, 3, 7], [-1, 3, 6], [3, 2, 6]):
        b = fmad.KvBatch(torch.tensor(start, dtype=torch.int32, device="cuda"), 6, 6, 100,
                         torch.tensor(np.asarray(c.rows), dtype=torch.int32, device="cuda"))
        assert run(b) == 2
    c.lens[c.rows[0]] = 10 ** 9
    assert run(batch(c, [3, 3])) == 2
    c.lens[c.rows[0]] = 1000
    assert run(batch(c, [3, 3])) == 0


def test_the_binding_refuses():
    require_gpu()
    c = Cache([20], 16, 2, 64, seed=1, poison=False)
    b = batch(c, [4])
    q = torch.zeros((4, 4, 64), device="cuda", dtype=torch.bfloat16)
    good = dict(q=q, out=torch.empty_like(q), window=3, sinks=2)
    fmad.sink_attention(c.handle, 0, b, **good)
    for bad in (dict(q=q[0]), dict(q=q[:3]), dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :, ::2]), dict(q=q[:, :3]),
                dict(out=q[:, :2]), dict(workspace=torch.empty(64)), dict(scale=0.0), dict(window=-1), dict(sinks=-1),
                dict(layer=1)):
        with pytest.raises(fmad.FmError):
            fmad.sink_attention(c.handle, bad.pop("layer", 0), b, **{**good, **bad})
