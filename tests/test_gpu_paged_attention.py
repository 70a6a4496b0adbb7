"""Attention of a chunk over a paged cache against its definition in 64 bits.

Tolerance, element by element, with S = sum_j p_j |v_j| from the reference: the output's rounding to bf16 is at most
2^-8 |o| (half a step), the probabilities' rounding 2^-8 S (bf16) or 2^-11 S (f16, E4M3 cache). The scores are fp32 sums
of at most 128 exact products: their error is below 128 * 2^-23 * sum |q k| * scale < 2^-10 for these inputs (sum |q k|
scale < 60), so p is off by at most 2^-10 relative; the approximate 2^x, the fp32 sums and the splits' join add less
than 2^-12. Together 2^-8 |o| + (2^-8 or 2^-11, + 2^-9) S."""
import numpy as np
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import Cache, attention_ref, batch

pytestmark = pytest.mark.gpu


def attend(c, new, H, causal=True, window=0, scale=None, seq=True, lead=0, trail=0, layer=0, seed=5, max_len=None,
           q_pad=0):
    """(q, out, batch): out starts at 7 everywhere, rows of no entry must stay so."""
    b = batch(c, new, seq, lead, trail, max_len=max_len)
    Dh = c.k.shape[-1]
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn((b.tokens, H + q_pad, Dh), generator=g).mul_(1.5).to(torch.bfloat16).cuda()
    q = wide[:, :H]
    out = torch.full((b.tokens, H + q_pad, Dh), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, H), dtype=torch.uint8, device="cuda")
    fmad.paged_attention(c.handle, layer, b, q, out[:, :H], ws, scale, causal, window)
    torch.cuda.synchronize()
    assert fmad.standalone_status() == 0
    assert (out[:, H:] == 7).all()
    return q, out[:, :H], b


def check(c, new, q, out, b, causal, window, scale, layer=0):
    start = b.start.cpu().numpy()
    assert (out[:start[0]] == 7).all() and (out[start[-1]:] == 7).all()
    for i, n in enumerate(new):
        if n == 0:
            continue
        rows = slice(int(start[i]), int(start[i + 1]))
        ref, size = attention_ref(c, i, q[rows], scale, causal, window, layer)
        tol = ref.abs() * 2.0 ** -8 + size * ((2.0 ** -11 if c.fp8 else 2.0 ** -8) + 2.0 ** -9)
        err = (out[rows].double() - ref).abs()
        assert bool((err <= tol).all()), (i, n, c.lens_host[i], float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("lens,new,page", [
    ([1], [1], 16), ([17], [1], 16), ([127, 128, 129, 255, 256, 257], [1] * 6, 32), ([789], [1], 16),
    ([300, 5, 64], [7, 5, 1], 64), ([130, 513], [128, 129], 128), ([700], [300], 256), ([40], [40], 16),
    ([2000, 3], [33, 2], 16),
])
def test_lengths(Dh, fp8, lens, new, page):
    require_gpu()
    c = Cache(lens, page, 2, Dh, fp8, seed=len(lens) + page)
    q, out, b = attend(c, new, 8)
    check(c, new, q, out, b, True, 0, Dh ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 1), (6, 2), (5, 5), (14, 2), (40, 1)])
def test_heads(H, Hkv, fp8):
    require_gpu()
    c = Cache([333, 90], 32, Hkv, 128, fp8, heads_first=Hkv % 2 == 0, seed=H)
    new = [61, 1]
    q, out, b = attend(c, new, H, lead=3, trail=2, q_pad=1)
    check(c, new, q, out, b, True, 0, 128 ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 100), (True, 128), (True, 5000), (False, 0), (False, 50)])
def test_masks(causal, window, fp8):
    require_gpu()
    c = Cache([777, 140, 2, 1300], 16, 2, 64, fp8, seed=window)
    new = [300, 140, 1, 5]
    q, out, b = attend(c, new, 6, causal, window, scale=0.2)
    check(c, new, q, out, b, causal, window, 0.2)


def test_empty_sequences_and_rows():
    """Length 0, no new tokens, more new tokens than the length (negative positions see nothing), no entries."""
    require_gpu()
    c = Cache([0, 50, 20, 0], 16, 2, 128, seed=9)
    new = [3, 0, 30, 0]
    for causal in (True, False):
        q, out, b = attend(c, new, 4, causal, trail=1)
        assert (out[:3] == 0).all() and (out[3:13] == 0).all() and (out[33:] == 7).all()
        check(c, new, q, out, b, causal, 0, 128 ** -0.5)
    none = fmad.KvBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), 0, 0, 0)
    fmad.paged_attention(c.handle, 0, none, q[:0], out[:0])


@pytest.mark.parametrize("fp8", [False, True])
def test_long_key_axis_is_split(fp8):
    require_gpu()
    c = Cache([20011, 4000, 1], 64, 1, 128, fp8, heads_first=True, seed=2)
    new = [1, 16, 1]
    b = batch(c, new)
    assert fmad.paged_attention_workspace_size(c.handle, b, 8) > 0
    q, out, b = attend(c, new, 8, lead=1, trail=1)
    check(c, new, q, out, b, True, 0, 128 ** -0.5)
    # a length bound that is too small costs speed, not results
    q, out, b = attend(c, new, 8, max_len=700)
    check(c, new, q, out, b, True, 0, 128 ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
def test_splits_of_a_wide_chunk(fp8):
    require_gpu()
    c = Cache([6000], 32, 1, 128, fp8, seed=3)
    q, out, b = attend(c, [50], 8, False)
    check(c, [50], q, out, b, False, 0, 128 ** -0.5)
    c = Cache([3000], 32, 2, 64, fp8, seed=4)
    q, out, b = attend(c, [200], 8, True, 300)
    check(c, [200], q, out, b, True, 300, 64 ** -0.5)


def test_large_scores_move_the_reference_maximum():
    """Scores that grow along the keys by far more than 2^8 (every tile rescales) and that are hugely negative."""
    require_gpu()
    c = Cache([1000], 16, 1, 128, seed=4, poison=False)
    ramp = torch.linspace(-4, 4, 1000)
    for i in range(1000):
        pg = int(c.table[c.rows[0], i // 16])
        c.k[0, pg, i % 16, 0] = 0
        c.k[0, pg, i % 16, 0, 0] = float(ramp[i])
    b = batch(c, [4])
    for sign in (1.0, -1.0):
        q = torch.zeros((4, 2, 128), dtype=torch.bfloat16, device="cuda")
        q[:, :, 0] = 64.0 * sign
        out = torch.empty_like(q)
        ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, 2), dtype=torch.uint8, device="cuda")
        fmad.paged_attention(c.handle, 0, b, q, out, ws, scale=1.0)
        # one product per score: exact; scores up to 256 in fp32 times log2(e): off by 2^-15, p by 2^-15
        ref, size = attention_ref(c, 0, q, 1.0, True, 0)
        assert bool(((out.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + size * (2.0 ** -8 + 2.0 ** -9)).all())


@pytest.mark.parametrize("exponent", [-60, -20, 0, 40])
def test_queries_of_any_size_with_an_8_bit_cache(exponent):
    """Rows of q are scaled to f16 exactly: tiny and huge queries with the scale that brings the scores back."""
    require_gpu()
    c = Cache([200], 16, 1, 128, True, seed=6)
    g = torch.Generator().manual_seed(1)
    q = (torch.randn((3, 2, 128), generator=g) * 2.0 ** exponent).to(torch.bfloat16).cuda()
    q[1] = 0
    out = torch.empty_like(q)
    b = batch(c, [3])
    scale = 128 ** -0.5 * 2.0 ** -exponent
    ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, 2), dtype=torch.uint8, device="cuda")
    fmad.paged_attention(c.handle, 0, b, q, out, ws, scale=scale)
    ref, size = attention_ref(c, 0, q, scale, True, 0)
    assert bool(((out.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + size * (2.0 ** -11 + 2.0 ** -9)).all())


def test_layers_and_sequence_order():
    require_gpu()
    c = Cache([60, 70], 32, 2, 64, layers=3, seed=8)
    for layer in (0, 2):
        q, out, b = attend(c, [5, 6], 4, layer=layer)
        check(c, [5, 6], q, out, b, True, 0, 0.125, layer)
    # no seq: entry i is sequence i
    c = Cache([60, 70], 32, 2, 64, seed=8, rows=[0, 1])
    q, out, b = attend(c, [5, 6], 4, seq=False)
    check(c, [5, 6], q, out, b, True, 0, 0.125)
    # one sequence named by two entries
    c.rows, c.lens_host = [1, 1], [70, 70]
    q, out, b = attend(c, [5, 6], 4)
    check(c, [5, 6], q, out, b, True, 0, 0.125)


def test_graph_replay_other_stream_and_repeatability():
    require_gpu()
    c = Cache([5000, 300], 64, 2, 128, True, seed=11)
    b = batch(c, [2, 9])
    q = torch.randn((11, 8, 128), device="cuda").to(torch.bfloat16)
    ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, 8), dtype=torch.uint8, device="cuda")
    eager, replay = torch.empty_like(q), torch.zeros_like(q)
    fmad.paged_attention(c.handle, 0, b, q, eager, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fmad.paged_attention(c.handle, 0, b, q, replay, ws)
    for _ in range(3):
        replay.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, replay)
    other = torch.empty_like(q)
    fmad.paged_attention(c.handle, 0, b, q, other, ws, stream=s)
    s.synchronize()
    assert torch.equal(eager, other)
    # the graph reads the lengths at replay
    c.lens[c.rows[0]] = 4000
    c.lens_host[0] = 4000
    g.replay()
    torch.cuda.synchronize()
    check(c, [2, 9], q, replay, b, True, 0, 128 ** -0.5)


def test_device_side_faults_are_reported():
    """A token without a page, an entry outside the packed rows, an entry beyond max_tokens: bit 2, no fault."""
    require_gpu()
    c = Cache([100, 40], 16, 1, 64, seed=12, poison=False)
    q = torch.randn((6, 2, 64), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def run(b):
        fmad.paged_attention(c.handle, 0, b, q, out, ws)
        return fmad.standalone_status()

    assert run(batch(c, [3, 3])) == 0
    assert run(batch(c, [3, 3], max_tokens=2)) == 2
    saved = c.table.clone()
    c.table[c.rows[0], 2] = -1
    assert run(batch(c, [3, 3])) == 2
    c.table[c.rows[0], 2] = 10 ** 6
    assert run(batch(c, [3, 3])) == 2
    c.table.copy_(saved)
    for start in ([0, 3, 7], [-1, 3, 6], [3, 2, 6]):
        b = fmad.KvBatch(torch.tensor(start, dtype=torch.int32, device="cuda"), 6, 6, 100,
                         torch.tensor(np.asarray(c.rows), dtype=torch.int32, device="cuda"))
        assert run(b) == 2
    for seq in ([99, 0], [-1, 0]):
        b = fmad.KvBatch(torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda"), 6, 3, 100,
                         torch.tensor(seq, dtype=torch.int32, device="cuda"))
        assert run(b) == 2
    c.lens[c.rows[0]] = 10 ** 9
    assert run(batch(c, [3, 3])) == 2
    c.lens[c.rows[0]] = 100
    assert run(batch(c, [3, 3])) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_a_loose_bound_on_the_new_tokens(fp8):
    """A bound above the packed rows gives the same variant, workspace and results."""
    require_gpu()
    c = Cache([700, 30], 16, 2, 128, fp8, seed=4)
    ids = torch.tensor(np.asarray(c.rows), dtype=torch.int32, device="cuda")
    for new in ([1, 1], [60, 2]):
        start = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda")
        q = torch.randn((sum(new), 4, 128), device="cuda").to(torch.bfloat16)
        outs = []
        for bound in (sum(new), 1 << 28):
            b = fmad.KvBatch(start, sum(new), bound, 700, ids)
            ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, 4), dtype=torch.uint8, device="cuda")
            outs.append(torch.full_like(q, 7.0))
            fmad.paged_attention(c.handle, 0, b, q, outs[-1], ws)
        assert fmad.standalone_status() == 0 and torch.equal(*outs)
        check(c, new, q, outs[0], batch(c, new), True, 0, 128 ** -0.5)


def test_the_binding_refuses():
    require_gpu()
    c = Cache([20], 16, 2, 64, seed=1, poison=False)
    b = batch(c, [4])
    q = torch.zeros((4, 4, 64), device="cuda", dtype=torch.bfloat16)
    good = dict(q=q, out=torch.empty_like(q))
    fmad.paged_attention(c.handle, 0, b, **good)
    for bad in (dict(q=q[0]), dict(q=q[:3]), dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :, ::2]), dict(q=q[:, :3]),
                dict(out=q[:, :2]), dict(out=torch.empty((4, 64, 4), device="cuda", dtype=torch.bfloat16).transpose(1, 2)),
                dict(workspace=torch.empty(64)), dict(scale=0.0), dict(window=-1), dict(layer=1)):
        with pytest.raises(fmad.FmError):
            fmad.paged_attention(c.handle, bad.pop("layer", 0), b, **{**good, **bad})


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 200)])
def test_whole_prefills(causal, window, Dh, fp8):
    """Most of each sequence is new: ragged entries of many row blocks, some empty, some with a short history."""
    require_gpu()
    lens = [900, 1, 300, 17, 513, 256, 700]
    new = [900, 1, 0, 17, 513, 200, 690]
    c = Cache(lens, 32, 2, Dh, fp8, seed=9)
    q, out, b = attend(c, new, 8, causal, window, lead=3, trail=2)
    check(c, new, q, out, b, causal, window, Dh ** -0.5)
