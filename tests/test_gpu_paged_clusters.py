"""Splits of a chunk's keys that meet in their cluster (fm_shared_attention without sharing, fm_sink_attention) against splits
that meet in the workspace (fm_paged_attention): the same sums in the same order, so the same bits; and first tokens with
every number of splits against their definition (tolerance: as in test_gpu_sink_attention.py)."""
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import Cache, batch
from test_gpu_sink_attention import attend, check

pytestmark = pytest.mark.gpu

# lengths, new tokens, H, Hkv: one row tile and two, groups of one to eight heads, rows that fill no tile, rows without keys
SHAPES = [([700, 300], [300, 70], 8, 1), ([6000], [100], 16, 2), ([5000, 4000, 3000, 200], [60, 33, 60, 1], 10, 2),
          ([3000, 2500], [30, 17], 8, 1), ([16000, 9000], [64, 33], 8, 1), ([2000, 1900, 300, 40, 5, 0], [20, 19, 18, 20, 5, 0], 6, 6),
          ([9000], [17], 7, 1), ([4000] * 5, [128] * 5, 1, 1), ([12000, 20], [40, 30], 5, 1), ([2600, 2600], [260, 257], 3, 3),
          ([1500] * 3, [200, 199, 1], 16, 2), ([1200], [100], 16, 2), ([1500, 700], [30, 17], 8, 1), ([2000], [17], 7, 1),
          ([900, 1000], [64, 3], 8, 1)]


def no_groups():
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    return fmad.KvGroups(none, none[:0], 0, 0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_the_same_bits(shape, Dh, fp8):
    require_gpu()
    lens, new, H, Hkv = SHAPES[shape]
    c = Cache(lens, 32, Hkv, Dh, fp8, heads_first=True, seed=shape)
    b, groups = batch(c, new, True, 1, 2), no_groups()
    q = torch.randn((b.tokens, H, Dh), generator=torch.Generator().manual_seed(shape)).mul_(1.5).to(torch.bfloat16).cuda()
    need = fmad.paged_attention_workspace_size(c.handle, b, H)
    less = fmad.shared_attention_workspace_size(c.handle, b, groups, H)
    assert less in (0, need)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for causal in (True, False):
        a, e = (torch.full((b.tokens, H, Dh), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        fmad.paged_attention(c.handle, 0, b, q, e, ws, causal=causal)
        fmad.shared_attention(c.handle, 0, b, groups, q, a, ws[:less] if less else None, causal=causal)
        torch.cuda.synchronize()
        assert torch.equal(a, e)
        # a row of NaN, a value of NaN
        q[1, 0, 3] = float("nan")
        row = int(c.rows[0])
        page = c.table[row, (lens[0] - 1) // 32].long()
        bits = c.v.view(torch.uint8) if fp8 else c.v.view(torch.int16)
        saved = bits[:, page].clone()
        bits[:, page, (lens[0] - 1) % 32, 0, 5] = 0x7F if fp8 else 0x7FC0
        fmad.paged_attention(c.handle, 0, b, q, e, ws, causal=causal)
        fmad.shared_attention(c.handle, 0, b, groups, q, a, ws[:less] if less else None, causal=causal)
        torch.cuda.synchronize()
        assert bool(a[1, 0].isnan().all()) and torch.equal(a.view(torch.int16), e.view(torch.int16))
        bits[:, page] = saved
        q[1, 0, 3] = 0.5
    assert fmad.standalone_status() == 0


def test_the_shapes_are_divided():
    """Most of the shapes above have splits, and most of these meet in clusters."""
    require_gpu()
    divided = met = 0
    for lens, new, H, Hkv in SHAPES:
        c = Cache(lens, 32, Hkv, 64, seed=1)
        b = batch(c, new)
        need = fmad.paged_attention_workspace_size(c.handle, b, H)
        divided += need > 0
        met += need > 0 and fmad.shared_attention_workspace_size(c.handle, b, no_groups(), H) == 0
    assert divided >= 7 and met >= 5


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_first_tokens(shape, Dh, fp8):
    """Windows of 2 to 9 tiles of keys: every number of splits."""
    require_gpu()
    lens, new, H, Hkv = SHAPES[shape]
    c = Cache(lens, 64, Hkv, Dh, fp8, seed=shape)
    for window, sinks in ((200, 30), (500, 130), (900, 5)):
        q, out, b = attend(c, new, H, window, sinks, lead=1, trail=1)
        check(c, new, q, out, b, window, sinks)


def test_two_streams_at_once():
    require_gpu()
    c = Cache([6000, 5000], 64, 2, 128, seed=3)
    b, groups = batch(c, [100, 60]), no_groups()
    q = torch.randn((160, 16, 128), device="cuda").to(torch.bfloat16)
    want = torch.empty_like(q)
    ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, 16), dtype=torch.uint8, device="cuda")
    fmad.paged_attention(c.handle, 0, b, q, want, ws)
    need = fmad.shared_attention_workspace_size(c.handle, b, groups, 16)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[torch.empty_like(q) for _ in range(6)] for _ in streams]
    mine = [torch.empty(max(need, 1), dtype=torch.uint8, device="cuda") for _ in streams]
    for i in range(6):
        for s, o, w in zip(streams, outs, mine):
            fmad.shared_attention(c.handle, 0, b, groups, q, o[i], w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(want, x) for o in outs for x in o) and fmad.standalone_status() == 0
