"""Attention of forks right behind kernels that write everything it reads: its second kernel starts beside its first one and
sees these writes through a word of the workspace, which may hold anything before the call and holds nothing after it."""
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import batch
from test_gpu_shared_attention import Forks, check

pytestmark = pytest.mark.gpu


def setup(most, fp8=False, seed=21):
    c = Forks([(8100, [40] * 90), (3000, [17] * 20)], 16, 2, 64, fp8, seed=seed)
    new = [most] * 110
    b, groups = batch(c, new), c.groups()
    need = fmad.shared_attention_workspace_size(c.handle, b, groups, 8)
    assert need > 16
    return c, new, b, groups, need


@pytest.mark.parametrize("most", [1, 5])
def test_the_word_may_hold_anything_before_and_nothing_after(most):
    require_gpu()
    c, new, b, groups, need = setup(most)
    q = torch.randn((b.tokens, 8, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    outs = []
    for fill in (0, 0xFF, 0x5B):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            outs.append(torch.full_like(q, 7.0))
            fmad.shared_attention(c.handle, 0, b, groups, q, outs[-1], ws)
        torch.cuda.synchronize()
        words = ws.view(torch.int64)
        assert not (words == 0x5B1D93E6C7F0A42D).any()
    assert all(torch.equal(outs[0], x) for x in outs) and fmad.standalone_status() == 0
    check(c, new, q, outs[0], b)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_every_input_is_written_right_before_the_call(captured, fp8):
    """Starts, sequences, lengths, table, groups, queries, keys and values alternate between two batches, written by kernels
    of the same stream without a wait between them."""
    require_gpu()
    parts = [setup(2, fp8, seed) for seed in (31, 32)]
    (c, new, b, groups, need), other = parts[0], parts[1][0]
    assert other.k.shape == c.k.shape and other.table.shape == c.table.shape
    live = [c.k, c.v, c.table, c.lens, b.start, b.seq, groups.first, groups.shared]
    sides = []
    for x, _, bb, gg, _ in parts:
        q = torch.randn((b.tokens, 8, 64), generator=torch.Generator().manual_seed(x.table.sum().item())).to(torch.bfloat16).cuda()
        sides.append([t.clone() for t in (x.k, x.v, x.table, x.lens, bb.start, bb.seq, gg.first, gg.shared)] + [q])
    if fp8:   # one cache, so one pair of scales
        other.k_scale.copy_(c.k_scale), other.v_scale.copy_(c.v_scale)
    q = torch.empty_like(sides[0][-1])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(8)]

    def steps():
        for i, out in enumerate(outs):
            for dst, src in zip(live + [q], sides[i % 2]):
                (dst.view(torch.uint8) if dst.dtype == torch.float8_e4m3fn else dst).copy_(
                    src.view(torch.uint8) if src.dtype == torch.float8_e4m3fn else src)
            fmad.shared_attention(c.handle, 0, b, groups, q, out, ws)

    if captured:
        steps()
        torch.cuda.synchronize()
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            steps()
        for out in outs:
            out.zero_()
        g.replay()
        g.replay()
    else:
        steps()
    torch.cuda.synchronize()
    assert fmad.standalone_status() == 0
    for i, out in enumerate(outs[:2]):
        x, n, bb, _, _ = parts[i]
        for t, src in zip((x.k, x.v, x.table, x.lens), sides[i]):
            (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).copy_(src.view(torch.uint8) if src.dtype == torch.float8_e4m3fn else src)
        check(x, n, sides[i][-1], out, bb)
    assert all(torch.equal(outs[i % 2], out) for i, out in enumerate(outs))
