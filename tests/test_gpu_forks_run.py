"""Candidate plans of one observation, as they run: the observation's chunks go through layers with normalised heads (local
layers with a window and visible first tokens, global ones), the sequence is forked, every fork adds its tokens, and a policy
reads the chosen fork's prefix. Every stage is held to its definition on the inputs that it got."""
import subprocess
import sys

import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import Cache, attention_ref, batch
from test_gpu_prefix_pages import i32, policy
from test_gpu_sink_attention import reference as sink_ref

pytestmark = pytest.mark.gpu

WINDOW, SINKS, EPS = 600, 48, 1e-6


@pytest.mark.parametrize("fp8", [False, True])
def test_candidates_of_one_observation(fp8):
    require_gpu()
    H, Hkv, Dh, L, page, n, observed = 8, 1, 128, 2, 64, 120, 8007
    g = torch.Generator().manual_seed(0)
    c = Cache([], page, Hkv, Dh, fp8, L, seqs=n, spare_pages=observed // page + 3 + 2 * n, poison=False)
    c.table = torch.full((n, observed // page + 4), -1, dtype=torch.int32, device="cuda")
    c.handle = fmad.KvCache(c.k, c.v, c.table, c.lens, c.refs, c.k_scale, c.v_scale)
    rope, status = fmad.Rope(Dh, theta=10000.0), i32([0, 0])
    work = torch.empty(fmad.kv_workspace_size(c.handle, n), dtype=torch.uint8, device="cuda")
    gains = [(torch.randn(Dh, generator=g) * 0.2 + 1).cuda() for _ in range(2)]

    def layers(seq, new, groups=None, checked=None):
        fmad.kv_reserve(c.handle, i32(seq), i32(new), status, work)
        c.rows, c.lens_host = list(seq), [int(x) for x in c.lens[torch.tensor(seq)]]
        b, T = batch(c, new), int(sum(new))
        start = b.start.tolist()
        if groups is None:
            need = fmad.paged_attention_workspace_size(c.handle, b, H)
        else:
            need = fmad.shared_attention_workspace_size(c.handle, b, groups, H)
            assert need > 0   # the prefix is computed by itself
            need = max(need, fmad.paged_attention_workspace_size(c.handle, b, H))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        qkv = torch.randn((T, H + 2 * Hkv, Dh), generator=g).to(torch.bfloat16).cuda()
        for l in range(L):
            q, out = (torch.empty((T, H, Dh), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            fmad.norm_rope_append(c.handle, l, b, rope, qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], q, *gains, EPS)
            if l == 0:
                fmad.sink_attention(c.handle, l, b, q, out, ws, window=WINDOW, sinks=SINKS)
            elif groups is None:
                fmad.paged_attention(c.handle, l, b, q, out, ws)
            else:
                fmad.shared_attention(c.handle, l, b, groups, q, out, ws)
            for i in range(len(seq)) if checked is None else checked:
                rows = slice(start[i], start[i + 1])
                if l == 0:
                    ref, size = sink_ref(c, i, q[rows], Dh ** -0.5, True, WINDOW, SINKS, l)
                else:
                    ref, size = attention_ref(c, i, q[rows], Dh ** -0.5, True, 0, l)
                # as in the attention's own tests
                tol = ref.abs() * 2.0 ** -8 + size * ((2.0 ** -11 if fp8 else 2.0 ** -8) + 2.0 ** -9)
                assert bool(((out[rows].double() - ref).abs() <= tol).all()), (l, i)
                # queries have the size of their gain: the rotation keeps a pair's norm, bf16 rounds by 2^-8
                x = qkv[rows, :H].double()
                x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * gains[0].double()
                assert bool(((q[rows].double().norm(dim=-1) / x.norm(dim=-1) - 1).abs() <= 2.0 ** -7).all())
            qkv = (qkv + torch.cat((out, qkv[:, H:] * 0), 1)).contiguous()
        assert status.tolist()[0] == 0 and fmad.standalone_status() == 0

    layers([3], [4000])
    layers([3], [observed - 4000])
    others = [s for s in range(n) if s != 3]
    fmad.kv_fork(c.handle, i32([3] * (n - 1)), i32(others), status)
    seq = [3] + others
    groups = fmad.KvGroups(i32([0, n]), i32([observed]), n, observed)
    layers(seq, [1] * n, groups)
    layers(seq, [1 + i % 2 for i in range(n)], groups)
    assert int(c.refs[c.table[3, 0].long()]) == n and int(c.refs[c.table[3, observed // page].long()]) == 1
    # the best candidates go on alone
    fmad.kv_release(c.handle, i32(others[5:]), status)
    layers(seq[:6], [1] * 6, None)
    cfg, p = policy("expert_bf16_m63", P=64)
    p.refresh_prefix_pages(0, 64, c.handle, 3, observed - 60)
    c.rows, c.lens_host = [3], [int(c.lens[3])]
    k = p.buffer("prefix_k", torch.bfloat16, (L, 64, Hkv, Dh))
    for l in range(L):
        assert torch.equal(k[l][:62], c.dense(0, l)[0][observed - 60:observed + 2].float().to(torch.bfloat16))
    fmad.device_status(p.handle)


def test_first_calls_inside_a_capture():
    """A fresh process whose first call of every operator is captured."""
    require_gpu()
    code = """
import torch, sys
sys.path[:0] = [%r, %r]
import flow_matching_action_denoise_gb300 as fmad
from _kv import batch
from test_gpu_shared_attention import Forks
c = Forks([(8100, [20] * 110)], 64, 2, 128, seed=1)
one, many = batch(c, [1] * 110), batch(c, [20] * 110)
groups, rope = c.groups(), fmad.Rope(64)
x = [torch.randn((b.tokens, 20, 128), device="cuda").to(torch.bfloat16) for b in (one, many)]
q = [torch.empty_like(t[:, :16].contiguous()) for t in x]
outs = [[torch.zeros_like(t) for t in q for _ in range(2)] for _ in range(2)]
need = max([fmad.paged_attention_workspace_size(c.handle, b, 16) for b in (one, many)] +
           [fmad.shared_attention_workspace_size(c.handle, b, groups, 16) for b in (one, many)])
ws = torch.empty(need, dtype=torch.uint8, device="cuda")
kept = c.k.clone(), c.v.clone()
def work(out):
    c.k.copy_(kept[0]), c.v.copy_(kept[1])
    for i, b in enumerate((one, many)):
        fmad.norm_rope_append(c.handle, 0, b, rope, x[i][:, :16], x[i][:, 16:18], x[i][:, 18:], q[i])
        fmad.sink_attention(c.handle, 0, b, q[i], out[2 * i], ws, window=300, sinks=20)
        fmad.shared_attention(c.handle, 0, b, groups, q[i], out[2 * i + 1], ws)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    work(outs[0])
g.replay()
torch.cuda.synchronize()
work(outs[1])
torch.cuda.synchronize()
assert fmad.standalone_status() == 0
assert all(torch.equal(a, b) and bool((a != 0).any()) for a, b in zip(*outs))
print("same")
""" % (fmad.__path__[0] + "/..", __file__.rsplit("/", 1)[0])
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
