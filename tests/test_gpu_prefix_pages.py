"""The paged cache as it is used: a prefix model's layer step after step over pages (norm -> projection -> rotary append
-> attention), forks of its sequences, and the hand-over to a policy; caches past 32-bit offsets; first calls inside a
capture; two streams at once."""
import subprocess
import sys
import os

import numpy as np
import pytest
import torch

import fm_synth
import flow_matching_action_denoise_gb300 as fmad

from _gpu import aligned_empty, load_scales, require_gpu
from _kv import Cache, attention_ref, batch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def policy(name, **kw):
    cfg = fm_synth.config(name, L=2, S=1, **kw)
    layers = [fm_synth.layer_weights(cfg, l) for l in range(cfg.L)]
    scales = None if cfg.act_fmt == "bf16" else load_scales(name)[:2]
    return cfg, fmad.Policy(cfg, layers, fm_synth.final_weights(cfg), act_scales=scales)


@pytest.mark.parametrize("name,fp8,page,heads_first", [
    ("expert_bf16_m63", False, 16, False), ("expert_bf16_m63", True, 64, True), ("expert_fp8attn_m50", False, 32, True),
    ("expert_fp8attn_m50", True, 256, False)])
def test_refresh_prefix_pages_equals_refresh_prefix(name, fp8, page, heads_first):
    """Rows gathered from pages leave the policy's prefix buffers bit for bit as the same rows handed over densely."""
    require_gpu()
    cfg, a = policy(name, P=150)
    _, b = policy(name, P=150)
    c = Cache([200, 170], page, cfg.Hkv, cfg.Dh, fp8, cfg.L, heads_first=heads_first, seed=3)
    names = ["prefix_k", "prefix_v"] + (["prefix_k8", "prefix_v8"] if "fp8attn" in name else [])
    for entry, begin, end, tok in ((0, 0, 150, 0), (1, 37, 101, 66), (0, 149, 150, 199), (1, 8, 16, 5)):
        dense = [torch.stack([c.dense(entry, l)[j][tok:tok + end - begin] for l in range(cfg.L)]).to(torch.float32)
                 .to(torch.bfloat16).contiguous() for j in range(2)]
        a.refresh_prefix(begin, end, *dense)
        b.refresh_prefix_pages(begin, end, c.handle, int(c.rows[entry]), tok)
        torch.cuda.synchronize()
        assert fmad.device_status(b.handle) == 0
        for n in names:
            assert torch.equal(a.buffer(n), b.buffer(n)), (n, entry)
    noise = torch.randn((cfg.M, cfg.A), device="cuda")
    assert torch.equal(a.decode(noise), b.decode(noise))


def test_refresh_prefix_pages_refuses_and_reports():
    require_gpu()
    cfg, p = policy("expert_bf16_m63", P=100)
    c = Cache([90], 16, 1, 128, layers=2, seed=1)
    row = int(c.rows[0])
    for args, status in [((0, 101, c.handle, row), 2), ((5, 5, c.handle, row), 2), ((-1, 5, c.handle, row), 2),
                         ((0, 10, c.handle, 99), 1), ((0, 10, c.handle, -1), 1), ((0, 10, c.handle, row, -1), 2),
                         ((0, 10, c.handle, row, 10 ** 6), 2),
                         ((0, 10, Cache([90], 16, 1, 128, layers=1).handle, 0), 2),
                         ((0, 10, Cache([90], 16, 2, 128, layers=2).handle, 0), 2),
                         ((0, 10, Cache([90], 16, 1, 64, layers=2).handle, 0), 2)]:
        with pytest.raises(fmad.FmError) as e:
            p.refresh_prefix_pages(*args)
        assert e.value.status == status, args
    # tokens behind the length and a token without a page: zero rows and bit 2
    p.refresh_prefix_pages(0, 96, c.handle, row)
    torch.cuda.synchronize()
    assert fmad.device_status(p.handle) == 2 and fmad.device_status(p.handle) == 0
    k = p.buffer("prefix_k", torch.bfloat16, (2, 100, 1, 128))
    assert (k[:, 90:96] == 0).all() and torch.equal(k[:, :90, 0].float(), torch.stack([c.dense(0, l)[0][:, 0] for l in (0, 1)]).float())
    c.table[row, 1] = -1
    p.refresh_prefix_pages(0, 40, c.handle, row)
    assert fmad.device_status(p.handle) == 2
    assert (k[:, 16:32] == 0).all() and not (k[:, 32:40] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_prefix_model_over_pages(fp8):
    """Two layers of norm -> E4M3 projection -> rotary append -> attention over a growing, forked cache that a policy then
    reads. Every stage is held to its definition on the inputs that it got."""
    require_gpu()
    d, H, Hkv, Dh, L, page = 1024, 8, 1, 128, 2, 16
    N = (H + 2 * Hkv) * Dh
    g = torch.Generator().manual_seed(0)
    weights = []
    for _ in range(L):
        w = (torch.randn((N, d), generator=g) * 0.05).cuda()
        _, ptr = buf = aligned_empty(fmad.fm_packed_weight_bytes(N, d, fmad.FMT_FP8), "cuda")
        ws = torch.empty(1, device="cuda")
        fmad.fm_pack_weight(w, None, N, d, fmad.FMT_FP8, ptr, ws)
        codes = (w / ws).clamp(-448, 448).to(torch.float8_e4m3fn)
        weights.append((buf, ws, codes))
    c = Cache([], page, Hkv, Dh, fp8, L, seqs=6, spare_pages=60, poison=False)
    c.table = torch.full((6, 20), -1, dtype=torch.int32, device="cuda")
    c.handle = fmad.KvCache(c.k, c.v, c.table, c.lens, c.refs, c.k_scale, c.v_scale)
    rope = fmad.Rope(Dh, theta=10000.0)
    status = i32([0, 0])
    work = torch.empty(fmad.kv_workspace_size(c.handle, 6), dtype=torch.uint8, device="cuda")
    gamma = torch.ones(d, device="cuda")

    def step(seq, new, x):
        """One pass of the layers over the packed rows x [tokens][d]."""
        fmad.kv_reserve(c.handle, i32(seq), i32(new), status, work)
        assert status.tolist()[0] == 0
        T = int(sum(new))
        c.rows, c.lens_host = list(seq), [int(c.lens[s]) for s in seq]
        b = batch(c, new)
        assert b.tokens == T
        for l, (buf, ws, wc) in enumerate(weights):
            codes = torch.empty((T, d), dtype=torch.float8_e4m3fn, device="cuda")
            scales, x_new = torch.empty(T, device="cuda"), torch.empty_like(x)
            fmad.norm_quant(x, None, gamma, 1e-6, x_new, codes, scales)
            partials = torch.empty((1, T, N), device="cuda")
            fmad.fm_test_skinny_gemm(codes, T, d, buf[1], N, fmad.FMT_FP8, 8, 8, partials)
            product = codes.double() @ wc.double().T
            assert float((partials[0].double() - product).abs().max()) <= 1e-5 * float(product.abs().max())
            qkv = (partials[0] * scales[:, None] * ws).to(torch.bfloat16).view(T, H + 2 * Hkv, Dh)
            q = torch.empty((T, H, Dh), dtype=torch.bfloat16, device="cuda")
            fmad.rope_append(c.handle, l, b, rope, qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], q)
            out = torch.empty_like(q)
            fmad.paged_attention(c.handle, l, b, q, out,
                                 torch.empty(fmad.paged_attention_workspace_size(c.handle, b, H), dtype=torch.uint8, device="cuda"))
            start = b.start.tolist()
            for i in range(len(seq)):
                rows = slice(start[i], start[i + 1])
                ref, size = attention_ref(c, i, q[rows], Dh ** -0.5, True, 0, l)
                # as in the attention's own tests
                tol = ref.abs() * 2.0 ** -8 + size * ((2.0 ** -11 if fp8 else 2.0 ** -8) + 2.0 ** -9)
                assert bool(((out[rows].double() - ref).abs() <= tol).all())
                # the rows just stored: values rounded once
                v = c.dense(i, l)[1][-(start[i + 1] - start[i]):]
                given = qkv[rows, H + Hkv:].double()
                unit = float(c.v_scale[l]) if fp8 else 0.0
                assert bool(((v - given).abs() <= given.abs() * (2.0 ** -4 + 2.0 ** -20 if fp8 else 0.0) + unit * 2.0 ** -10).all())
            x = (x_new + out.reshape(T, d).float())
        assert fmad.standalone_status() == 0
        return x

    x = torch.randn((90, d), generator=g).cuda()
    step([3, 1], [50, 40], x)                          # two prompts
    step([3, 1], [30, 1], x[:31])                      # a chunk beside a single token
    fmad.kv_fork(c.handle, i32([3, 3]), i32([0, 5]), status)
    before = c.dense_of = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8))]
    step([0, 3, 5], [1, 7, 2], x[:10])                 # the fork and its source go their own ways
    assert c.refs[c.table[3, :4].long()].tolist() == [3, 3, 3, 3]
    fmad.kv_release(c.handle, i32([1, 5]), status)
    fmad.kv_compact(c.handle, status, work)
    assert status.tolist()[0] == 0 and bool((c.refs[:int((c.refs > 0).sum())] > 0).all())
    step([0, 3], [3, 1], x[:4])
    del before
    # the policy takes sequence 3's first 64 tokens as its prefix
    cfg, p = policy("expert_bf16_m63", P=64)
    p.refresh_prefix_pages(0, 64, c.handle, 3)
    c.rows, c.lens_host = [3], [int(c.lens[3])]
    k = p.buffer("prefix_k", torch.bfloat16, (L, 64, Hkv, Dh))
    for l in range(L):
        assert torch.equal(k[l], c.dense(0, l)[0][:64].float().to(torch.bfloat16))
    p.decode(torch.randn((cfg.M, cfg.A), device="cuda"))
    torch.cuda.synchronize()
    assert fmad.device_status(p.handle) == 0


@pytest.mark.parametrize("heads_first", [False, True])
def test_offsets_past_32_bits(heads_first):
    """A pool of 2^32 + elements (8.6 GB for K, as much for V): the sequences live on its last pages."""
    require_gpu()
    page, Hkv, Dh, pages = 256, 8, 128, 16500
    shape = (1, pages, Hkv, page, Dh) if heads_first else (1, pages, page, Hkv, Dh)
    k, v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 32
    if heads_first:
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    c = Cache([300], page, Hkv, Dh)    # for its reference only
    c.k, c.v, c.rows, c.lens_host = k, v, [0], [300]
    c.table = i32([pages - 1, pages - 2, -1] + [-1] * 3).view(2, 3)
    c.lens, c.refs = i32([300, 0]), torch.zeros(pages, dtype=torch.int32, device="cuda")
    c.refs[-2:] = 1
    c.handle = fmad.KvCache(k, v, c.table, c.lens, c.refs)
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn((300, 8 + 16, Dh), generator=g).to(torch.bfloat16).cuda()
    b = batch(c, [300])
    q = torch.empty((300, 8, Dh), dtype=torch.bfloat16, device="cuda")
    fmad.rope_append(c.handle, 0, b, fmad.Rope(64), qkv[:, :8], qkv[:, 8:16], qkv[:, 16:], q)
    assert torch.equal(c.dense(0)[1].to(torch.bfloat16), qkv[:, 16:])
    for new in (300, 2):
        bb = batch(c, [new])
        out = torch.empty((new, 8, Dh), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, bb, 8), dtype=torch.uint8, device="cuda")
        fmad.paged_attention(c.handle, 0, bb, q[-new:], out, ws)
        ref, size = attention_ref(c, 0, q[-new:], Dh ** -0.5, True, 0)
        assert bool(((out.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + size * (2.0 ** -8 + 2.0 ** -9)).all())
    # a fork's copy of the begun page lands on the lowest pages, compaction brings the rest after it
    want = c.dense(0)
    status, work = i32([0, 0]), torch.empty(fmad.kv_workspace_size(c.handle, 2), dtype=torch.uint8, device="cuda")
    fmad.kv_fork(c.handle, i32([0]), i32([1]), status)
    fmad.kv_reserve(c.handle, i32([1]), i32([1]), status, work)
    fmad.kv_compact(c.handle, status, work)
    assert status.tolist() == [0, 2] and c.table.tolist() == [[2, 1, -1], [2, 0, -1]] and c.lens.tolist() == [300, 301]
    got = c.dense(0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.rows, c.lens_host = [1], [300]
    got = c.dense(0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fmad.standalone_status() == 0


def test_first_calls_inside_a_capture():
    """A fresh process whose first call of every operator is captured."""
    require_gpu()
    code = """
import torch, sys
sys.path[:0] = [%r, %r]
import flow_matching_action_denoise_gb300 as fmad
from _kv import Cache, batch
c = Cache([300, 40], 16, 2, 128, seed=1)
small, large = batch(c, [1, 1]), batch(c, [60, 40])
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
q1, q2 = (torch.randn((n, 8, 128), device="cuda").to(torch.bfloat16) for n in (2, 100))
kv = torch.randn((100, 2, 128), device="cuda").to(torch.bfloat16)
outs = [[torch.zeros_like(q) for q in (q1, q2)] for _ in range(2)]
x = torch.randn(8, 256, device="cuda")
codes, scales = torch.empty((8, 256), dtype=torch.uint8, device="cuda"), torch.empty(8, device="cuda")
ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
status, rope, zero, ids = i32([0, 0]), fmad.Rope(64), i32([0, 0]), i32([int(r) for r in c.rows])
qo = torch.empty_like(q2)
def work(out):
    fmad.norm_quant(x, None, None, 1e-6, None, codes, scales)
    fmad.kv_reserve(c.handle, ids, zero, status, ws)
    fmad.kv_fork(c.handle, zero[:0], zero[:0], status)
    fmad.kv_release(c.handle, zero[:0], status)
    fmad.rope_append(c.handle, 0, large, rope, q2, kv, kv, qo)
    fmad.paged_attention(c.handle, 0, small, q1, out[0], ws)
    fmad.paged_attention(c.handle, 0, large, q2, out[1], ws)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    work(outs[0])
g.replay()
torch.cuda.synchronize()
work(outs[1])
torch.cuda.synchronize()
assert fmad.standalone_status() == 0
assert all(torch.equal(a, b) and bool(a.abs().sum() > 0) for a, b in zip(*outs))
print("captured first")
""" % (ROOT, os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_two_streams_at_once():
    """Calls on two streams with their own workspaces and outputs over one cache that neither changes."""
    require_gpu()
    c = Cache([9000, 1200, 33], 64, 2, 128, True, seed=4)
    jobs = []
    for new in ([1, 1, 1], [40, 300, 33]):
        b = batch(c, new)
        q = torch.randn((b.tokens, 8, 128), device="cuda").to(torch.bfloat16)
        ws = [torch.empty(fmad.paged_attention_workspace_size(c.handle, b, 8), dtype=torch.uint8, device="cuda") for _ in range(2)]
        alone = torch.empty_like(q)
        fmad.paged_attention(c.handle, 0, b, q, alone, ws[0])
        jobs.append((b, q, ws, alone, torch.empty_like(q)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        for s, (b, q, ws, alone, out) in zip(streams, jobs):
            fmad.paged_attention(c.handle, 0, b, q, out, ws[1], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(alone, out) for _, _, _, alone, out in jobs)
    assert fmad.standalone_status() == 0


def test_many_entries():
    """A thousand sequences of one token, and more entries than a wave of long chunks."""
    require_gpu()
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 90, 1000)]
    c = Cache(lens, 16, 1, 64, seed=6)
    for new in ([1] * 1000, [min(n, 1 + i % 40) for i, n in enumerate(lens)]):
        b = batch(c, new)
        q = torch.randn((b.tokens, 4, 64), device="cuda").to(torch.bfloat16)
        out = torch.empty_like(q)
        ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, 4), dtype=torch.uint8, device="cuda")
        fmad.paged_attention(c.handle, 0, b, q, out, ws)
        start = b.start.tolist()
        for i in range(0, 1000, 37):
            rows = slice(start[i], start[i + 1])
            ref, size = attention_ref(c, i, q[rows], 0.125, True, 0)
            assert bool(((out[rows].double() - ref).abs() <= ref.abs() * 2.0 ** -8 + size * (2.0 ** -8 + 2.0 ** -9)).all())
    assert fmad.standalone_status() == 0


def test_python_refuses_what_the_library_cannot_see():
    require_gpu()
    c = Cache([40], 16, 1, 64, seed=1)
    b = batch(c, [2])
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    bad = [(q.float(), q), (q, q.half()), (q[:1], q), (q, q[:, :2]), (q.transpose(0, 1).contiguous().transpose(0, 1), q),
           (q.cpu(), q), (q, q.cpu())]
    for a, out in bad:
        with pytest.raises((fmad.FmError, ValueError)):
            fmad.paged_attention(c.handle, 0, b, a, out)
    with pytest.raises(fmad.FmError):
        fmad.KvCache(c.k, c.v.transpose(2, 3), c.table, c.lens)
    with pytest.raises(fmad.FmError):
        fmad.KvCache(c.k.float(), c.v.float(), c.table, c.lens)
    with pytest.raises(fmad.FmError):
        fmad.KvCache(c.k, c.v, c.table.long(), c.lens)
    with pytest.raises(fmad.FmError):
        fmad.KvCache(c.k.to(torch.float8_e4m3fn), c.v.to(torch.float8_e4m3fn), c.table, c.lens)
    with pytest.raises(fmad.FmError):
        fmad.kv_release(c.handle, i32([0]), i32([0]))            # a status of one word
    with pytest.raises(fmad.FmError):
        fmad.norm_quant(q.view(2, 256), None, None, 1e-6, None, torch.empty((2, 256), dtype=torch.int8, device="cuda"),
                        torch.empty(2, device="cuda"))


def test_refresh_prefix_pages_of_sessions_and_in_a_capture():
    """A session takes its own prefix from the pages and leaves its policy's alone; a captured hand-over follows the pages."""
    require_gpu()
    cfg, a = policy("expert_bf16_m63", P=64)
    s = a.session()
    c = Cache([80, 70], 16, cfg.Hkv, cfg.Dh, layers=cfg.L, seed=4)
    a.refresh_prefix_pages(0, 64, c.handle, int(c.rows[0]))
    mine = a.buffer("prefix_k").clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.refresh_prefix_pages(0, 64, c.handle, int(c.rows[1]), 6)
    for x in (c.k, c.v):
        x.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert fmad.device_status(s.handle) == 0 and torch.equal(a.buffer("prefix_k"), mine)
    want = torch.stack([c.dense(1, l)[0][6:70] for l in range(cfg.L)]).to(torch.bfloat16)
    assert torch.equal(s.buffer("prefix_k", torch.bfloat16, want.shape), want)
    dense = [torch.stack([c.dense(1, l)[j][6:70] for l in range(cfg.L)]).to(torch.bfloat16).contiguous() for j in range(2)]
    a.refresh_prefix(0, 64, *dense)
    assert torch.equal(a.buffer("prefix_v"), s.buffer("prefix_v"))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("order,pad", [((1, 0, 3, 2, 4), 16), ((1, 0, 2, 3, 4), 0), ((0, 3, 1, 2, 4), 32), ((3, 1, 0, 2, 4), 0)])
def test_pools_of_any_order_and_gaps(order, pad, fp8):
    """Pools whose dims lie in other orders, with gaps behind the rows, give bit for bit what a dense pool gives: growth
    with a copied page, append, attention (many rows and single tokens), compaction, a policy's prefix."""
    require_gpu()
    results = []
    for free in (False, True):
        c = Cache([70, 33, 150], 16, 2, 64, fp8, layers=2, seqs=8, rows=[0, 1, 2], seed=7, poison=False, spare_pages=12)
        if free:
            pools = []
            for x in (c.k, c.v):
                y = x.permute(order)
                raw = torch.zeros((*y.shape[:-1], 64 + pad), dtype=x.dtype, device="cuda")
                back = [order.index(i) for i in range(5)]
                view = raw[..., :64].permute(back)
                view.copy_(x)
                pools.append(view)
            c.k, c.v = pools
            c.handle = fmad.KvCache(c.k, c.v, c.table, c.lens, c.refs, c.k_scale, c.v_scale)
        h, st = c.handle, torch.zeros(2, dtype=torch.int32, device="cuda")
        ws = torch.empty(max(fmad.kv_workspace_size(h, 4), fmad.kv_workspace_size(h)), dtype=torch.uint8, device="cuda")
        fmad.kv_fork(h, i32([0]), i32([3]), st)
        fmad.kv_reserve(h, i32([0, 3, 1, 2]), i32([40, 3, 1, 1]), st, ws)
        assert st.tolist()[0] == 0
        b = fmad.KvBatch(i32([0, 40, 43, 44, 45]), 45, 40, 160, i32([0, 3, 1, 2]))
        g = torch.Generator().manual_seed(1)
        q, k, v = (torch.randn((45, n, 64), generator=g).to(torch.bfloat16).cuda() for n in (8, 2, 2))
        outs = [torch.empty_like(q)]
        fmad.rope_append(h, 1, b, fmad.Rope(64), q, k, v, outs[0])
        for batch_ in (b, fmad.KvBatch(i32([43, 44, 45]), 45, 1, 160, i32([1, 2]))):
            for layer in (0, 1):
                outs.append(torch.zeros_like(q))
                need = fmad.paged_attention_workspace_size(h, batch_, 8)
                fmad.paged_attention(h, layer, batch_, outs[0], outs[-1], torch.empty(need, dtype=torch.uint8, device="cuda"))
        fmad.kv_release(h, i32([1]), st)
        fmad.kv_compact(h, st, ws)
        assert st.tolist()[0] == 0 and st.tolist()[1] > 0 and fmad.standalone_status() == 0
        for i, n in ((0, 110), (3, 73), (2, 151)):
            at = torch.arange(n, device="cuda")
            pg = c.table[i][at // 16].long()
            outs += [x[:, pg, at % 16].float() for x in (c.k, c.v)]
        results.append(outs + [c.table.clone(), c.lens.clone(), c.refs.clone()])
    assert all(torch.equal(a, b) for a, b in zip(*results))
