"""The append with normalised heads against its definition in 64 bits.

Tolerances. The mean square is a sum of at most 256 products in fp32 along a tree of depth below 24: 2^-19 relative, the root
halves that; root, reciprocal and two products add 2^-22 each: y is off by less than 2^-18. Cosine and sine are off by 2^-22
at most (as in the plain append's tests), so a rotated value by 2^-17 of its pair's norm. Then one rounding: 2^-8 relative
(bf16), or 2^-4 of the value and half of E4M3's smallest step (2^-10) in code units."""
import math

import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import Cache, batch
from test_gpu_rope_append import frequencies, rotate

pytestmark = pytest.mark.gpu


def normalised(x, gamma, eps):
    """x [T][heads][Dh] float64."""
    y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    return y if gamma is None else y * gamma.double()


def near(got, ref, size, scale=None):
    err = (got.double() - ref).abs()
    if scale is None:
        tol = ref.abs() * 2.0 ** -8 + size * 2.0 ** -17
    else:
        tol = (ref.abs() * (2.0 ** -4 + 2.0 ** -21) + size * 2.0 ** -17) / scale + 2.0 ** -10
        err = (got.double() - ref / scale).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def heads(T, n, Dh, seed, sizes=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, n, Dh), generator=g)
    return (x * torch.exp(2 * torch.randn((T, n, 1), generator=g)) if sizes else x).to(torch.bfloat16).cuda()


def run(lens, new, page, H, Hkv, Dh, rot, half=True, fp8=False, heads_first=False, gains=True, eps=1e-6, positions=None,
        layer=0, layers=1, lead=0, trail=0, in_place=False, seq=True, rows=None, merged=True, x=None):
    c = Cache(lens, page, Hkv, Dh, fp8, layers, heads_first=heads_first, seed=rot + page, poison=False, rows=rows)
    if fp8:   # codes of normalised values stay below 448
        c.k_scale.fill_(0.0625), c.v_scale.fill_(0.25)
    before = [t.clone() for t in (c.k, c.v)]
    b = batch(c, new, seq, lead, trail)
    T = b.tokens
    qkv = heads(T, H + 2 * Hkv, Dh, 3) if x is None else x
    if fp8:
        qkv[:, H + Hkv:] = qkv[:, H + Hkv:].clamp(-100, 100)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    if not merged:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    src = [t.clone() for t in (q, k, v)]
    q_out = q if in_place else torch.full((T, H, Dh), 7.0, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(4)
    qg, kg = ((torch.randn(Dh, generator=g) + 1).cuda() for _ in range(2)) if gains else (None, None)
    rope = fmad.Rope(rot, half=half)
    f, _ = frequencies(rot, 10000.0, 0, 1, 1, 2, 1)
    pos_in = None if positions is None else torch.tensor(positions, dtype=torch.int32, device="cuda")
    fmad.norm_rope_append(c.handle, layer, b, rope, q, k, v, q_out, qg, kg, eps, pos_in)
    torch.cuda.synchronize()
    assert fmad.standalone_status() == 0
    start = b.start.cpu().tolist()
    touched = torch.zeros((c.k.shape[1], page), dtype=torch.bool, device="cuda")
    for i, n in enumerate(new):
        rows_ = slice(start[i], start[i + 1])
        place = torch.arange(lens[i] - n, lens[i], device="cuda")
        pos = place if pos_in is None else pos_in[rows_]
        qn, kn = (normalised(t[rows_].double(), gain, eps) for t, gain in ((src[0], qg), (src[1], kg)))
        (qr, qs), (kr, ks) = ((rotate(t, pos, rot, half, f, 1.0) if rot else (t, t.abs())) for t in (qn, kn))
        near(q_out[rows_], qr, qs)
        vr = src[2][rows_].double()
        pg = c.table[c.rows[i]][place // page].long()
        touched[pg, place % page] = True
        near(c.k[layer].to(torch.float64)[pg, place % page], kr, ks, c.k_scale[layer].double() if fp8 else None)
        near(c.v[layer].to(torch.float64)[pg, place % page], vr, vr.abs(), c.v_scale[layer].double() if fp8 else None)
    if not in_place:
        assert (q_out[:start[0]] == 7).all() and (q_out[start[-1]:] == 7).all()
    for t, old in zip((c.k, c.v), before):   # every other cell of the cache is as it was
        same = (t.view(torch.uint8) == old.view(torch.uint8)) if fp8 else (t.view(torch.int16) == old.view(torch.int16))
        for l in range(layers):
            mask = touched if l == layer else torch.zeros_like(touched)
            assert bool(same[l].all(-1).all(-1)[~mask].all())


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Dh,rot", [(128, 128), (128, 64), (64, 16), (64, 0), (256, 48), (16, 16), (80, 80), (96, 48), (208, 208)])
def test_layouts(Dh, rot, fp8, half):
    """Heads of 1 to 16 pieces, some of them no power of two; heads inside and outside of tokens."""
    require_gpu()
    run([50, 3, 200], [7, 3, 1], 16, 5, 2, Dh, rot, half, fp8, heads_first=rot == 48, lead=2, trail=1)


def test_shapes_and_strides():
    require_gpu()
    run([33], [33], 16, 1, 1, 128, 32, merged=False)
    run([33, 64], [1, 64], 64, 7, 7, 64, 32, False, layers=3, layer=2)
    run([20], [9], 256, 3, 1, 128, 128, in_place=True)
    run([20], [9], 256, 3, 1, 80, 80, in_place=True, gains=False, eps=0.0)
    run([20, 30], [9, 1], 16, 40, 1, 128, 128, False, seq=False, rows=[0, 1])
    run([2000, 900, 1], [1500, 900, 1], 128, 16, 2, 128, 128)      # enough tokens for eight heads a thread
    run([900, 1000], [900, 700], 32, 14, 2, 112, 64, fp8=True)
    run([40], [6], 16, 2, 1, 128, 128, positions=[0, 1, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 30 + 7, 2 ** 31 - 1])


@pytest.mark.parametrize("Dh", [16, 80, 128, 256])
def test_heads_of_any_size(Dh):
    """Squares that overflow or vanish in fp32: powers of two times ordinary heads keep their norm, eps 0."""
    require_gpu()
    sizes = torch.tensor([2.0 ** e for e in (0, 124, -116, 70, 63, 64, 62, -70, -63, -60, -50, 1)])
    x = torch.randn((12, 8, Dh), generator=torch.Generator().manual_seed(Dh)).clamp(-7, 7)
    x[x.abs() < 2.0 ** -9] = 2.0 ** -9
    x = (x * sizes[:, None, None]).to(torch.bfloat16).cuda()
    run([12], [12], 16, 4, 2, Dh, 16, eps=0.0, x=x)


def test_eps_beside_tiny_heads():
    require_gpu()
    x = (torch.randn((24, 4, 64), generator=torch.Generator().manual_seed(1)) * 2.0 ** -60).to(torch.bfloat16).cuda()
    for eps in (1e-36, 1e-30, 0.0, 1.0):
        run([24], [24], 16, 2, 1, 64, 64, eps=float(torch.tensor(eps, dtype=torch.float32)), x=x.clone())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Dh", [64, 80, 256])
def test_zero_and_not_finite_heads(Dh, fp8):
    """A head of zeros stays zero; one with a NaN or an infinity is NaN throughout, no other head changes a bit."""
    require_gpu()
    H, Hkv, T = 5, 3, 6
    clean = heads(T, H + 2 * Hkv, Dh, 7, sizes=False)
    bad = clean.clone()
    spots = [(0, 0, 0, math.nan), (1, 4, Dh - 1, math.inf), (2, 5, 3, -math.inf), (3, 6, Dh // 2, math.nan), (4, 2, 9, math.inf),
             (4, 2, 10, -math.inf)]
    for t, h, d, x in spots:
        bad[t, h, d] = x
    clean[5, 1] = bad[5, 1] = 0
    outs = []
    for x in (clean, bad):
        c = Cache([T], 16, Hkv, Dh, fp8, seed=1, poison=False)
        if fp8:
            c.k_scale.fill_(0.0625), c.v_scale.fill_(0.25)
        q_out = torch.empty((T, H, Dh), dtype=torch.bfloat16, device="cuda")
        fmad.norm_rope_append(c.handle, 0, batch(c, [T]), fmad.Rope(16), x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], q_out, eps=0.0)
        assert fmad.standalone_status() == 0
        k, v = c.dense(0)
        outs.append(torch.cat((q_out.double(), k, v), 1))
    assert (outs[0][5, 1] == 0).all() and not outs[0].isnan().any()
    for t, h in {(t, h) for t, h, _, _ in spots}:
        assert outs[1][t, h].isnan().all()
        outs[1][t, h] = outs[0][t, h]
    assert torch.equal(*outs)


def test_keys_and_values_only_and_faults():
    require_gpu()
    c = Cache([20], 16, 2, 64, seed=1, poison=False)
    b = batch(c, [4])
    k, v = heads(4, 2, 64, 1), heads(4, 2, 64, 2)
    fmad.norm_rope_append(c.handle, 0, b, fmad.Rope(0), None, k, v, None, None, None)
    kk, vv = c.dense(0)
    near(kk[16:], normalised(k.double(), None, 1e-6), 0 * kk[16:])
    assert torch.equal(vv[16:].to(torch.bfloat16), v)
    # a token without a page: bit 2, nothing stored, its queries turned all the same
    q = heads(4, 3, 64, 5)
    outs = []
    for page in (c.table[c.rows[0], 1].item(), -1, 10 ** 6):
        c.table[c.rows[0], 1] = page
        before, q_out = c.k.clone(), torch.zeros_like(q)
        fmad.norm_rope_append(c.handle, 0, b, fmad.Rope(64), q, k, v, q_out)
        good = 0 <= page < 100
        assert fmad.standalone_status() == (0 if good else 2)
        assert torch.equal(before, c.k) != good
        outs.append(q_out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_bounds_on_the_new_tokens():
    require_gpu()
    k, v, q = (heads(40, n, 64, n) for n in (1, 1, 3))
    stores, outs = [], []
    for bound in (30, 1 << 30, 7):
        c = Cache([50, 60], 16, 1, 64, seed=2, poison=False)
        out = torch.full_like(q, 7.0)
        fmad.norm_rope_append(c.handle, 0, batch(c, [30, 10], max_tokens=bound), fmad.Rope(64), q, k, v, out)
        assert fmad.standalone_status() == (2 if bound == 7 else 0)
        outs.append(out)
        stores.append((c.k.clone(), c.v.clone()))
    assert torch.equal(outs[0], outs[1]) and all(torch.equal(a, b) for a, b in zip(*stores[:2]))
    kept = [*range(7), *range(30, 37)]
    assert torch.equal(outs[2][kept], outs[0][kept])
    assert outs[2][7:30].eq(7).all() and outs[2][37:].eq(7).all()


def test_graph_replay_and_other_stream():
    require_gpu()
    c = Cache([300, 70], 32, 2, 128, True, seed=3, poison=False)
    b, rope = batch(c, [40, 2]), fmad.Rope(128)
    x = heads(42, 12, 128, 9, sizes=False)
    args = (x[:, :8], x[:, 8:10], x[:, 10:])
    eager = torch.zeros((42, 8, 128), dtype=torch.bfloat16, device="cuda")
    fmad.norm_rope_append(c.handle, 0, b, rope, *args, eager)
    torch.cuda.synchronize()
    first = c.k.view(torch.uint8).clone()
    replay, s, g = torch.zeros_like(eager), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fmad.norm_rope_append(c.handle, 0, b, rope, *args, replay)
    for _ in range(2):
        c.k.view(torch.uint8).zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, replay)
    where = c.k.view(torch.uint8) != 0
    assert torch.equal(c.k.view(torch.uint8)[where], first[where])
    other = torch.zeros_like(eager)
    fmad.norm_rope_append(c.handle, 0, b, rope, *args, other, stream=s)
    s.synchronize()
    assert torch.equal(eager, other)


def test_the_binding_refuses():
    require_gpu()
    c = Cache([20], 16, 2, 64, seed=1, poison=False)
    b, rope = batch(c, [4]), fmad.Rope(64)
    q, k = (torch.zeros((4, n, 64), device="cuda", dtype=torch.bfloat16) for n in (4, 2))
    good = dict(q=q, k=k, v=k, q_out=q, q_gamma=torch.ones(64, device="cuda"))
    fmad.norm_rope_append(c.handle, 0, b, rope, **good)
    ones = torch.ones(64, device="cuda")
    for bad in (dict(q_out=None), dict(q=q[0]), dict(k=k.float()), dict(v=k.cpu()), dict(v=q), dict(q_gamma=ones[:32]),
                dict(q_gamma=ones.double()), dict(k_gamma=ones.cpu()), dict(k_gamma=torch.ones(128, device="cuda")[::2]),
                dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf)):
        with pytest.raises(fmad.FmError):
            fmad.norm_rope_append(c.handle, 0, b, rope, **{**good, **bad})
