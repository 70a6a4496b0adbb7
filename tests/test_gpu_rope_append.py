"""Rotary positions and the store into the paged cache against their definition in 64 bits.

Tolerances: the angle's fraction of a turn is exact to 2^-31 half turns plus the table's 2^-52 turns a position, so
cos and sin are off by less than 2^-28 + the function's 2 ulp (2^-22): with |x| the pair's norm the rotated value is off
by at most 2^-20 |x| in fp32, then rounded: 2^-8 relative (bf16) or 2^-4 of the value and half of E4M3's smallest step
(2^-10) in code units."""
import math

import numpy as np
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import Cache, batch

pytestmark = pytest.mark.gpu


def frequencies(rot, theta, scaling, factor, original, fast, slow):
    if scaling == fmad.ROPE_BASE:
        theta = theta * factor ** (rot / (rot - 2))
    i = np.arange(rot // 2, dtype=np.float64)
    f = theta ** (-2 * i / rot)
    if scaling == fmad.ROPE_LINEAR:
        f = f / factor
    mag = 1.0
    if scaling == fmad.ROPE_BY_PARTS:
        # the pair index whose wavelength turns `t` times within the original length
        at = lambda t: rot * np.log(original / (2 * np.pi * t)) / (2 * np.log(theta))
        lo, hi = max(np.floor(at(fast)), 0), min(np.ceil(at(slow)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        mag = 0.1 * math.log(factor) + 1
    return f, mag


def rotate(x, pos, rot, half, f, mag):
    """x [T][heads][Dh] float64 turned by pos * f."""
    out = x.clone()
    ang = pos.double()[:, None] * torch.from_numpy(f).to(x.device)
    c, s = (torch.cos(ang) * mag)[:, None], (torch.sin(ang) * mag)[:, None]
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if half else (x[..., 0:rot:2], x[..., 1:rot:2])
    u, w = a * c - b * s, b * c + a * s
    if half:
        out[..., :rot // 2], out[..., rot // 2:rot] = u, w
    else:
        out[..., 0:rot:2], out[..., 1:rot:2] = u, w
    size = out.clone().abs()
    norm = torch.sqrt(a * a + b * b) * mag
    if half:
        size[..., :rot // 2], size[..., rot // 2:rot] = norm, norm
    else:
        size[..., 0:rot:2], size[..., 1:rot:2] = norm, norm
    return out, size


def near(got, ref, size, scale=None):
    err = (got.double() - ref).abs()
    if scale is None:
        tol = ref.abs() * 2.0 ** -8 + size * 2.0 ** -20
    else:
        # codes: the reciprocal's and the product's fp32 roundings are 2^-22 of the value
        tol = (ref.abs() * (2.0 ** -4 + 2.0 ** -21) + size * 2.0 ** -20) / scale + 2.0 ** -10
        err = (got.double() - ref / scale).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def run(lens, new, page, H, Hkv, Dh, rot, half, fp8=False, heads_first=False, scaling=0, merged=True, positions=None,
        layer=0, layers=1, theta=10000.0, lead=0, trail=0, in_place=False, seq=True, rows=None):
    c = Cache(lens, page, Hkv, Dh, fp8, layers, heads_first=heads_first, seed=rot + page, poison=False, rows=rows)
    before = [t.clone() for t in (c.k, c.v)]
    b = batch(c, new, seq, lead, trail)
    T = b.tokens
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn((T, H + 2 * Hkv, Dh), generator=g).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    if not merged:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    src = [x.clone() for x in (q, k, v)]
    q_out = q if in_place else torch.full((T, H, Dh), 7.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(theta=theta, scaling=scaling, factor=4.0, original_len=512.0, beta_fast=16.0, beta_slow=1.0)
    rope = fmad.Rope(rot, half=half, **kw)
    f, mag = frequencies(rot, theta, scaling, 4.0, 512.0, 16.0, 1.0)
    pos_in = None if positions is None else torch.tensor(positions, dtype=torch.int32, device="cuda")
    fmad.rope_append(c.handle, layer, b, rope, q, k, v, q_out, pos_in)
    torch.cuda.synchronize()
    assert fmad.standalone_status() == 0
    start = b.start.cpu().tolist()
    touched = torch.zeros((c.k.shape[1], page), dtype=torch.bool, device="cuda")
    for i, n in enumerate(new):
        rows_ = slice(start[i], start[i + 1])
        place = torch.arange(lens[i] - n, lens[i], device="cuda")
        pos = place if pos_in is None else pos_in[rows_]
        qr, size = rotate(src[0][rows_].double(), pos, rot, half, f, mag)
        near(q_out[rows_], qr, size)
        kr, ksize = rotate(src[1][rows_].double(), pos, rot, half, f, mag)
        vr = src[2][rows_].double()
        pg = c.table[c.rows[i]][place // page].long()
        touched[pg, place % page] = True
        for t, ref, sz, s in ((c.k, kr, ksize, c.k_scale), (c.v, vr, vr.abs(), c.v_scale)):
            near(t[layer].to(torch.float64)[pg, place % page], ref, sz, s[layer].double() if fp8 else None)
    if not in_place:
        assert (q_out[:start[0]] == 7).all() and (q_out[start[-1]:] == 7).all()
    # every other cell of the cache is as it was
    for t, old in zip((c.k, c.v), before):
        same = (t.view(torch.uint8) == old.view(torch.uint8)) if fp8 else (t.view(torch.int16) == old.view(torch.int16))
        for l in range(layers):
            mask = touched if l == layer else torch.zeros_like(touched)
            assert bool(same[l].all(-1).all(-1)[~mask].all())


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Dh,rot", [(128, 128), (128, 64), (64, 16), (64, 64), (256, 48), (16, 16)])
def test_layouts(Dh, rot, fp8, half):
    require_gpu()
    run([50, 3, 200], [7, 3, 1], 16, 5, 2, Dh, rot, half, fp8, heads_first=rot == 64, lead=2, trail=1)


@pytest.mark.parametrize("scaling", range(4))
def test_scaling(scaling):
    require_gpu()
    run([900], [300], 32, 4, 1, 64, 64, True, scaling=scaling)


def test_far_positions():
    """Positions up to 2^31 - 1, where a 32-bit angle has no digits left."""
    require_gpu()
    far = [0, 1, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 30 + 7, 2 ** 31 - 1]
    for half in (True, False):
        run([40], [6], 16, 2, 1, 128, 128, half, positions=far, theta=500000.0)


def test_shapes_and_strides():
    require_gpu()
    run([33], [33], 16, 1, 1, 128, 32, True, merged=False)
    run([33, 64], [1, 64], 64, 7, 7, 64, 32, False, layers=3, layer=2)
    run([20], [9], 256, 3, 1, 128, 128, True, in_place=True)
    run([20, 30], [9, 1], 16, 3, 1, 128, 128, False, seq=False, rows=[0, 1])
    run([2000, 900, 1], [1500, 900, 1], 128, 16, 2, 128, 128, True)      # enough tokens for eight heads a thread


def test_keys_and_values_only_and_no_rotation():
    require_gpu()
    c = Cache([20], 16, 2, 64, seed=1, poison=False)
    b = batch(c, [4])
    k, v = (torch.randn((4, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    fmad.rope_append(c.handle, 0, b, fmad.Rope(16), None, k, v, None)
    rope = fmad.Rope(16)
    rope.struct.rotary_dim = 0
    fmad.rope_append(c.handle, 0, b, rope, None, k, v, None)
    kk, vv = c.dense(0)
    assert torch.equal(kk[16:].to(torch.bfloat16), k) and torch.equal(vv[16:].to(torch.bfloat16), v)


def test_saturation_and_device_side_faults():
    require_gpu()
    c = Cache([20], 16, 1, 64, True, seed=1, poison=False)
    c.k_scale.fill_(1.0), c.v_scale.fill_(2.0)
    b = batch(c, [4])
    k = torch.full((4, 1, 64), 1000.0, device="cuda").to(torch.bfloat16)
    k[1] = -3e38
    fmad.rope_append(c.handle, 0, b, fmad.Rope(16), None, k, k, None)
    vv = c.v[0].float()[c.table[c.rows[0], 1].long(), 0:4]
    assert vv[0].eq(448).all() and vv[1].eq(-448).all()
    assert fmad.standalone_status() == 0
    old = c.table[c.rows[0], 1].clone()
    for page in (-1, 10 ** 6):
        c.table[c.rows[0], 1] = page
        before = c.k.view(torch.uint8).clone()
        fmad.rope_append(c.handle, 0, b, fmad.Rope(16), None, k, k, None)
        assert fmad.standalone_status() == 2 and torch.equal(before, c.k.view(torch.uint8))
    c.table[c.rows[0], 1] = old
    c.lens[c.rows[0]] = 2      # fewer than the new tokens: the first two have no place
    fmad.rope_append(c.handle, 0, b, fmad.Rope(16), None, k, k, None)
    assert fmad.standalone_status() == 2


def test_bounds_on_the_new_tokens():
    """A bound above the packed rows changes nothing; rows behind a bound that is too small are left as they were."""
    require_gpu()
    k, v, q = (torch.randn((40, n, 64), device="cuda").to(torch.bfloat16) for n in (1, 1, 3))
    stores, outs = [], []
    for bound in (30, 1 << 30, 7):
        c = Cache([50, 60], 16, 1, 64, seed=2, poison=False)
        out = torch.full_like(q, 7.0)
        fmad.rope_append(c.handle, 0, batch(c, [30, 10], max_tokens=bound), fmad.Rope(64), q, k, v, out)
        assert fmad.standalone_status() == (2 if bound == 7 else 0)
        outs.append(out)
        stores.append((c.k.clone(), c.v.clone()))
    assert torch.equal(outs[0], outs[1]) and all(torch.equal(a, b) for a, b in zip(*stores[:2]))
    kept = [*range(7), *range(30, 37)]
    assert torch.equal(outs[2][kept], outs[0][kept])
    assert outs[2][7:30].eq(7).all() and outs[2][37:].eq(7).all()


def test_the_binding_refuses():
    require_gpu()
    c = Cache([20], 16, 2, 64, seed=1, poison=False)
    b, rope = batch(c, [4]), fmad.Rope(64)
    q, k = (torch.zeros((4, n, 64), device="cuda", dtype=torch.bfloat16) for n in (4, 2))
    good = dict(q=q, k=k, v=k, q_out=q)
    fmad.rope_append(c.handle, 0, b, rope, **good)
    for bad in (dict(q_out=None), dict(q=q[0]), dict(q=q[:3]), dict(k=k.float()), dict(v=k.cpu()), dict(k=k[:, :, ::2]),
                dict(v=q), dict(q_out=q.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(4, dtype=torch.int64, device="cuda"))):
        with pytest.raises(fmad.FmError):
            fmad.rope_append(c.handle, 0, b, rope, **{**good, **bad})
