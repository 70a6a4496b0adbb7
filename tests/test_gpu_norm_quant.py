"""Residual + RMS norm + E4M3 output against its definition in 64 bits.

Tolerances: the row's mean is an fp32 sum of d squares in at most 32 + 16 + 5 sequential additions per thread, lane and
warp, the factor and products add a few roundings: y and the scale are within 64 * 2^-24 = 2^-18 relative. A code is
E4M3(y / scale): 2^-4 of the value and half of the smallest step (2^-10) in code units, plus 2^-17 for y and the scale."""
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu

pytestmark = pytest.mark.gpu


def reference(x, r, gamma, eps, block):
    s = x.double() + (r.double() if r is not None else 0)
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    if gamma is not None:
        y = y * gamma.double()
    T, d = y.shape
    b = block or d
    cols = -(-d // b)
    scale = torch.stack([y[:, i * b:(i + 1) * b].abs().amax(1) for i in range(cols)], 1) / 448
    wide = scale.repeat_interleave(b, 1)[:, :d]
    return s, torch.where(wide > 0, y / wide, torch.zeros_like(y)), scale


def run(T, d, f32, res, gamma, block, eps=1e-6, alias=False, pad=0, x=None, store=True):
    g = torch.Generator().manual_seed(T + d)
    t = torch.float32 if f32 else torch.bfloat16
    if x is None:
        x = torch.randn((T, d), generator=g) * torch.exp(torch.randn((T, 1), generator=g))
    wide = torch.zeros((T, d + pad), dtype=t, device="cuda")
    wide[:, :d] = x.to(t).cuda()
    x = wide[:, :d]
    r = torch.randn((T, d + pad), generator=g).to(torch.bfloat16).cuda()[:, :d] if res else None
    gm = (1 + 0.3 * torch.randn(d, generator=g)).cuda() if gamma else None
    x0 = x.clone()
    out = x if alias else torch.full((T, d + pad), 3.0, dtype=t, device="cuda")[:, :d]
    codes = torch.empty((T, d), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((T, -(-d // 128) if block else 1), device="cuda")
    fmad.norm_quant(x, r, gm, eps, out if store else None, codes, scales, block)
    torch.cuda.synchronize()
    s, c, sc = reference(x0, r, gm, eps, block)
    if store:
        # one fp32 addition, and bf16's rounding
        assert bool(((out.double() - s).abs() <= s.abs() * (2.0 ** -24 if f32 else 2.0 ** -8 + 2.0 ** -23)).all())
    else:
        assert torch.equal(x, x0)
    assert bool(((scales.double() - sc).abs() <= sc * 2.0 ** -18).all())
    err = (codes.double() - c).abs()
    assert bool((err <= c.abs() * (2.0 ** -4 + 2.0 ** -17) + 2.0 ** -10).all()), float(err.max())
    return codes, scales


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,d", [(1, 16), (3, 144), (10, 1024), (7, 256), (2, 2048), (5, 4096), (2, 8192), (3, 16384),
                                 (1, 4112), (700, 272), (2300, 1040), (5000, 2048), (1500, 4096), (800, 8208)])
def test_shapes(T, d, f32, block):
    require_gpu()
    run(T, d, f32, True, True, block)


@pytest.mark.parametrize("res,gamma", [(False, True), (True, False), (False, False)])
def test_without_parts(res, gamma):
    require_gpu()
    run(20, 528, False, res, gamma, 128)
    run(20, 528, True, res, gamma, 0, eps=0.5, store=False)


def test_strides_and_in_place():
    require_gpu()
    run(33, 1024, False, True, True, 0, alias=True, pad=24)
    run(9000, 512, True, True, True, 128, alias=True, pad=8)


def test_zeros_and_extremes():
    require_gpu()
    x = torch.randn(6, 512)
    x[0] = 0
    x[1] = 0
    x[1, 300] = 5.0
    x[2] *= 1e-30
    x[3] *= 1e15
    x[4, :128] = 0
    codes, scales = run(6, 512, True, False, True, 128, eps=0.0 + 1e-12, x=x)
    assert (codes.float()[0] == 0).all() and (scales[0] == 0).all()
    assert (codes.float()[4, :128] == 0).all() and scales[4, 0] == 0
    run(6, 512, True, False, False, 0, eps=1e-12, x=x)


def test_not_finite_stays_in_its_row():
    require_gpu()
    x = torch.randn(40, 256, device="cuda")
    clean = [torch.empty((40, 256), dtype=torch.uint8, device="cuda"), torch.empty(40, device="cuda")]
    dirty = [torch.empty_like(t) for t in clean]
    fmad.norm_quant(x, None, None, 1e-6, None, *clean)
    x[11, 5], x[12, 7] = float("nan"), float("inf")
    fmad.norm_quant(x, None, None, 1e-6, None, *dirty)
    keep = [i for i in range(40) if i not in (11, 12)]
    assert torch.equal(clean[0][keep], dirty[0][keep]) and torch.equal(clean[1][keep], dirty[1][keep])
    assert bool((dirty[0][11] & 0x7F == 0x7F).any())


def test_graph_and_stream():
    require_gpu()
    x = torch.randn(64, 2048, device="cuda")
    r = torch.randn(64, 2048, device="cuda").to(torch.bfloat16)
    a, b = ([torch.empty_like(x), torch.empty((64, 2048), dtype=torch.uint8, device="cuda"),
             torch.empty((64, 16), device="cuda")] for _ in range(2))
    fmad.norm_quant(x, r, None, 1e-6, *a, block=128)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fmad.norm_quant(x, r, None, 1e-6, *b, block=128)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, w) for u, w in zip(a, b))


def test_the_binding_refuses():
    require_gpu()
    x = torch.zeros((4, 64), device="cuda")
    r = x.to(torch.bfloat16)
    good = dict(x=x, r=r, gamma=x[0], eps=1e-6, x_out=x, codes=torch.empty((4, 64), dtype=torch.uint8, device="cuda"),
                scales=torch.empty(4, device="cuda"))
    fmad.norm_quant(**good)
    for bad in (dict(x=x[0]), dict(x=x.half()), dict(x=x.cpu()), dict(x=x[:, ::2]), dict(r=x), dict(r=r[:3]), dict(gamma=r[0]),
                dict(gamma=x[0, :32]), dict(x_out=r), dict(codes=good["codes"][:3]), dict(scales=good["scales"][:3]),
                dict(block=128, scales=torch.empty(5, device="cuda")), dict(block=64), dict(eps=-1.0)):
        with pytest.raises(fmad.FmError):
            fmad.norm_quant(**{**good, **bad})
