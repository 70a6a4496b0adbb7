"""Norm rows at the ends of fp32's range: finite rows whose squares overflow or vanish, rows that are not finite.

Tolerances as in the operator's own tests: squares of a row scaled by a power of two have the roundings of an ordinary row."""
import math

import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from test_gpu_norm_quant import reference

pytestmark = pytest.mark.gpu

# every way rows are spread over threads: 8, 16, 32 lanes, a CTA a row, several vectors a thread
SHAPES = [(3, 64), (40, 128), (9, 256), (7, 1040), (5, 4096), (3, 16384), (30000, 256), (10000, 512), (5000, 1024), (2600, 2048)]


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,d", SHAPES)
def test_finite_rows_of_any_size(T, d, f32, block):
    """Powers of two times ordinary rows; eps 0, so that the smallest keep their norm."""
    require_gpu()
    g = torch.Generator().manual_seed(T + d)
    x = torch.randn((T, d), generator=g).clamp(-7, 7)
    x[x.abs() < 2.0 ** -9] = 2.0 ** -9   # keeps the smallest rows' elements out of the subnormals
    sizes = [0, 124, -116, 70, 63, 64, 62, -70, -63, -60, -50, 1]
    x = x * torch.tensor([2.0 ** sizes[i % len(sizes)] for i in range(T)])[:, None]
    x = x.to(torch.float32 if f32 else torch.bfloat16).cuda()
    codes = torch.empty((T, d), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((T, -(-d // 128) if block else 1), device="cuda")
    out = torch.empty_like(x)
    fmad.norm_quant(x, None, None, 0.0, out, codes, scales, block)
    _, c, sc = reference(x, None, None, 0.0, block)
    assert torch.equal(out, x)
    assert bool(((scales.double() - sc).abs() <= sc * 2.0 ** -18).all())
    err = (codes.double() - c).abs()
    assert bool((err <= c.abs() * (2.0 ** -4 + 2.0 ** -17) + 2.0 ** -10).all())


def test_eps_beside_tiny_rows():
    """eps as small as the mean square itself."""
    require_gpu()
    g = torch.Generator().manual_seed(1)
    x = (torch.randn((24, 512), generator=g) * 2.0 ** -60).cuda()
    for eps in (1e-36, 1e-30, 0.0):
        codes = torch.empty((24, 512), dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(24, device="cuda")
        fmad.norm_quant(x, None, None, eps, None, codes, scales)
        # eps as the kernel gets it
        _, c, sc = reference(x, None, None, float(torch.tensor(eps, dtype=torch.float32)), 0)
        assert bool(((scales[:, None].double() - sc).abs() <= sc * 2.0 ** -18).all())
        assert bool(((codes.double() - c).abs() <= c.abs() * (2.0 ** -4 + 2.0 ** -17) + 2.0 ** -10).all())


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("T,d", SHAPES)
def test_not_finite_rows_are_nan_throughout(T, d, block):
    require_gpu()
    x = torch.randn((T, d), device="cuda")
    cols = -(-d // 128) if block else 1

    def run(x):
        codes, scales = torch.empty((T, d), dtype=torch.uint8, device="cuda"), torch.empty((T, cols), device="cuda")
        fmad.norm_quant(x, None, None, 1e-6, None, codes, scales, block)
        return codes, scales

    clean = run(x)
    rows = sorted({0, T - 1, T // 2})
    for i, v in zip(rows, (math.nan, math.inf, -math.inf)):
        x[i, (37 * i + 5) % d] = v
    codes, scales = run(x)
    for i in rows:
        assert bool((codes[i] & 0x7F == 0x7F).all()) and bool(scales[i].isnan().all()), i
        codes[i], scales[i] = clean[0][i], clean[1][i]
    assert torch.equal(codes, clean[0]) and torch.equal(scales, clean[1])
    # both infinities, and sums of x and r that leave the range
    x[0, 0], x[0, 1] = math.inf, -math.inf
    codes, scales = run(x)
    assert bool((codes[0] & 0x7F == 0x7F).all()) and bool(scales[0].isnan().all())
