"""Rotary positions of no element: queries pass, keys and values are stored as they are."""
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import Cache, batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("half", [True, False])
def test_no_rotation(half):
    require_gpu()
    c = Cache([20, 9], 16, 2, 64, seed=1, poison=False)
    b = batch(c, [4, 9])
    q, k, v = (torch.randn((13, n, 64), device="cuda").to(torch.bfloat16) for n in (6, 2, 2))
    out = torch.empty_like(q)
    fmad.rope_append(c.handle, 0, b, fmad.Rope(0, half=half), q, k, v, out)
    assert fmad.standalone_status() == 0 and torch.equal(out, q)
    for i, (rows, at) in enumerate(((slice(0, 4), 16), (slice(4, 13), 0))):
        kk, vv = c.dense(i)
        assert torch.equal(kk[at:].to(torch.bfloat16), k[rows]) and torch.equal(vv[at:].to(torch.bfloat16), v[rows])
