"""Paged attention whose keys are split through the workspace: rows that no split computes, rows that hold a NaN,
and batches whose entries times splits would not fit a grid. Tolerance as in the attention's own tests."""
import numpy as np
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import Cache, attention_ref, batch

pytestmark = pytest.mark.gpu

# (lengths, new tokens, heads, bound): up to 16 stacked rows, up to 128, more
SPLIT = [([6000, 5000], [2, 1], 8, 1), ([20011, 300, 9000], [2, 3, 1], 4, 2), ([6000], [9], 8, 5), ([12000, 700], [50, 3], 8, 40)]


def attend(c, b, q, H, fill=1.0, causal=True):
    """(out, status): out starts at 7 and the workspace at `fill`, a plausible share of every split."""
    nb = fmad.paged_attention_workspace_size(c.handle, b, H)
    assert nb > 0
    ws = torch.full((nb // 4,), fill, device="cuda")
    out = torch.full_like(q, 7.0)
    fmad.paged_attention(c.handle, 0, b, q, out, ws, causal=causal)
    return out, fmad.standalone_status()


def near(c, i, q, out, rows):
    """The entry's first `rows` rows are what its definition says."""
    ref, size = attention_ref(c, i, q, c.k.shape[-1] ** -0.5, True, 0)
    tol = ref.abs() * 2.0 ** -8 + size * ((2.0 ** -11 if c.fp8 else 2.0 ** -8) + 2.0 ** -9)
    assert bool(((out[:rows].double() - ref[:rows]).abs() <= tol[:rows]).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,new,H,bound", SPLIT)
def test_rows_behind_a_tight_bound_stay_as_they_were(lens, new, H, bound, fp8):
    require_gpu()
    c = Cache(lens, 64, 1, 128, fp8, seed=H)
    b = batch(c, new, lead=2, trail=3, max_tokens=bound)
    q = torch.randn((b.tokens, H, 128), device="cuda").to(torch.bfloat16)
    out, status = attend(c, b, q, H)
    assert status == 2
    start = b.start.tolist()
    assert (out[:start[0]] == 7).all() and (out[start[-1]:] == 7).all()
    for i, n in enumerate(new):
        near(c, i, q[start[i]:start[i + 1]], out[start[i]:start[i + 1]], min(n, bound))
        assert (out[start[i] + min(n, bound):start[i + 1]] == 7).all(), i


@pytest.mark.parametrize("lens,new,H,bound", SPLIT)
def test_rows_of_a_refused_entry_stay_as_they_were(lens, new, H, bound):
    require_gpu()
    lens, new = lens + [4000], new + [1]
    c = Cache(lens, 64, 1, 128, seed=H)
    for at in range(len(new)):
        for seq in (99, -1):
            ids = torch.tensor(np.asarray(c.rows), dtype=torch.int32, device="cuda")
            ids[at] = seq
            b = batch(c, new)
            b = fmad.KvBatch(b.start, b.tokens, max(new), max(lens), ids)
            q = torch.randn((b.tokens, H, 128), device="cuda").to(torch.bfloat16)
            out, status = attend(c, b, q, H)
            assert status == 2
            start = b.start.tolist()
            for i, n in enumerate(new):
                if i == at:
                    assert (out[start[i]:start[i + 1]] == 7).all()
                else:
                    near(c, i, q[start[i]:start[i + 1]], out[start[i]:start[i + 1]], n)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,new,H,bound", SPLIT)
def test_a_nan_query_row_is_not_hidden(lens, new, H, bound, fp8):
    """Every score of the row is NaN, so is its sum, and no split has a maximum: the row is NaN as it is without splits,
    and every other row keeps its bits."""
    require_gpu()
    c = Cache(lens, 64, 1, 128, fp8, seed=H)
    b = batch(c, new)
    q = torch.randn((b.tokens, H, 128), device="cuda").to(torch.bfloat16)
    clean, status = attend(c, b, q, H)
    assert status == 0
    token, head = b.tokens - 1, H - 1
    q[token, head, 5] = float("nan")
    out, status = attend(c, b, q, H)
    assert status == 0
    assert out[token, head].isnan().all()
    out[token, head] = clean[token, head]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,new,H", [([30], [1], 8), ([1500, 90], [1, 2], 8), ([260, 40], [12, 5], 8), ([700, 300], [300, 70], 8),
                                        ([4000, 300], [4000, 300], 8)])
def test_a_nan_query_row_in_shorter_calls(lens, new, H, fp8):
    """The same where one CTA or one cluster has all of a row's keys (all but the fourth), up to the widest row blocks."""
    require_gpu()
    c = Cache(lens, 16, 1, 64, fp8, seed=H)
    b = batch(c, new)
    nb = fmad.paged_attention_workspace_size(c.handle, b, H)
    assert (nb == 0) == (new[0] != 300)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    q = torch.randn((b.tokens, H, 64), device="cuda").to(torch.bfloat16)
    clean, out = torch.empty_like(q), torch.empty_like(q)
    fmad.paged_attention(c.handle, 0, b, q, clean, ws)
    token, head = b.tokens - 1, H - 1
    q[token, head, 5] = float("nan")
    fmad.paged_attention(c.handle, 0, b, q, out, ws)
    assert fmad.standalone_status() == 0
    assert out[token, head].isnan().all()
    out[token, head] = clean[token, head]
    assert torch.equal(out, clean)


def test_entries_times_splits_beyond_a_grid():
    """Thousands of entries under a very loose length bound: the call divides its keys less, it is not refused."""
    require_gpu()
    c = Cache([300, 41], 64, 2, 64, seed=3, rows=[0, 1])
    n, H = 4096, 16
    start = torch.arange(0, 3 * n + 1, 3, dtype=torch.int32, device="cuda")
    ids = torch.arange(n, dtype=torch.int32, device="cuda") % 2
    q = torch.randn((3 * n, H, 64), device="cuda").to(torch.bfloat16)
    b = fmad.KvBatch(start, 3 * n, 3, 1 << 29, ids)
    ws = torch.empty(fmad.paged_attention_workspace_size(c.handle, b, H), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    fmad.paged_attention(c.handle, 0, b, q, out, ws)
    assert fmad.standalone_status() == 0
    for i in (0, 1, 2047, 4094, 4095):
        near(c, i % 2, q[3 * i:3 * i + 3], out[3 * i:3 * i + 3], 3)
