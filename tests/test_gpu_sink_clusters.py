"""Windows with first tokens whose splits meet in their cluster: the plan reaches every size of cluster, with one and with two
query tiles a CTA and in the kernel for few rows, and every one of them is right (tolerance: as in test_gpu_sink_attention.py)."""
import numpy as np
import pytest
import torch

import flow_matching_action_denoise_gb300 as fmad
from _gpu import require_gpu
from _kv import Cache, batch
from test_gpu_sink_attention import attend, check

pytestmark = pytest.mark.gpu

# query tiles, CTAs of a cluster, entries, new tokens, H, Hkv, window, first tokens
CHUNKS = [(1, 2, 10, 17, 4, 4, 200, 30), (1, 3, 10, 17, 4, 4, 500, 130), (1, 4, 1, 17, 4, 4, 200, 30), (1, 5, 1, 17, 4, 4, 900, 5),
          (1, 6, 1, 17, 4, 4, 1500, 300), (1, 7, 1, 128, 4, 4, 1100, 60), (1, 8, 1, 17, 4, 4, 500, 130), (2, 2, 8, 257, 8, 1, 500, 130),
          (2, 3, 10, 40, 12, 3, 200, 30), (2, 4, 6, 40, 12, 3, 500, 130), (2, 5, 1, 40, 12, 3, 200, 30), (2, 6, 1, 40, 12, 3, 1500, 300),
          (2, 7, 1, 257, 6, 6, 1500, 300), (2, 8, 1, 40, 12, 3, 500, 130)]


def ragged(most, n, seed, least=0):
    return [most] + [int(x) for x in np.random.default_rng(seed).integers(least, most + 1, n - 1)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("tiles,cluster,n,most,H,Hkv,window,sinks", CHUNKS)
def test_chunks(tiles, cluster, n, most, H, Hkv, window, sinks, Dh, fp8):
    require_gpu()
    lens = ragged(3000, n, cluster)
    new = [min(a, b) for a, b in zip(ragged(most, n, tiles), lens)]
    c = Cache(lens, 32, Hkv, Dh, fp8, seed=cluster)
    b = batch(c, new, True, 1, 1)
    plan = fmad.paged_plan(c.handle, b, H, window, sinks)
    assert (plan.few_rows, plan.row_tiles, plan.cluster, plan.splits) == (0, tiles, cluster, cluster)
    q, out, b = attend(c, new, H, window, sinks, lead=1, trail=1)
    check(c, new, q, out, b, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cluster,n", [(8, 20), (7, 35), (6, 40), (5, 50), (4, 65), (3, 80), (2, 120)])
def test_single_tokens(cluster, n, fp8):
    """16-bit rows of 128 dims: two CTAs an SM. With an E4M3 cache four, where twice as many entries meet in the same sizes."""
    require_gpu()
    n = 2 * n if fp8 else n
    lens = ragged(2900, n, cluster, 700)
    c = Cache(lens, 64, 1, 128, fp8, seed=cluster)
    new = [1] * n
    plan = fmad.paged_plan(c.handle, batch(c, new), 8, 2048, 64)
    assert (plan.few_rows, plan.cluster) == (1, cluster) and plan.clusters_at_once >= n
    q, out, b = attend(c, new, 8, 2048, 64)
    check(c, new, q, out, b, 2048, 64)


def test_the_plan_of_every_call():
    require_gpu()
    c = Cache([3000, 2000], 64, 2, 64, seed=1)
    b = batch(c, [40, 30])
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    plain, groups = fmad.paged_plan(c.handle, b, 8), fmad.paged_plan(c.handle, b, 8, groups=fmad.KvGroups(none, none[:0], 0, 0))
    assert plain.splits == groups.splits > 1 and plain.cluster == 0 and groups.cluster in (0, plain.splits)
    assert groups.own_splits == 0 and (plain.cluster == 0) == (fmad.paged_attention_workspace_size(c.handle, b, 8) > 0)
    # a window alone is fm_paged_attention, first tokens alone as well
    assert fmad.paged_plan(c.handle, b, 8, 0, 50).splits == plain.splits and fmad.paged_plan(c.handle, b, 8, 300, 0).cluster == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Dh", [64, 128])
def test_clusters_leave_places_free(Dh, fp8):
    """Single tokens' clusters all run at once, those of 2 and 4 CTAs with one place free, the others with a fourteenth of the
    places; and no smaller size is taken where the next one fits."""
    require_gpu()
    c = Cache([4096], 64, 1, Dh, fp8, seed=1)
    start, seq = torch.arange(401, dtype=torch.int32, device="cuda"), torch.zeros(400, dtype=torch.int32, device="cuda")
    plans = {n: fmad.paged_plan(c.handle, fmad.KvBatch(start[:n + 1], n, 1, 4096, seq[:n]), 8, 2048, 64) for n in range(1, 400)}
    places = {p.cluster: p.clusters_at_once for p in plans.values() if p.cluster}
    assert set(places) == set(range(2, 9))
    most = {s: r - 1 if s in (2, 4) else r * 13 // 14 for s, r in places.items()}
    for n, p in plans.items():
        assert p.splits == max([s for s in most if n <= most[s]] + [1]), n
