"""fm_test_paged_plan on the host: what it refuses, and that a plan is consistent with the workspace queries (no GPU: the plan
is then for the SM count of a GB300)."""
import ctypes

import pytest

import flow_matching_action_denoise_gb300 as fmad
from test_kv_host import BAD_CACHES, at, batch, cache, lib  # noqa: F401
from test_kv_host_shared import groups


def plan(lib, c=None, b=None, g=None, H=4, window=0, sinks=0):  # noqa: F811
    p, c, b = fmad.FmPagedPlan(*[77] * 6), c or cache(), b or batch()
    st = lib.fm_test_paged_plan(at(c), at(b), at(g) if g else None, H, window, sinks, ctypes.byref(p))
    return st, [getattr(p, n) for n, _ in p._fields_]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(lib, kw, status):  # noqa: F811
    assert plan(lib, c=cache(**kw)) == (status, [77] * 6)


def test_arguments(lib):  # noqa: F811
    c, b = cache(), batch()
    assert lib.fm_test_paged_plan(at(c), at(b), None, 4, 0, 0, None) == 1
    for kw in (dict(window=-1), dict(sinks=-1), dict(g=groups(), window=3), dict(g=groups(), sinks=3)):
        assert plan(lib, **kw)[0] == 1
    assert plan(lib, H=3)[0] == 2 and plan(lib, b=batch(n=-1))[0] == 2 and plan(lib, g=groups(n=-1))[0] == 2
    assert plan(lib, b=batch(tokens=0)) == (0, [0] * 6)


def test_plans_and_workspaces(lib):  # noqa: F811
    long = cache(table_stride=4096)
    for b, few, tiles in ((batch(n=1, tokens=1, max_tokens=1, max_len=60000), 1, 0), (batch(n=1, tokens=60, max_tokens=60, max_len=60000), 0, 1),
                          (batch(n=1, tokens=600, max_tokens=600, max_len=60000), 0, 2)):
        need = ctypes.c_size_t()
        assert lib.fm_paged_attention_workspace_size(at(long), at(b), 4, ctypes.byref(need)) == 0
        st, (f, t, splits, cluster, at_once, own) = plan(lib, long, b)
        assert st == 0 and (f, t, cluster, at_once, own) == (few, tiles, 0, 0, 0) and splits > 1
        assert need.value == splits * b.tokens * 4 * (64 * 4 + 8)
        # a window and first tokens: up to eight splits meet in a cluster, of which some fit at once
        st, (f, t, splits, cluster, at_once, own) = plan(lib, long, b, window=700, sinks=60)
        assert st == 0 and (f, t) == (few, tiles) and 1 < splits == cluster <= 8 and at_once > 0
    many = batch(n=96, tokens=96, max_tokens=1, max_len=16100)
    st, p = plan(lib, cache(table_stride=4096, seqs=100), many, groups(max_entries=96, max_shared=16000), 16)
    assert st == 0 and p[0] == 0 and p[2] > 1 and p[5] >= 1


def test_a_loose_bound_on_new_tokens_changes_no_plan(lib):  # noqa: F811
    """max_tokens counts up to the batch's tokens, as in the calls themselves."""
    long = cache(table_stride=4096)
    for kw in (dict(), dict(window=700, sinks=60)):
        tight = plan(lib, long, batch(n=1, tokens=3, max_tokens=3, max_len=60000), **kw)
        assert tight[0] == 0 and plan(lib, long, batch(n=1, tokens=3, max_tokens=1 << 29, max_len=60000), **kw)[1] == tight[1]
