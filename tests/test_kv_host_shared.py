"""fm_shared_attention refuses bad arguments on the host (no GPU: nothing here launches a kernel)."""
import ctypes
import math

import pytest

import flow_matching_action_denoise_gb300 as fmad
from test_kv_host import BAD_CACHES, P, at, batch, cache, lib  # noqa: F401


def groups(**kw):
    g = fmad.FmKvGroups(first=P, shared=P, n=1, max_entries=2, max_shared=90)
    for k, v in kw.items():
        setattr(g, k, v)
    return g


def call(lib, c=None, b=None, g=None, layer=0, q=P, qs=256, H=4, scale=0.1, out=P, os_=256, ws=P, nb=1 << 40):  # noqa: F811
    c, b, g = c or cache(), b or batch(), g or groups()
    return lib.fm_shared_attention(at(c), layer, at(b), at(g), q, qs, H, scale, 1, out, os_, ws, nb, None)


def size(lib, c=None, b=None, g=None, H=4):  # noqa: F811
    n = ctypes.c_size_t(77)
    c, b, g = c or cache(), b or batch(), g or groups()
    return lib.fm_shared_attention_workspace_size(at(c), at(b), at(g), H, ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(lib, kw, status):  # noqa: F811
    assert call(lib, c=cache(**kw)) == status and size(lib, c=cache(**kw)) == (status, 77)


def test_arguments(lib):  # noqa: F811
    assert call(lib, layer=2) == 1 and call(lib, q=None) == 1 and call(lib, out=None) == 1
    assert call(lib, H=3) == 2 and call(lib, H=0) == 2 and size(lib, H=3) == (2, 77)
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(lib, scale=s) == 1
    assert call(lib, qs=248) == 2 and call(lib, os_=260) == 2 and call(lib, q=P + 8) == 3
    for kw in (dict(n=-1), dict(tokens=-1), dict(max_tokens=-1), dict(n=70000), dict(seq=None, n=5)):
        assert call(lib, b=batch(**kw)) == 2 and size(lib, b=batch(**kw)) == (2, 77)
    for kw, st in ((dict(n=-1), 2), (dict(n=65536), 2), (dict(max_entries=-1), 2), (dict(max_shared=-1), 2), (dict(first=None), 1),
                   (dict(shared=None), 1)):
        assert call(lib, g=groups(**kw)) == st and size(lib, g=groups(**kw)) == (st, 77)
    c, b = cache(), batch()
    assert lib.fm_shared_attention(at(c), 0, at(b), None, P, 256, 4, 0.1, 1, P, 256, P, 1 << 40, None) == 1
    assert lib.fm_shared_attention_workspace_size(at(c), at(b), at(groups()), 4, None) == 1
    assert call(lib, b=batch(tokens=0)) == 0 and call(lib, b=batch(n=0)) == 0


def test_workspace(lib):  # noqa: F811
    """Sharing needs a place for the prefixes' shares; few entries, few shared tokens or no groups need none."""
    c = cache(table_stride=1024)
    many = dict(n=96, tokens=96, max_tokens=1, max_len=16100, seq=P)
    c.seqs = 100
    assert size(lib, c, batch(**many), groups(max_entries=96, max_shared=30), 16) == (0, 0)
    assert size(lib, c, batch(**many), groups(max_entries=96, max_shared=0), 16) == (0, 0)
    assert size(lib, c, batch(**many), groups(n=0, first=None, shared=None), 16) == (0, 0)
    g = groups(max_entries=96, max_shared=16000)
    st, need = size(lib, c, batch(**many), g, 16)
    share = 96 * 16 * (64 * 4 + 8)
    assert st == 0 and need > 0 and need % share == 0 and need // share <= 64
    kw = dict(c=c, b=batch(**many), g=g, H=16, qs=1024, os_=1024)
    assert call(lib, nb=need - 1, **kw) == 4 and call(lib, ws=None, **kw) == 1 and call(lib, ws=P + 8, **kw) == 3
    # sizes at their limits: no overflow on the way to a plan
    big = dict(n=65535, tokens=2 ** 31 - 1, max_tokens=2 ** 31 - 1, max_len=2 ** 31 - 1, seq=P)
    assert size(lib, c, batch(**big), groups(n=65535, max_entries=2 ** 31 - 1, max_shared=2 ** 31 - 1), 2)[0] in (0, 2)
    big.update(max_tokens=1)
    assert size(lib, c, batch(**big), groups(n=65535, max_entries=2 ** 31 - 1, max_shared=2 ** 31 - 1), 2)[0] == 0
