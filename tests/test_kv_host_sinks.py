"""fm_sink_attention refuses bad arguments on the host (no GPU: nothing here launches a kernel)."""
import math

import pytest

from test_kv_host import BAD_CACHES, P, at, batch, cache, lib  # noqa: F401


def call(lib, c=None, b=None, layer=0, q=P, qs=256, H=4, scale=0.1, window=9, sinks=4, out=P, os_=256, ws=P, nb=1 << 40):  # noqa: F811
    c, b = c or cache(), b or batch()
    return lib.fm_sink_attention(at(c), layer, at(b), q, qs, H, scale, 1, window, sinks, out, os_, ws, nb, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(lib, kw, status):  # noqa: F811
    assert call(lib, c=cache(**kw)) == status


def test_arguments(lib):  # noqa: F811
    assert call(lib, sinks=-1) == 1 and call(lib, window=-1) == 1 and call(lib, window=0, sinks=-5) == 1
    assert call(lib, layer=2) == 1 and call(lib, q=None) == 1 and call(lib, out=None) == 1
    assert call(lib, H=3) == 2 and call(lib, H=0) == 2
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(lib, scale=s) == 1
    assert call(lib, qs=248) == 2 and call(lib, os_=260) == 2 and call(lib, q=P + 8) == 3
    for kw in (dict(n=-1), dict(tokens=-1), dict(max_tokens=-1), dict(n=70000), dict(seq=None, n=5)):
        assert call(lib, b=batch(**kw)) == 2
    # both stretches are long: the keys are split, as far as the workspace query says and no further
    far = dict(table_stride=1 << 20)
    assert call(lib, c=cache(**far), b=batch(max_len=1 << 20), window=1 << 19, sinks=1 << 18, nb=8) == 4
    assert call(lib, b=batch(tokens=0)) == 0 and call(lib, b=batch(n=0)) == 0
