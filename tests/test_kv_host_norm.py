"""fm_norm_rope_append refuses bad arguments on the host with the status codes of fm_rope_append and its own (no GPU:
nothing here launches a kernel)."""
import math

import pytest

import flow_matching_action_denoise_gb300 as fmad
from test_kv_host import BAD_CACHES, P, at, batch, cache, lib  # noqa: F401


def call(lib, c=None, b=None, rope=None, layer=0, q=P, qs=128, H=2, k=P, ks=128, v=P, vs=128, out=P, os_=128, qg=P, kg=P,  # noqa: F811
         eps=1e-6):
    c, b, rope = c or cache(), b or batch(), rope or fmad.FmRope(P, 16, 0, 1.0)
    return lib.fm_norm_rope_append(at(c), layer, at(b), at(rope), q, qs, H, k, ks, v, vs, out, os_, qg,
                                   kg, eps, None, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(lib, kw, status):  # noqa: F811
    assert call(lib, c=cache(**kw)) == status


def test_arguments(lib):  # noqa: F811
    for eps in (-1e-9, math.nan, math.inf):
        assert call(lib, eps=eps) == 1
    assert call(lib, qg=P + 2) == 3 and call(lib, kg=P + 1) == 3 and call(lib, q=P + 8) == 3
    assert call(lib, layer=2) == 1 and call(lib, H=-1) == 2 and call(lib, q=None) == 1 and call(lib, k=None) == 1
    assert call(lib, qs=120) == 2 and call(lib, ks=124) == 2 and call(lib, vs=64) == 2 and call(lib, os_=132) == 2
    assert call(lib, rope=fmad.FmRope(P, 80, 0, 1.0)) == 2 and call(lib, rope=fmad.FmRope(None, 16, 0, 1.0)) == 1
    assert call(lib, rope=fmad.FmRope(P, 16, 2, 1.0)) == 1 and call(lib, rope=fmad.FmRope(P, 16, 0, math.nan)) == 1
    for kw in (dict(n=-1), dict(tokens=-1), dict(max_tokens=-1), dict(n=70000), dict(seq=None, n=5)):
        assert call(lib, b=batch(**kw)) == 2
    # nothing to do: nothing is launched
    assert call(lib, b=batch(tokens=0)) == 0 and call(lib, b=batch(n=0)) == 0
