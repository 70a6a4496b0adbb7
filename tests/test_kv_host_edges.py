"""The paged prefix cache's entry points at the ends of their ranges, on the host (nothing here launches a kernel)."""
import ctypes

import pytest

import flow_matching_action_denoise_gb300 as fmad
from test_kv_host import P, at, batch, cache, lib   # noqa: F401  (lib is a fixture)


@pytest.mark.parametrize("n", [300, 4096, 20000, 65535])
@pytest.mark.parametrize("H", [2, 4, 16, 64])
def test_any_number_of_entries_under_any_length_bound(lib, n, H):   # noqa: F811
    """A bound on the lengths that is far too large never makes a batch too large."""
    c, size = cache(seqs=70000), ctypes.c_size_t()
    for new in (1, 3, 9, 17, 100):
        for max_len in (1000, 10 ** 5, 1 << 20, 1 << 29, (1 << 31) - 1):
            b = batch(n=n, tokens=n * new, max_tokens=new, max_len=max_len)
            assert lib.fm_paged_attention_workspace_size(at(c), at(b), H, ctypes.byref(size)) == 0


@pytest.mark.parametrize("kw", [
    dict(pages=1 << 30, page_stride=(1 << 39) - 64, layers=3, layer_stride=(1 << 39) - 16),
    dict(pages=1 << 30, page_stride=(1 << 39) - 16, layers=3, layer_stride=(1 << 39) - 16),
    dict(pages=1 << 30, page_stride=1 << 34, layers=1), dict(page_stride=(1 << 63) - 8), dict(layer_stride=-(1 << 63)),
])
def test_strides_whose_products_leave_64_bits(lib, kw):   # noqa: F811
    size = ctypes.c_size_t()
    assert lib.fm_kv_workspace_size(at(cache(**kw)), 1, ctypes.byref(size)) == 2


def test_queries_rotated_in_place_keep_their_stride(lib):   # noqa: F811
    """With another stride a row would be written over one that is still to be read."""
    c, b, r = cache(), batch(), fmad.FmRope(P, 64, 0, 1.0)
    for qs, os_ in ((256, 264), (512, 256)):
        assert lib.fm_rope_append(at(c), 0, at(b), at(r), P, qs, 4, 2 * P, 128, 3 * P, 128, P, os_, None, None) == 2


def test_norm_rows_stored_in_place_keep_their_stride(lib):   # noqa: F811
    for xs, os_ in ((256, 264), (512, 256)):
        assert lib.fm_norm_quant(P, xs, 1, None, 0, None, 4, 256, 1e-6, P, os_, 2 * P, 3 * P, 0, None) == 2


def test_no_rotation_needs_no_table():
    none = fmad.Rope(0, device="cpu")
    assert none.struct.rotary_dim == 0 and none.freq.numel() == 0
    for dim in (8, -16, 272):
        with pytest.raises(fmad.FmError):
            fmad.Rope(dim, device="cpu")
