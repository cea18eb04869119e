"""What attention over a paged cache refuses at the ends of its ranges, before any HIP call."""
import ctypes

import pytest

import mqa_logits_top_amd as idx
from test_dense_cpu import BF16, FP8, UNSUPPORTED, OK, SHAPE, F, _cache, _paged, _rows


@pytest.mark.parametrize("fmt", [FP8, BF16])
@pytest.mark.parametrize("heads", [(1 << 20) - 8, (1 << 21) - 8, 1 << 21, (1 << 21) + 8, 1 << 22])
def test_launches_rounded_up_to_eight_items_stay_below_2_32_lanes(heads, fmt):
    """One token of so many cache heads: E4M3 launches have workgroups of 256 lanes for 8 items of each head."""
    lib, n = idx.load_library(), ctypes.c_size_t()
    wide = dict(T=1, H=heads, D=64, ld_t=heads * 64, ld_h=64)
    a = _paged(q=_rows(**wide), out=_rows(data=2 * F, **wide), k=_cache(rows=16, H=heads, D=64, fmt=fmt),
               v=_cache(rows=16, H=heads, D=64, fmt=fmt), B=1, n_pages=1, ld_pages=1)
    fits = fmt == BF16 or 8 * heads * 256 < 1 << 32
    assert lib.idx_paged_attn_workspace(a, ctypes.byref(n)) == (OK if fits else UNSUPPORTED)
    if not fits:
        assert lib.idx_paged_attn(a, F, 1 << 40, None) == UNSUPPORTED


def test_results_in_the_queries_place_lie_as_they_do():
    lib, n = idx.load_library(), ctypes.c_size_t()
    size = lambda q, out: lib.idx_paged_attn_workspace(_paged(q=q, out=out), ctypes.byref(n))
    assert size(_rows(), _rows()) == OK and size(_rows(ld_t=2048), _rows(ld_t=2048)) == OK
    assert size(_rows(ld_t=2048), _rows()) == SHAPE and size(_rows(), _rows(ld_t=2048)) == SHAPE
    assert lib.idx_paged_attn(_paged(q=_rows(), out=_rows(ld_t=2048)), F, 1 << 40, None) == SHAPE
    one = dict(T=1)
    assert size(_rows(ld_t=2048, **one), _rows(**one)) == OK
