"""Attention over paged caches and the RMS norm without a GPU: what their entry points refuse before any HIP call."""
import ctypes

import pytest
import torch

import mqa_logits_top_amd as idx

OK, NULL, SHAPE, PARAM, FORMAT, WORKSPACE, UNSUPPORTED, ALIGN = 0, 1, 2, 3, 4, 5, 6, 8
F = 1 << 20          # 16-byte aligned, never dereferenced: every call here fails host checks or has no rows
FP8, FP4, BF16, F16, F32 = range(5)


@pytest.fixture(scope="module")
def lib():
    return idx.load_library()


def _rows(T=4, H=8, D=128, dtype=BF16, **kw):
    return idx.idx_rows(**(dict(data=F, ld_t=H * D, ld_h=D, dtype=dtype, T=T, H=H, D=D) | kw))


def _cache(rows=128, H=2, D=128, fmt=BF16, **kw):
    per = {FP8: H, FP4: H * D // 32}.get(fmt, 0)
    return idx.idx_cache(**(dict(data=F, scale=F if per else None, rows=rows, ld=H * D, ld_scale=per, fmt=fmt, H=H,
                                 D=D) | kw))


def _paged(**kw):
    base = dict(q=_rows(), out=_rows(data=2 * F), k=_cache(), v=_cache(), pages=F, ld_pages=4, n_pages=4, page=16, cu_q=F,
                len_k=F, B=2, window=0, first=0, scale=0.1, lse=F)
    return idx.idx_paged(**(base | kw))


def test_paged_refusals(lib):
    n = ctypes.c_size_t()
    size = lambda **kw: lib.idx_paged_attn_workspace(_paged(**kw), ctypes.byref(n))

    def both(want, **kw):
        assert size(**kw) == want, kw
        if want:
            assert lib.idx_paged_attn(_paged(**kw), F, 1 << 40, None) == want, kw

    assert lib.idx_paged_attn(None, F, 1 << 40, None) == NULL
    assert lib.idx_paged_attn_workspace(None, ctypes.byref(n)) == NULL
    assert lib.idx_paged_attn_workspace(_paged(), None) == NULL
    both(OK)
    for a in ("cu_q", "len_k", "pages"):
        both(NULL, **{a: None})
        both(ALIGN, **{a: F + 2})
    both(ALIGN, lse=F + 2)
    both(OK, lse=None)
    both(NULL, q=_rows(data=None))
    both(NULL, out=_rows(data=None))
    both(NULL, k=_cache(data=None))
    both(SHAPE, out=_rows(T=3)), both(SHAPE, out=_rows(H=4)), both(SHAPE, q=_rows(H=7), out=_rows(H=7))
    both(SHAPE, k=_cache(H=4)), both(SHAPE, k=_cache(rows=64)), both(SHAPE, k=_cache(ld=512))
    both(SHAPE, k=_cache(D=64), v=_cache(D=64))
    both(SHAPE, B=-1), both(SHAPE, n_pages=-1), both(SHAPE, ld_pages=3), both(SHAPE, ld_pages=-1)
    both(OK, ld_pages=0, B=1)
    both(FORMAT, q=_rows(dtype=F32), out=_rows(dtype=F32)), both(FORMAT, out=_rows(dtype=F16))
    both(FORMAT, v=_cache(fmt=FP8))
    both(UNSUPPORTED, k=_cache(fmt=F16), v=_cache(fmt=F16)), both(UNSUPPORTED, k=_cache(fmt=FP4), v=_cache(fmt=FP4))
    both(OK, k=_cache(fmt=FP8), v=_cache(fmt=FP8))
    d = dict(D=256)
    both(UNSUPPORTED, q=_rows(**d), out=_rows(**d), k=_cache(**d), v=_cache(**d))
    for page in (0, -16, 3, 24, -2 ** 31):
        both(UNSUPPORTED, page=page)
    both(UNSUPPORTED, page=1 << 30, n_pages=2)
    both(OK, page=1 << 30, n_pages=1)
    both(UNSUPPORTED, page=1 << 20, n_pages=1 << 11, ld_pages=1 << 11)
    both(UNSUPPORTED, B=(1 << 16) + 1)
    heads = dict(H=1 << 8, ld_t=1 << 15)
    both(UNSUPPORTED, B=1 << 16, q=_rows(**heads), out=_rows(data=2 * F, **heads), k=_cache(H=1 << 8), v=_cache(H=1 << 8))
    both(UNSUPPORTED, q=_rows(T=1 << 23), out=_rows(T=1 << 23))
    both(PARAM, window=-1), both(PARAM, first=-1), both(PARAM, scale=float("nan")), both(PARAM, scale=float("inf"))
    both(PARAM, scale=3e38)
    both(ALIGN, q=_rows(data=F + 8)), both(ALIGN, q=_rows(ld_t=1028)), both(ALIGN, k=_cache(data=F + 8))
    both(ALIGN, k=_cache(ld=264, fmt=FP8), v=_cache(ld=264, fmt=FP8))
    # nothing to do
    assert lib.idx_paged_attn(_paged(q=_rows(T=0, data=None), out=_rows(T=0, data=None)), None, 0, None) == OK
    assert lib.idx_paged_attn(_paged(B=0, cu_q=None, len_k=None, pages=None), None, 0, None) == OK


def test_paged_workspace_refusals(lib):
    n = ctypes.c_size_t()
    a = _paged(page=64, n_pages=1024, ld_pages=1024)
    assert lib.idx_paged_attn_workspace(a, ctypes.byref(n)) == OK
    if n.value:
        assert lib.idx_paged_attn(a, None, n.value, None) == NULL
        assert lib.idx_paged_attn(a, F, n.value - 1, None) == WORKSPACE
        assert lib.idx_paged_attn(a, F + 16, n.value, None) == ALIGN


def _norm(**kw):
    base = dict(x=_rows(), residual=_rows(data=None), total=_rows(data=None), out=_rows(data=2 * F), weight=F,
                weight_dtype=BF16, eps=1e-6)
    to = kw.pop("to", None)
    n = idx.idx_norm(**(base | kw))
    if to is not None:
        n.to = ctypes.pointer(to)
    return n


def test_norm_refusals(lib):
    call = lambda **kw: lib.idx_rms_norm(_norm(**kw), None)
    none = dict(out=_rows(data=None))
    assert lib.idx_rms_norm(None, None) == NULL
    assert call(x=_rows(data=None)) == NULL and call(**none) == NULL
    assert call(x=_rows(T=0)) == OK and call(x=_rows(H=0)) == OK
    assert call(x=_rows(T=-1)) == SHAPE and call(out=_rows(T=3)) == SHAPE and call(out=_rows(D=64, data=2 * F)) == SHAPE
    wide = lambda D, **kw: _rows(H=1, D=D, **kw)
    assert call(x=wide(100), out=wide(100, data=2 * F)) == UNSUPPORTED
    assert call(x=wide(32776), out=wide(32776, data=2 * F)) == UNSUPPORTED
    assert call(x=_rows(dtype=FP8)) == FORMAT and call(weight_dtype=FP4) == FORMAT and call(out=_rows(dtype=9)) == FORMAT
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == PARAM
    assert call(weight=F + 8) == ALIGN and call(x=_rows(data=F + 8)) == ALIGN and call(out=_rows(ld_t=1028)) == ALIGN
    many = dict(T=1 << 25, H=8)
    assert call(x=_rows(**many), out=_rows(data=2 * F, **many)) == UNSUPPORTED
    # the residual and its sum
    r, t = _rows(data=3 * F, dtype=F32), _rows(data=4 * F, dtype=F32)
    assert call(residual=r) == SHAPE or call(residual=r) == NULL
    assert call(residual=r, total=_rows(data=4 * F)) == FORMAT
    assert call(residual=_rows(T=3, data=3 * F), total=_rows(data=4 * F)) == SHAPE
    assert call(residual=r, total=_rows(data=4 * F, dtype=F32, ld_h=0)) == SHAPE
    assert call(residual=r, total=_rows(data=2 * F, dtype=F32)) == SHAPE          # out's place
    assert call(residual=r, total=_rows(data=3 * F, dtype=F32, ld_t=2048)) == SHAPE
    assert call(residual=r, total=_rows(data=F, dtype=F32)) == SHAPE              # over x, of another width
    assert call(residual=r, total=t, out=_rows(data=3 * F)) == SHAPE              # over the residual, of another width
    assert call(out=_rows(data=F, ld_t=2048)) == SHAPE
    # codes
    to = lambda **kw: _cache(**(dict(fmt=FP8, H=8) | kw))
    assert call(to=to(fmt=BF16)) == UNSUPPORTED and call(to=to(fmt=FP4)) == UNSUPPORTED and call(to=to(fmt=7)) == FORMAT
    assert call(to=to(H=4)) == SHAPE and call(to=to(D=64)) == SHAPE and call(to=to(rows=3)) == SHAPE
    assert call(to=to(data=None)) == NULL and call(to=to(scale=None)) == NULL and call(to=to(data=F + 8)) == ALIGN
    assert call(to=to(ld=512)) == SHAPE
    one = dict(x=wide(1536), out=wide(1536, data=2 * F))
    assert call(to=to(H=16, D=96), **one) == UNSUPPORTED and call(to=to(H=1, D=1024), **one) == SHAPE
    two = dict(x=wide(2048), out=wide(2048, data=2 * F))
    assert call(to=to(H=2, D=1024), **two) == UNSUPPORTED


def test_binding_refuses_tensors_without_a_gpu():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        idx.idx_rms_norm(x)
    with pytest.raises(ValueError):
        idx.idx_rms_norm(x, total=x)
    with pytest.raises(ValueError):
        idx.idx_rms_norm(x.clone().requires_grad_())
