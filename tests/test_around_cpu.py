"""The operators around the indexer without a GPU: what their entry points refuse before any HIP call, and the
frequency helper."""
import ctypes

import numpy as np
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
    base = dict(data=F, ld_t=H * D, ld_h=D, dtype=dtype, T=T, H=H, D=D)
    return idx.idx_rows(**(base | kw))


def _rotary(**kw):
    return idx.idx_rotary(**(dict(freq=F, pos=F, rot=64, rot0=0, layout=0, inverse=0, mscale=1.0) | kw))


def _cache(rows=100, H=8, D=128, fmt=FP8, **kw):
    per = {FP8: H, FP4: H * D // 32}.get(fmt, 0)
    return idx.idx_cache(**(dict(data=F, scale=F if per else None, rows=rows, ld=H * D, ld_scale=per, fmt=fmt, H=H,
                                 D=D) | kw))


def test_rope_refusals(lib):
    rope = lambda x=None, r=None, o=None: lib.idx_rope(x or _rows(), r or _rotary(), o or _rows(data=2 * F), None)
    assert lib.idx_rope(None, _rotary(), _rows(), None) == NULL
    assert rope(x=_rows(data=None)) == NULL
    assert rope(r=_rotary(freq=None)) == NULL and rope(r=_rotary(pos=None)) == NULL
    assert rope(x=_rows(T=-1)) == SHAPE and rope(o=_rows(T=3)) == SHAPE and rope(o=_rows(H=4)) == SHAPE
    assert rope(x=_rows(D=100), o=_rows(D=100)) == UNSUPPORTED
    assert rope(x=_rows(D=520), o=_rows(D=520)) == UNSUPPORTED
    assert rope(x=_rows(dtype=FP8)) == FORMAT and rope(x=_rows(dtype=9)) == FORMAT
    assert rope(o=_rows(dtype=F16)) == FORMAT
    for bad in (dict(rot=0), dict(rot=-8), dict(rot=60), dict(rot=136), dict(rot0=4), dict(rot0=72), dict(rot0=-8),
                dict(rot0=2 ** 31 - 8)):
        assert rope(r=_rotary(**bad)) == SHAPE, bad
    assert rope(r=_rotary(layout=2)) == FORMAT and rope(r=_rotary(mscale=float("nan"))) == PARAM
    assert rope(x=_rows(data=F + 8)) == ALIGN and rope(x=_rows(ld_h=132)) == ALIGN and rope(x=_rows(ld_t=1028)) == ALIGN
    assert rope(r=_rotary(freq=F + 4)) == ALIGN and rope(r=_rotary(pos=F + 2)) == ALIGN
    assert rope(x=_rows(ld_t=-1024)) == SHAPE
    # outputs whose rows share memory, and in place with other strides
    assert rope(o=_rows(data=2 * F, ld_h=0)) == SHAPE and rope(o=_rows(data=2 * F, ld_t=512)) == SHAPE
    assert rope(o=_rows(ld_t=2048)) == SHAPE
    many = dict(T=2 ** 24, H=8, ld_t=1024)                              # 2^27 rows of 16 lanes
    assert rope(x=_rows(**many), o=_rows(data=2 * F, **many)) == UNSUPPORTED
    most = dict(T=2 ** 31 - 1, H=2 ** 28, ld_t=0, ld_h=0)               # rows that share memory
    assert rope(x=_rows(**most), o=_rows(data=2 * F)) == SHAPE
    assert rope(x=_rows(T=0, data=None), o=_rows(T=0, data=None)) == OK
    assert rope(x=_rows(H=0, data=None), o=_rows(H=0, data=None)) == OK


def test_write_refusals(lib):
    def write(x=None, c=None, r=None, slot=F, n=1):
        w = (idx.idx_write * 1)(idx.idx_write(x=x or _rows(), slot=slot, to=c or _cache()))
        if r is not None:
            w[0].rotary = ctypes.pointer(r)
        return lib.idx_cache_write(w, n, None)
    assert lib.idx_cache_write(None, 1, None) == NULL and lib.idx_cache_write(None, 0, None) == OK
    assert write(n=9) == PARAM and write(n=-1) == PARAM
    assert write(c=_cache(data=None)) == NULL and write(c=_cache(scale=None)) == NULL
    assert write(c=_cache(fmt=5)) == FORMAT
    assert write(c=_cache(H=4)) == SHAPE and write(c=_cache(D=64)) == SHAPE
    assert write(c=_cache(rows=3), slot=None) == SHAPE                 # rows 0 .. 3 to three slots
    assert write(c=_cache(ld=512)) == SHAPE and write(c=_cache(ld_scale=7)) == SHAPE
    assert write(c=_cache(rows=-1)) == SHAPE and write(c=_cache(rows=2 ** 31)) == SHAPE
    assert write(x=_rows(D=72), c=_cache(D=72, fmt=FP4)) == UNSUPPORTED
    assert write(c=_cache(data=F + 4)) == ALIGN and write(c=_cache(scale=F + 2)) == ALIGN
    assert write(c=_cache(ld=1028)) == ALIGN and write(slot=F + 2) == ALIGN
    assert write(r=_rotary(rot=136)) == SHAPE and write(r=_rotary(pos=None)) == NULL
    assert write(x=_rows(T=0, data=None)) == OK
    assert write(c=_cache(rows=0, data=None, scale=None)) == OK        # no slot to write
    eight = (idx.idx_write * 8)(*[idx.idx_write(x=_rows(T=2 ** 21), slot=F, to=_cache()) for _ in range(8)])
    assert lib.idx_cache_write(eight, 8, None) == UNSUPPORTED           # 2^31 lanes together


def test_read_refusals(lib):
    read = lambda c=None, o=None, at=F: lib.idx_cache_read(c or _cache(), at, o or _rows(), None)
    assert lib.idx_cache_read(None, F, _rows(), None) == NULL
    assert read(o=_rows(H=4)) == SHAPE and read(o=_rows(D=64)) == SHAPE and read(o=_rows(dtype=FP8)) == FORMAT
    assert read(c=_cache(scale=None)) == NULL and read(at=F + 1) == ALIGN and read(o=_rows(data=F + 2)) == ALIGN
    assert read(o=_rows(ld_h=0)) == SHAPE
    assert read(o=_rows(T=0, data=None)) == OK


def _attn(**kw):
    base = dict(q=_rows(T=2, H=16), out=_rows(T=2, H=16, data=2 * F), k=_cache(), v=_cache(), sel=F, ld_sel=64000,
                n_sel=64000, pool=1, ks=None, ke=None, slot_of_key=None, L=100, scale=0.1, lse=None)
    return idx.idx_attn(**(base | kw))


def test_attn_refusals(lib):
    n = ctypes.c_size_t(99)
    size = lambda **kw: lib.idx_sparse_attn_workspace(_attn(**kw), n)
    assert size() == OK and n.value > 0
    assert lib.idx_sparse_attn_workspace(_attn(), None) == NULL and lib.idx_sparse_attn_workspace(None, n) == NULL
    r = lambda **kw: _rows(**(dict(T=2, H=16) | kw))
    for status, bad in [
            (SHAPE, dict(q=r(T=3))), (SHAPE, dict(out=r(H=8))), (SHAPE, dict(k=_cache(H=4))),
            (SHAPE, dict(k=_cache(H=5), v=_cache(H=5))), (SHAPE, dict(v=_cache(rows=99))),
            (SHAPE, dict(k=_cache(D=64))), (SHAPE, dict(k=_cache(ld=2048))), (SHAPE, dict(v=_cache(ld_scale=16))),
            (UNSUPPORTED, dict(k=_cache(ld=2 ** 31), v=_cache(ld=2 ** 31))), (SHAPE, dict(n_sel=-1)), (SHAPE, dict(ld_sel=63999)), (SHAPE, dict(L=101)),
            (SHAPE, dict(L=-1)), (FORMAT, dict(q=r(dtype=F32), out=r(dtype=F32))), (FORMAT, dict(out=r(dtype=F16))),
            (FORMAT, dict(k=_cache(fmt=BF16))), (UNSUPPORTED, dict(k=_cache(fmt=F16), v=_cache(fmt=F16))),
            (UNSUPPORTED, dict(k=_cache(fmt=FP4), v=_cache(fmt=FP4))),
            (UNSUPPORTED, dict(q=r(D=96), out=r(D=96), k=_cache(D=96), v=_cache(D=96))),
            (UNSUPPORTED, dict(pool=3, ks=F, ke=F)), (UNSUPPORTED, dict(pool=0)), (UNSUPPORTED, dict(pool=128, ks=F, ke=F)),
            (UNSUPPORTED, dict(q=r(T=2 ** 25), out=r(T=2 ** 25))), (PARAM, dict(scale=3e38)), (PARAM, dict(scale=float("inf"))), (NULL, dict(ks=F)), (NULL, dict(pool=8)), (NULL, dict(sel=None)),
            (NULL, dict(q=r(data=None))), (ALIGN, dict(sel=F + 2)), (ALIGN, dict(lse=F + 1)),
            (ALIGN, dict(k=_cache(ld=1032), v=_cache(ld=1032))), (ALIGN, dict(ks=F + 1, ke=F)), (ALIGN, dict(slot_of_key=F + 3)), (ALIGN, dict(q=r(data=F + 8)))]:
        assert size(**bad) == status, bad
        assert lib.idx_sparse_attn(_attn(**bad), F, 1 << 30, None) == status, bad
    assert size(slot_of_key=F, L=1 << 20) == OK
    assert size() == OK
    assert lib.idx_sparse_attn(_attn(), None, 0, None) == NULL
    assert lib.idx_sparse_attn(_attn(), F, n.value - 1, None) == WORKSPACE
    assert lib.idx_sparse_attn(_attn(), F + 16, n.value, None) == ALIGN
    empty = dict(q=r(T=0, data=None), out=r(T=0, data=None))
    assert size(**empty) == OK and n.value == 0
    assert lib.idx_sparse_attn(_attn(**empty), None, 0, None) == OK


def test_freq_refusals(lib):
    f, m = (ctypes.c_double * 64)(), ctypes.c_double()
    call = lambda rot=64, base=1e4, kind=0, factor=2.0, orig=4096.0, fast=32.0, slow=1.0: lib.idx_rope_freqs(
        rot, base, kind, factor, orig, fast, slow, f, m)
    assert call() == OK and m.value == 1.0
    assert lib.idx_rope_freqs(64, 1e4, 0, 1.0, 1.0, 1.0, 1.0, None, m) == NULL
    assert call(rot=0) == SHAPE and call(rot=63) == SHAPE and call(rot=514) == SHAPE and call(rot=2, kind=2) == SHAPE
    assert call(base=1.0) == PARAM and call(base=float("nan")) == PARAM and call(kind=4) == FORMAT
    assert call(kind=1, factor=0.5) == PARAM and call(kind=3, orig=0.0) == PARAM
    assert call(kind=3, fast=1.0, slow=2.0) == PARAM and call(kind=3, slow=0.0) == PARAM


def test_freqs_against_formulas():
    i = np.arange(32)
    plain = 10000.0 ** (-2.0 * i / 64)
    f, m = idx.idx_rope_freqs(64)
    np.testing.assert_allclose(f.numpy(), plain, rtol=1e-13)
    assert m == 1.0
    f, _ = idx.idx_rope_freqs(64, scaling=idx.IDX_ROPE_LINEAR, factor=4.0)
    np.testing.assert_allclose(f.numpy(), plain / 4, rtol=1e-13)
    f, _ = idx.idx_rope_freqs(64, scaling=idx.IDX_ROPE_BASE, factor=4.0)
    np.testing.assert_allclose(f.numpy(), (10000.0 * 4 ** (64 / 62)) ** (-2.0 * i / 64), rtol=1e-12)
    f, m = idx.idx_rope_freqs(64, scaling=idx.IDX_ROPE_PARTS, factor=16.0, original=4096.0)
    where = lambda b: 64 * np.log(4096 / (b * 2 * np.pi)) / (2 * np.log(10000.0))
    lo, hi = np.floor(where(32.0)), np.ceil(where(1.0))
    r = np.clip((i - lo) / (hi - lo), 0, 1)
    np.testing.assert_allclose(f.numpy(), plain * (1 - r) + plain / 16 * r, rtol=1e-12)
    assert abs(m - (0.1 * np.log(16.0) + 1)) < 1e-15


def test_binding_refuses_tensors_off_the_gpu():
    """The binding's own checks: tensors on the CPU, and formats and shapes that do not fit."""
    x, pos = torch.zeros((2, 4, 128), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        idx.Rotary(torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="on the GPU"):
        idx.Cache(torch.zeros((4, 1, 128), dtype=torch.uint8), torch.ones((4, 1)))
    with pytest.raises(ValueError, match="unknown cache format"):
        idx.Cache(torch.zeros((4, 1, 128), dtype=torch.uint8), fmt=7)
    with pytest.raises(ValueError, match="on the GPU"):
        idx._rows(x, "x")
    with pytest.raises(ValueError, match="at most 8"):
        idx.idx_cache_write([None] * 9)
    assert idx.idx_cache_write([]) is None
    with pytest.raises(idx.IdxError):
        idx.idx_rope_freqs(63)


def test_binding_refuses_rows_that_require_a_gradient():
    """No entry point records a gradient: a call that would drop one without a word is an error, unless autograd
    is off."""
    x = torch.zeros((2, 4, 128), dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError, match="requires a gradient"):
        idx._rows(x, "x")
    with pytest.raises(ValueError, match="requires a gradient"):
        idx._rows(x * 2, "x")
    for quiet in (torch.no_grad, torch.inference_mode):
        with quiet(), pytest.raises(ValueError, match="on the GPU"):
            idx._rows(x, "x")


def _workgroups_of_a_row(lib, T, H, G, n=2048, L=4000, fmt=FP8, D=128):
    """Workgroups that a row's list is divided over, from the workspace that joins them (1: no workspace), for rows of
    16 heads a wave on caches of `T` requests."""
    bytes_ = ctypes.c_size_t()
    cache = _cache(rows=T * L, H=H, D=D, fmt=fmt)
    a = _attn(q=_rows(T=T, H=H * G, D=D), out=_rows(T=T, H=H * G, D=D, data=2 * F), k=cache, v=cache, n_sel=n, ld_sel=n,
              L=T * L)
    assert lib.idx_sparse_attn_workspace(a, bytes_) == OK
    part = T * H * -(-G // 16) * 16 * (D + 4) * 4
    assert bytes_.value % part == 0
    return max(bytes_.value // part, 1)


def test_lists_are_divided_by_the_work_there_is(lib):
    """How a list is divided goes by the items (rows x cache heads x blocks of 16 heads), not by which of the three they
    come from, and changes at few sizes."""
    of = lambda *a, **kw: _workgroups_of_a_row(lib, *a, **kw)
    assert of(128, 1, 16) == of(16, 8, 4) == of(32, 1, 64) == of(64, 1, 32) == 2
    assert of(64, 1, 16) == of(8, 8, 4) == of(16, 1, 64) == 4
    for H in (4, 8, 16):                 # past the number of CUs, from memory
        assert {of(T, H, 4) for T in range(272 // H, 384 // H + 1)} == {4}, H
        assert {of(T, H, 4, n=512) for T in range(272 // H, 384 // H + 1)} == {1}, H
        assert {of(T, H, 4) for T in range(144 // H, 256 // H + 1)} == {1}, H
    assert {of(T, 1, 16) for T in range(129, 500)} == {1}
    counts = [of(T, 8, 4) for T in range(1, 97)]
    assert sum(a != b for a, b in zip(counts[15:], counts[16:])) == 3   # 2, 1, 4, 1
