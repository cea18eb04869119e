"""RMS norm with the residual's addition and E4M3 output against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import mqa_logits_top_amd as idx
from around_ref import HALF_STEP, SMALLEST, quantise_e4m3, read_e4m3
from dense_ref import norm_bound, rms_norm

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FP8 = idx.IDX_K_FP8_E4M3


def data(seed, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * gain).to(dtype)


def f64(x):
    return None if x is None else x.cpu().double().numpy()


def check(x, w=None, eps=1e-6, residual=None, group=0, out_dtype=None, with_out=True, **kw):
    """One call against the formula: values, sum, codes and scales."""
    T, N = x.shape[0], x[0].numel() if x.shape[0] else 0
    r = None if residual is None else residual.cuda()
    total = None if r is None else torch.full_like(r, 5.0)
    to = idx.Cache.empty(T, N // group, group) if group else None
    out = None if out_dtype is None else torch.zeros(x.shape, dtype=out_dtype, device="cuda")
    y = idx.idx_rms_norm(x.cuda(), None if w is None else w.cuda(), eps=eps, residual=r, total=total, out=out, to=to,
                         with_out=with_out, **kw)
    h, want = rms_norm(f64(x), f64(residual), f64(w), eps)
    off = norm_bound(h, want, x.shape[-1], residual is not None)
    if residual is not None:
        err = np.abs(f64(total) - h)
        assert (err <= (HALF_STEP[r.dtype] + 2.0 ** -23) * np.abs(h) + SMALLEST[r.dtype]).all(), "total"
        assert torch.equal(r.cpu(), residual), "the residual changed"
    if y is not None:
        err = np.abs(f64(y) - want)
        bound = off + (HALF_STEP[y.dtype] + 2.0 ** -22) * np.abs(want) + SMALLEST[y.dtype]
        assert (err <= bound).all(), f"out: {(err > bound).sum()} off, worst {np.max(err / bound):.2f}"
    else:
        assert not with_out
    if group:
        groups, goff = want.reshape(T, -1, group), off.reshape(T, -1, group)
        got, scale = read_e4m3(to.data.cpu().numpy(), np.ones((T, N // group), np.float32)), f64(to.scale)
        amax = np.abs(groups).max(-1)
        some = amax >= 2.0 ** -99
        assert (np.abs(scale - amax / 448) <= (goff.max(-1) / 448 + 2.0 ** -22 * amax / 448))[some].all(), "scales"
        assert (scale[amax == 0] == 1).all()
        # code * scale is within half a step of E4M3 (its spacing below 2^-6 is 2^-9) and what y and the scale are off
        back = got * scale[..., None]
        step = np.maximum(2.0 ** -4 * np.abs(back), 2.0 ** -10 * scale[..., None])
        assert (np.abs(back - groups) <= step * (1 + 2.0 ** -20) + 2 * goff + 2.0 ** -21 * np.abs(groups))[some].all(), "codes"
    return y, total, to


@pytest.mark.parametrize("D", [8, 16, 64, 72, 128, 256, 504, 512, 520, 1024, 2000, 2048, 4096, 4104, 5000, 8192, 8200, 16384, 16392,
                               32768])
@pytest.mark.parametrize("T", [1, 3, 300])
def test_rows_of_any_width(T, D):
    x, w = data(D, (T, D), BF16, 3.0), data(D + 1, (D,), BF16)
    check(x, w)
    check(x, w, residual=data(D + 2, (T, D), BF16), group=D)
    if D % 128 == 0:
        check(x, w, residual=data(D + 2, (T, D), F32), group=128, with_out=False)


@pytest.mark.parametrize("xt", [BF16, F16, F32])
@pytest.mark.parametrize("rt", [None, BF16, F16, F32])
@pytest.mark.parametrize("wt", [None, BF16, F16, F32])
@pytest.mark.parametrize("ot", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(5, 640), (70, 4096)])
def test_types(xt, rt, wt, ot, shape):
    x = data(1, shape, xt, 2.0)
    check(x, None if wt is None else data(2, shape[1:], wt), residual=None if rt is None else data(3, shape, rt), out_dtype=ot,
          group=64)


@pytest.mark.parametrize("H,D", [(1, 64), (3, 8), (7, 128), (64, 128), (5, 96), (2, 512), (2, 520), (9, 2048), (40, 72)])
@pytest.mark.parametrize("T", [1, 37, 260])
def test_heads(T, H, D):
    """Each head has a norm of its own; x is a slice of a wider projection."""
    x = data(4, (T, H + 2, D), BF16)[:, 1:H + 1]
    x = x if H > 1 else x.reshape(T, 1, D)
    w = data(5, (D,), F32)
    check(x, w)
    check(x, w, residual=data(6, (T, H, D), F16), group=D)


@pytest.mark.parametrize("group", [8, 16, 32, 64, 128, 256, 512])
@pytest.mark.parametrize("n", [1, 3, 16])
def test_groups(group, n):
    x = data(7, (33, group * n), F16)
    x[:, :group] *= 100
    check(x, data(8, (group * n,), F16), group=group)


def test_rows_and_groups_of_zeros():
    x = data(9, (6, 1024), BF16)
    x[2] = 0
    x[4, 256:384] = 0
    _, _, to = check(x, group=128)
    assert (to.scale[2] == 1).all() and (to.data[2] == 0).all() and to.scale[4, 2] == 1 and (to.data[4, 2] == 0).all()
    y = idx.idx_rms_norm(x.cuda(), eps=0.0)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[3]).all()


@pytest.mark.parametrize("D", [256, 4096])
def test_values_that_are_not_finite(D):
    x = data(10, (8, D), F32)
    x[1, 5], x[3, 7], x[5, 9] = float("nan"), float("inf"), -float("inf")
    to = idx.Cache.empty(8, D // 128, 128)
    y = idx.idx_rms_norm(x.cuda(), to=to).cpu()
    assert torch.isnan(y[1]).all()
    for r, c in ((3, 7), (5, 9)):
        assert torch.isnan(y[r, c]) and (y[r, torch.arange(D) != c] == 0).all()
    clean = [0, 2, 4, 6, 7]
    assert torch.equal(y[clean], idx.idx_rms_norm(x[clean].cuda()).cpu())
    back = idx.idx_cache_read(to, dtype=F32).cpu()
    assert torch.isnan(back[1]).all() and torch.isnan(back[3, 0]).all() and torch.isnan(back[5, 0]).all()
    assert (back[3, 1:] == 0).all() and torch.isfinite(back[clean]).all()


@pytest.mark.parametrize("D", [128, 2048, 8192])
def test_in_place(D):
    """The residual's sum over the residual or over x, the result over x or over the residual."""
    x, r, w = data(11, (9, D), BF16).cuda(), data(12, (9, D), BF16).cuda(), data(13, (D,), BF16).cuda()
    total = torch.empty_like(r)
    want = idx.idx_rms_norm(x, w, residual=r, total=total)
    r1 = r.clone()
    assert torch.equal(idx.idx_rms_norm(x, w, residual=r1), want) and torch.equal(r1, total)
    x1 = x.clone()
    assert torch.equal(idx.idx_rms_norm(x1, w, residual=r, total=x1), want) and torch.equal(x1, total)
    x2, r2 = x.clone(), r.clone()
    assert idx.idx_rms_norm(x2, w, residual=r2, out=x2) is x2
    assert torch.equal(x2, want) and torch.equal(r2, total)
    r3, t3 = r.clone(), torch.empty_like(r)
    idx.idx_rms_norm(x, w, residual=r3, total=t3, out=r3)
    assert torch.equal(r3, want) and torch.equal(t3, total)


def test_rows_behind_the_cache_slots_stay_and_strides():
    wide = data(14, (20, 3, 1024), BF16).cuda()
    x = wide[:, 1]
    data_ = torch.full((25, 8, 128), 9, dtype=torch.uint8, device="cuda")
    scale = torch.full((25, 8), 3.0, device="cuda")
    to = idx.Cache(data_, scale)
    out = torch.zeros((20, 2, 1024), dtype=BF16, device="cuda")
    idx.idx_rms_norm(x, out=out[:, 1], to=to)
    plain = idx.Cache.empty(20, 8, 128)
    want = idx.idx_rms_norm(x.contiguous(), to=plain)
    assert torch.equal(out[:, 1], want) and (out[:, 0] == 0).all()
    assert torch.equal(data_[:20], plain.data) and torch.equal(scale[:20], plain.scale)
    assert (data_[20:] == 9).all() and (scale[20:] == 3).all()
    # rows that share memory as input
    one = data(15, (1, 512), BF16).cuda()
    assert torch.equal(idx.idx_rms_norm(one.expand(7, 512)), idx.idx_rms_norm(one.repeat(7, 1)))


def test_codes_agree_with_a_cache_write():
    """Codes of y in fp32 are those that a write of it gives."""
    x = data(16, (40, 4096), BF16).cuda()
    to = idx.Cache.empty(40, 32, 128)
    y = idx.idx_rms_norm(x, out=torch.empty((40, 4096), device="cuda"), to=to)
    other = idx.Cache.empty(40, 32, 128)
    idx.idx_cache_write([idx.Write(y.view(40, 32, 128), other)])
    assert torch.equal(to.data, other.data) and torch.equal(to.scale, other.scale)
    codes, scale = quantise_e4m3(y.cpu().numpy().reshape(40, 32, 128))
    one = np.ones_like(scale)      # as values: the encoder has no negative zero
    assert np.array_equal(read_e4m3(to.data.cpu().numpy(), one), read_e4m3(codes, one))
    assert np.array_equal(to.scale.cpu().numpy(), scale)


def test_many_rows():
    x = data(17, (70001, 128), BF16)
    check(x, data(18, (128,), BF16), group=128)


def test_streams_and_graphs():
    x, r, w = data(19, (64, 4096), BF16).cuda(), data(20, (64, 4096), BF16).cuda(), data(21, (4096,), BF16).cuda()
    to, total, out = idx.Cache.empty(64, 32, 128), torch.empty_like(r), torch.empty_like(x)
    call = lambda **kw: idx.idx_rms_norm(x, w, residual=r, total=total, out=out, to=to, **kw)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (22, 23, 24):
        x.copy_(data(seed, (64, 4096), BF16))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, total, to.data, to.scale)]
        for t in (out, total, to.data, to.scale):
            t.zero_()
        torch.cuda.synchronize()
        call(stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        for a, b in zip(got, (out, total, to.data, to.scale)):
            assert torch.equal(a, b)


def test_nothing_to_do():
    assert idx.idx_rms_norm(torch.zeros((0, 64), dtype=BF16, device="cuda")).shape == (0, 64)
    assert idx.idx_rms_norm(torch.zeros((4, 0, 64), dtype=BF16, device="cuda")).shape == (4, 0, 64)


def test_refusals():
    x = data(25, (4, 256), BF16).cuda()
    bad = [dict(weight=torch.ones(128, device="cuda")), dict(weight=torch.ones(256, device="cuda", dtype=torch.float64)),
           dict(weight=torch.ones(512, device="cuda")[::2]), dict(weight=torch.ones(256)), dict(residual=x[:2]),
           dict(residual=x, total=x[:, :128]), dict(total=x), dict(out=x[:2]), dict(residual=x.cpu()),
           dict(weight=torch.ones(256, device="cuda", requires_grad=True)), dict(residual=x.clone().requires_grad_())]
    for kw in bad:
        with pytest.raises(ValueError):
            idx.idx_rms_norm(x, **kw)
    with pytest.raises(ValueError):
        idx.idx_rms_norm(x.clone().requires_grad_())
    with pytest.raises(ValueError):
        idx.idx_rms_norm(x.double())
    with pytest.raises(ValueError):
        idx.idx_rms_norm(x.flatten())
    for kw, status in ((dict(with_out=False), 1), (dict(to=idx.Cache.empty(4, 2, 128, idx.IDX_K_BF16)), 6),
                       (dict(to=idx.Cache.empty(3, 2, 128)), 2), (dict(to=idx.Cache.empty(4, 3, 128)), 2), (dict(eps=-1.0), 3)):
        with pytest.raises(idx.IdxError) as e:
            idx.idx_rms_norm(x, **kw)
        assert e.value.status == status
    with torch.no_grad():
        idx.idx_rms_norm(x.clone().requires_grad_())
