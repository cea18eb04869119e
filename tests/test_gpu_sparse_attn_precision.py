"""The precision of attention over selected keys does not depend on how many rows a call has, and weights far below
a row's largest are not lost."""
import numpy as np
import pytest
import torch

import mqa_logits_top_amd as idx
from around_ref import attend, read_e4m3

pytestmark = pytest.mark.gpu

FP8 = idx.IDX_K_FP8_E4M3


def _e4m3(seed, rows, H, D):
    c = idx.Cache.empty(rows, H, D, FP8)
    x = torch.randn((rows, H, D), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    idx.idx_cache_write([idx.Write(x.cuda(), c)])
    return c, read_e4m3(c.data.cpu().numpy(), c.scale.cpu().numpy())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 60, 500, 800])
@pytest.mark.parametrize("Hq,D,n", [(8, 128, 1), (32, 128, 1), (32, 64, 3), (64, 128, 2), (40, 64, 5)])
def test_e4m3_weights_in_two_parts(dtype, T, Hq, D, n):
    """A result of E4M3 caches is the formula's rounded once, but for 2^-16 of the weights: with one to five keys a
    row, weights of 8 bits would add up to another half step of bf16 (one key: its value times a rounded scale)."""
    rng = np.random.default_rng(T + Hq + n)
    (k, kd), (v, vd) = _e4m3(1, 300, 1, D), _e4m3(2, 300, 1, D)
    q = torch.randn((T, Hq, D), generator=torch.Generator().manual_seed(T)).to(dtype)
    sel = rng.integers(0, 300, (T, n)).astype(np.int32)
    out, _ = idx.idx_sparse_attn(q.cuda(), k, v, torch.from_numpy(sel).cuda(), 0.1)
    want, _, bound, _ = attend(q.double().numpy(), kd, vd, list(sel.astype(np.int64)), 0.1, 2.0 ** -16, dtype)
    err = np.abs(out.cpu().double().numpy() - want)
    assert (err <= bound).all(), f"{(err > bound).sum()} off, worst {np.max(err / bound):.2f} of the bound"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("T,Hq,D,n", [(1, 8, 64, 40000), (150, 16, 64, 20000), (800, 32, 64, 20000),
                                      (800, 32, 128, 20000), (400, 8, 128, 20000)])
def test_many_small_weights(dtype, first, T, Hq, D, n):
    """One key of score 0 and value 0, and n whose weight is exp(-17.75), 2^-25.6 of it, with values of 1/2 to 3/2:
    together they are the output.  A weight is rounded relatively, and by at most 2^-32 of the largest beside."""
    rng = np.random.default_rng(n)
    data = [torch.zeros((n + 1, 1, D), dtype=dtype) for _ in range(2)]
    at = 0 if first else n
    data[0][:, 0, 0] = -17.75
    data[0][at, 0, 0] = 0.0
    data[1][:] = torch.from_numpy(rng.uniform(0.5, 1.5, (n + 1, 1, D))).to(dtype)
    data[1][at] = 0.0
    fmt = idx.IDX_K_F16 if dtype == torch.float16 else idx.IDX_K_BF16
    k, v = (idx.Cache(x.cuda(), fmt=fmt) for x in data)
    q = torch.zeros((T, Hq, D), dtype=dtype)
    q[:, :, 0] = 1.0
    sel = torch.arange(n + 1, dtype=torch.int32, device="cuda").expand(T, n + 1).contiguous()
    out, lse = idx.idx_sparse_attn(q.cuda(), k, v, sel, 1.0)
    w = np.exp(np.where(np.arange(n + 1) == at, 0.0, -17.75))
    x = data[1][:, 0].double().numpy()
    want = (w @ x / w.sum())[None, None]
    # each weight rounded by `step` relative, and by 2^-32 of the largest in fp16, in numerator and divisor (whose
    # change by them is below 2^-15 relative); sums of n terms in fp32; the score (in units of ln 2, once rounded) and
    # the exponential 2^-19; the result's rounding, where fp16 has steps of 2^-24 at least
    step, half = (2.0 ** -11, 2.0 ** -11) if dtype == torch.float16 else (2.0 ** -8, 2.0 ** -8)
    bound = (step + 2.0 ** -15 + 2.0 ** -19 + n * 2.0 ** -23 + half) * want + 2.0 ** -25
    if dtype == torch.float16:
        bound = bound + 2.0 ** -32 * x.sum(0)
    err = np.abs(out.cpu().double().numpy() - want)
    assert (err <= bound).all(), f"{(err > bound).sum()} off, worst {np.max(err / bound):.2f} of the bound"
    assert np.abs(lse.cpu().double().numpy() - np.log(w.sum())).max() <= 2.0 ** -19 + n * 2.0 ** -23


@pytest.mark.parametrize("dtype,fp8,power", [(torch.bfloat16, False, p) for p in (20, 30, 40, 90)]
                         + [(torch.float16, False, p) for p in (18, 22, 26)]
                         + [(torch.bfloat16, True, p) for p in (20, 30, 40, 90)]
                         + [(torch.float16, True, p) for p in (18, 30, 40)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("T,Hq,D,n", [(1, 8, 64, 3000), (200, 16, 128, 600), (800, 32, 64, 300), (800, 32, 128, 300)])
def test_large_scores(dtype, fp8, power, sign, T, Hq, D, n):
    """Scores of 9, 11, 13 and 15 times D 2^power and a factor of each head's, products exact in fp32: the keys of the
    largest share the weight alike and the others, 30000 or more below in the exponent, have none."""
    rng = np.random.default_rng(power + n)
    half = power // 2 if dtype == torch.bfloat16 else power - 14
    size = rng.choice([9, 11, 13, 15], n)
    size[: n // 3] = 11                                                 # the largest comes late
    key = torch.from_numpy(sign * size * 2.0 ** half)[:, None, None].expand(n, 1, D)
    val = torch.from_numpy(rng.integers(-8, 9, (n, 1, D)) * 0.5)
    caches = []
    for x in (key, val):
        c = idx.Cache.empty(n, 1, D, FP8 if fp8 else idx.IDX_K_F16 if dtype == torch.float16 else idx.IDX_K_BF16)
        if fp8:                                                         # exact: codes of 4 bits, scales a power of two
            top = x.abs().amax(-1).clamp(min=0.5)
            unit = torch.exp2(torch.floor(torch.log2(top)))
            c.data.copy_((x / unit[..., None]).to(torch.float8_e4m3fn).view(torch.uint8))
            c.scale.copy_(unit)
        else:
            c.data.copy_(x)
        caches.append(c)
    factor = 2.0 ** (power - half) * (1 + torch.arange(Hq, dtype=torch.float64) % 16 / 16)
    q = factor[:, None].expand(T, Hq, D).to(dtype).cuda()
    scale = 0.1 * 2.0 ** -0.5
    sel = torch.arange(n, dtype=torch.int32, device="cuda").expand(T, n).contiguous()
    out, lse = idx.idx_sparse_attn(q, *caches, sel, scale)
    best = size == (size * sign).max() * sign
    want = val[torch.from_numpy(best)][:, 0].mean(0)
    # equal weights, rounded alike; sums of n products in fp32; the result's rounding
    half_step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    bound = half_step * want.abs() + (2.0 ** -16 + 2.0 ** -21 + n * 2.0 ** -23) * 4.0
    assert ((out.cpu().double() - want).abs() <= bound).all()
    s = float(np.float32(scale)) * sign * size[best][0] * factor * D * 2.0 ** half
    # the score: its factor rounded twice, itself once, the logarithm's share in fp32 steps of it
    assert ((lse.cpu().double() - (s + np.log(best.sum()))).abs() <= 2.0 ** -21 * s.abs()).all()
