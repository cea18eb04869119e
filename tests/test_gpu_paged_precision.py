"""How exactly attention over a paged cache weighs its values."""
import numpy as np
import pytest
import torch

import mqa_logits_top_amd as idx
from around_ref import read_e4m3

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
BITS = {BF16: 8, F16: 11}


def gpu(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def half_step(x, dtype):
    """Half the distance of the type's numbers at x."""
    lowest = -14 if dtype == F16 else -126
    return 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -200))), lowest) - BITS[dtype])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("single", [True, False])
def test_a_row_that_sees_one_quantised_key_gives_its_value(dtype, D, page, single):
    """The weight is 1 and the value code * scale: its two parts of 8 bits are off by at most 2^-16 of it, the sums by a few
    2^-24, and the result is rounded once."""
    H, n = 2, 300
    g = torch.Generator().manual_seed(200)
    k, v = idx.Cache.empty(n + 20, H, D), idx.Cache.empty(n + 20, H, D)
    for c in (k, v):
        x = torch.randn((n + 20, H, D), generator=g) * (1 + torch.rand((n + 20, H, 1), generator=g))
        idx.idx_cache_write([idx.Write(x.to(BF16).cuda(), c)])
    q = torch.randn((n, 8, D), generator=g).to(dtype).cuda()
    if single:                                   # requests of one token each
        pages, cu, lens = gpu(np.arange(n)[:, None]), gpu(np.arange(n + 1)), gpu([1] * n)
        pages, at, window = (pages, np.arange(n), 0) if page == 1 else (pages % (n // 16), np.arange(n) % (n // 16) * 16, 0)
    else:                                        # a chunk in a window of one key
        pages, cu, lens = gpu(np.arange((n + page - 1) // page)[None]), gpu([0, n]), gpu([n])
        at, window = np.arange(n), 1
    out, _ = idx.idx_paged_attn(q, k, v, pages, cu, lens, 0.1, page=page, window=window)
    want = np.repeat(read_e4m3(v.data.cpu().numpy(), v.scale.cpu().numpy())[at], 4, 1)
    err = np.abs(out.cpu().double().numpy() - want)
    bound = half_step(want, dtype) + (2.0 ** -16 + 2.0 ** -21) * np.abs(want)
    assert (err <= bound).all(), f"{(err > bound).sum()} off, worst {np.max(err / bound):.2f} of the bound"


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("new,n", [([1], 20), ([1], 9000), ([3, 3], 700), ([140], 700), ([130, 9], 12000), ([300] * 6, 420)])
def test_values_that_are_all_alike_come_out_as_they_are(dtype, D, page, new, n):
    """Nearly every weight is rounded the same way, by almost half a step, so that a sum of the weights before they are rounded
    would be off by that: an average of ones is one to a sum's 2^-24 a term, far below half a step of a result."""
    H, B = 2, len(new)
    k, v = (idx.Cache.empty((n + page - 1) // page * page, H, D, {BF16: idx.IDX_K_BF16, F16: idx.IDX_K_F16}[dtype])
            for _ in range(2))
    k.data[::16, :, 0] = 1                       # score 1, the others 0
    v.data[:] = 1
    q = torch.zeros((sum(new), 8, D), dtype=dtype, device="cuda")
    q[..., 0] = 1
    part = 1 + 0.96 * 2.0 ** -BITS[dtype]        # of the others' weights: rounded down to 1, by 0.96 of half a step
    scale = np.log(2) - np.log(part)             # their weights are exp(-scale) = part / 2
    pages = gpu(np.arange((n + page - 1) // page)).repeat(B, 1)
    out, lse = idx.idx_paged_attn(q, k, v, pages, gpu(np.cumsum([0] + new)), gpu([n] * B), scale, page=page)
    assert (out == 1).all(), out[out != 1]
    pos = np.concatenate([n - x + np.arange(x) for x in new])
    high = pos // 16 + 1
    want = scale + np.log(high + (pos + 1 - high) * part / 2)
    assert (np.abs(lse.cpu().double().numpy() - want[:, None]) <= 2.0 ** -20 + n * 2.0 ** -24).all()
