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
