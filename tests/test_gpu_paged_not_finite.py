"""Attention over a paged cache whose slots hold values that are not finite: what they change, and what they cost."""
import numpy as np
import pytest
import torch

import mqa_logits_top_amd as idx

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
KIND = {BF16: idx.IDX_K_BF16, F16: idx.IDX_K_F16}


def gpu(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def caches(seed, rows, H, D, dtype, fp8):
    g = torch.Generator().manual_seed(seed)
    out = [idx.Cache.empty(rows, H, D, idx.IDX_K_FP8_E4M3 if fp8 else KIND[dtype]) for _ in range(2)]
    for c in out:
        idx.idx_cache_write([idx.Write(torch.randn((rows, H, D), generator=g).to(dtype).cuda(), c)])
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [2, 100])
@pytest.mark.parametrize("n", [170, 3000])
def test_a_product_past_the_range_keeps_its_weight_beside_a_nan(n, T, D):
    """Key 3's value is 448 times a scale that fp32 holds and their product passes, with a weight of about 2^-60; key n - 1's is
    NaN in one dim.  The rows that see both show the NaN there and nothing of it elsewhere."""
    k, v = (idx.Cache.empty(n, 1, D) for _ in range(2))
    k.data[:, 0, 0] = 0x38                       # 1 in each key's first dim
    k.data[3] = 0
    v.data[:, 0, :] = 0x38
    v.data[3, 0, 1] = 0x7E                       # 448
    v.scale[3] = 8e35
    v.data[n - 1, 0, 2] = 0x7F
    q = torch.zeros((T, 8, D), dtype=BF16, device="cuda")
    q[..., 0] = 1
    scale = 60 * np.log(2)                       # of a key's weight over key 3's
    out, _ = idx.idx_paged_attn(q, k, v, gpu([np.arange((n + 15) // 16)]) if n % 16 == 0 else gpu([np.arange(n)]), gpu([0, T]),
                                gpu([n]), scale, page=16 if n % 16 == 0 else 1)
    out = out.float().cpu()
    pos = n - T + np.arange(T)
    small = 448 * 8e35 * 2.0 ** -60 / pos        # key 3's share: pos other keys of weight 1
    assert np.all(np.abs(out[:, :, 1].double().numpy() - (1 + small[:, None])) <= 2.0 ** -7 * (1 + small[:, None]))
    assert torch.isnan(out[T - 1, :, 2]).all() and torch.isfinite(out[:T - 1, :, 2]).all()
    rest = [d for d in range(D) if d not in (1, 2)]
    assert torch.isfinite(out[:, :, rest]).all()
