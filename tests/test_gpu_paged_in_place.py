"""Attention over a paged cache whose results take the queries' place."""
import numpy as np
import pytest
import torch

import mqa_logits_top_amd as idx

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def gpu(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("new,lens", [([1, 1, 1], [3000, 5, 700]), ([3, 9], [4000, 100]), ([150, 1, 40], [150, 900, 6000]),
                                      ([700], [700])])
def test_results_in_the_queries_place(new, lens, dtype, fp8):
    """Every workgroup has read its rows' queries before it, or the join behind all, writes them."""
    page, H, D, B = 16, 2, 128, len(new)
    held = [-(-n // page) for n in lens]
    order = np.random.default_rng(500).permutation(sum(held)).astype(np.int32)
    pages = np.zeros((B, max(held)), np.int32)
    for b, at in enumerate(np.cumsum(held) - held):
        pages[b, :held[b]] = order[at:at + held[b]]
    g = torch.Generator().manual_seed(501)
    k, v = (idx.Cache.empty(sum(held) * page, H, D, idx.IDX_K_FP8_E4M3 if fp8 else
                            {BF16: idx.IDX_K_BF16, F16: idx.IDX_K_F16}[dtype]) for _ in range(2))
    for c in (k, v):
        idx.idx_cache_write([idx.Write(torch.randn((c.rows, H, D), generator=g).to(dtype).cuda(), c)])
    wide = torch.randn((sum(new), 20, D), generator=g).to(dtype).cuda()
    args = (k, v, gpu(pages), gpu(np.cumsum([0] + new)), gpu(lens), 0.1)
    want, lse = idx.idx_paged_attn(wide[:, 2:18], *args, page=page)
    rest = wide.clone()
    q = wide[:, 2:18]
    out, lse2 = idx.idx_paged_attn(q, *args, page=page, out=q)
    assert out is q and torch.equal(q, want) and torch.equal(lse2, lse)
    assert torch.equal(wide[:, :2], rest[:, :2]) and torch.equal(wide[:, 18:], rest[:, 18:])
