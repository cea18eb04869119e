"""The operators around the indexer record no gradient: rows that require one are refused while autograd is on."""
import pytest
import torch

import mqa_logits_top_amd as idx

pytestmark = pytest.mark.gpu


def test_rows_that_require_a_gradient():
    plan, pos = idx.Rotary.make(64), torch.arange(3, dtype=torch.int32, device="cuda")
    x = torch.randn((3, 4, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    p = x.clone().requires_grad_()
    c = idx.Cache.empty(3, 4, 64, idx.IDX_K_BF16)
    sel = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    calls = (lambda t: idx.idx_rope(t, pos, plan), lambda t: idx.idx_cache_write([idx.Write(t, c)]),
             lambda t: idx.idx_sparse_attn(t, c, c, sel, 0.1)[0], lambda t: idx.idx_rope(x, pos, plan, out=t),
             lambda t: idx.idx_cache_read(c, out=t))
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call(p)
    assert torch.equal(p, x) and not c.data.any()
    for call in calls[:3]:
        want = call(x)
        with torch.no_grad():
            got = call(p)
        assert want is None or torch.equal(got, want)
