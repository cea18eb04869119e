"""RMS norm of rows whose squares fp32 does not hold, with an eps that does not cover them."""
import pytest
import torch

import mqa_logits_top_amd as idx
from test_gpu_rms_norm import check, data

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 2.0 ** -133, 2.0 ** -110, 2.0 ** -99])
@pytest.mark.parametrize("D", [64, 512, 1000, 1536, 4096, 8200, 32768])
def test_rows_of_any_magnitude(D, eps, dtype):
    """(Every eps is one that fp32 holds.)  Neighbouring rows from 1 down to the smallest normal numbers, alone and on a residual as small."""
    size = torch.tensor([1.0, 2.0 ** -60, 2.0 ** -75, 1.0, 2.0 ** -100, 2.0 ** 40, 2.0 ** -120])[:, None]
    x = (data(D, (7, D), F32) * size).to(dtype)
    x[5, :8] = 0
    check(x, data(D + 1, (D,), BF16), eps=eps, out_dtype=F32, group=D)
    check(x, None, eps=eps, residual=(data(D + 2, (7, D), F32) * size).to(dtype), out_dtype=F32)


def test_subnormal_and_empty_rows():
    x = torch.zeros((4, 256))
    x[0, 3], x[1, :] = 2.0 ** -149, 2.0 ** -130
    y = idx.idx_rms_norm(x.cuda(), eps=0.0).cpu()
    assert y[0, 3] == 16 and (y[0, 4:] == 0).all() and (y[1] == 1).all() and torch.isnan(y[2:]).all()
    y = idx.idx_rms_norm(x.cuda(), eps=1e-44).cpu()
    assert (y[2:] == 0).all() and torch.isfinite(y).all() and (y[1] > 0).all()


@pytest.mark.parametrize("D", [128, 1536, 8192])
def test_a_small_eps_changes_no_bit_of_other_rows(D):
    """Scaling by a power of two is exact: the bits are those of an eps that no scaling goes with."""
    x, w = data(400, (9, D), BF16, 3.0).cuda(), data(401, (D,), BF16).cuda()
    to = [idx.Cache.empty(9, 1, D) for _ in range(2)]
    a, b = (idx.idx_rms_norm(x, w, eps=e, to=c) for e, c in zip((0.0, 1e-29), to))
    assert torch.equal(a, b) and torch.equal(to[0].data, to[1].data) and torch.equal(to[0].scale, to[1].scale)
