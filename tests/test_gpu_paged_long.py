"""Attention over a paged cache at the largest lengths and batches that its header allows."""
import numpy as np
import pytest
import torch

import mqa_logits_top_amd as idx
from around_ref import attend, read_e4m3
from dense_ref import weight_step

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def gpu(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def caches(seed, rows, H, D, fp8):
    g = torch.Generator().manual_seed(seed)
    out = [idx.Cache.empty(rows, H, D, idx.IDX_K_FP8_E4M3 if fp8 else idx.IDX_K_BF16) for _ in range(2)]
    for c in out:
        idx.idx_cache_write([idx.Write(torch.randn((rows, H, D), generator=g).to(BF16).cuda(), c)])
    return out


def values(c):
    return (c.data.cpu().double().numpy() if c.scale is None
            else read_e4m3(c.data.cpu().numpy(), c.scale.cpu().numpy()))


def compare(out, lse, q, k, v, seen, scale, pick):
    """seen: the slots that each row of pick sees."""
    want, wl, bo, bl = attend(q[pick].cpu().double().numpy(), values(k), values(v), seen, scale,
                              weight_step(True, k.scale is not None), BF16)
    err = np.abs(out[pick].cpu().double().numpy() - want)
    assert (err <= bo).all(), f"out: {(~(err <= bo)).sum()} off, worst {np.nanmax(err / bo):.2f} of the bound"
    assert (np.abs(lse[pick].cpu().double().numpy() - wl) <= bl).all(), "lse"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("T", [1, 40])
def test_lengths_up_to_the_largest(T, page, fp8):
    """Positions up to 2^31 - 2, in a window; the pages of the table are a few, again and again."""
    n_pages, P, D, window, first = (2 ** 31 - 1) // page, 61, 64, 100, 3
    n = n_pages * page
    assert n > 2 ** 31 - 32
    k, v = caches(300, P * page, 1, D, fp8)
    pages = (torch.arange(n_pages, dtype=torch.int32, device="cuda") % P).view(1, n_pages)
    q = torch.randn((T, 8, D), generator=torch.Generator().manual_seed(301)).to(BF16).cuda()
    for length in (n, 2 ** 31 - 1, n - 50):
        out, lse = idx.idx_paged_attn(q, k, v, pages, gpu([0, T]), gpu([length]), 0.125, page=page, window=window, first=first)
        pick = sorted({0, T // 2, T - 1})
        seen = []
        for t in pick:
            p = min(length, n) - T + t
            s = np.concatenate([np.arange(first), np.arange(p - window + 1, p + 1)])
            seen.append(s // page % P * page + s % page)
        compare(out, lse, q, k, v, seen, 0.125, pick)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,rows,Hkv,G,D", [(65, 1, 2, 4, 128), (200, 1, 2, 4, 64), (1000, 1, 1, 8, 128), (130, 4, 1, 8, 128),
                                            (100, 24, 1, 8, 128), (300, 12, 1, 8, 64), (70, 60, 1, 4, 128)])
def test_many_requests_whose_keys_are_divided(B, rows, Hkv, G, D, fp8):
    """More requests than lanes, empty ones among them, with long ones early, in the 65th place and last: the division counts
    them 64 at a time."""
    rng = np.random.default_rng(310)
    page = 16
    new = rng.integers(0, 2 * rows, B) if rows > 1 else np.ones(B, int)
    long = [2, 64, B - 1]
    new[long] = np.maximum(new[long], rows)
    lens = new + rng.integers(0, 200, B)
    lens[long] = [7001, 5000, 9003]
    held = -(-lens // page)
    order = rng.permutation(held.sum()).astype(np.int32)
    pages = np.full((B, held.max() + 1), -7, np.int32)
    for b, at in enumerate(np.cumsum(held) - held):
        pages[b, :held[b]] = order[at:at + held[b]]
    cu, T = np.cumsum([0, *new]), int(new.sum())
    k, v = caches(311, int(held.sum()) * page, Hkv, D, fp8)
    q = torch.randn((T, Hkv * G, D), generator=torch.Generator().manual_seed(312)).to(BF16).cuda()
    for window, first in ((0, 0), (3000, 5)):
        out, lse = idx.idx_paged_attn(q, k, v, gpu(pages), gpu(cu), gpu(lens), 0.1, page=page, window=window, first=first)
        pick = sorted({int(cu[b + 1]) - 1 for b in long} | {int(cu[b]) for b in long} | set(rng.integers(0, T, 30).tolist()))
        seen = []
        for t in pick:
            b = int(np.searchsorted(cu, t, "right")) - 1
            p = lens[b] - new[b] + t - cu[b]
            s = np.arange(p + 1)
            s = s[(s > p - window) | (s < first)] if window else s
            seen.append(pages[b, s // page] * page + s % page)
        compare(out, lse, q, k, v, seen, 0.1, pick)
        again = idx.idx_paged_attn(q, k, v, gpu(pages), gpu(cu), gpu(lens), 0.1, page=page, window=window, first=first)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
