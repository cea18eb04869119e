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


def time_of(call, n=20):
    """Milliseconds of n captured calls, the least of 25 times."""
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(n):
            call()
    g.replay()
    best = float("inf")
    for _ in range(25):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,n", [([300], 20005), ([1] * 40, 1001), ([1], 90)])
@pytest.mark.parametrize("window", [0, 500])
def test_slots_that_no_row_sees_cost_nothing(new, n, window, fp8):
    """NaN behind the last key of a page, before the window and in the slot that a page outside the cache stands for: the bits
    and, within 15%, the time are those without."""
    page, H, D, B = 16, 2, 128, len(new)
    held = (n + page - 1) // page
    k, v = caches(210, (held + 1) * page, H, D, BF16, fp8)
    pages = np.random.default_rng(211).permutation(held).astype(np.int32) + 1     # slots 0 .. 15: no key's
    pages[held // 3] = -1
    q = torch.randn((sum(new), 16, D), generator=torch.Generator().manual_seed(212)).to(BF16).cuda()
    out, lse = torch.empty_like(q), torch.empty((sum(new), 16), device="cuda")
    args = (q, k, v, gpu(pages).repeat(B, 1), gpu(np.cumsum([0] + new)), gpu([n] * B), 0.1)
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    call = lambda: idx.idx_paged_attn(*args, page=page, window=window, first=3, out=out, lse=lse, ws=ws)
    clean = time_of(call)
    want = out.clone(), lse.clone()
    keys = np.arange(held * page)
    low = n - new[0] - window + 1 if window else 0                                # the first row's window
    seen = (keys < n) & (pages[keys // page] >= 0) & ((keys >= low) | (keys < 3))
    unseen = np.ones((held + 1) * page, bool)
    unseen[(pages[keys // page] * page + keys % page)[seen]] = False
    at = torch.from_numpy(unseen).cuda()
    for c in (k, v):
        c.data[at] = 0x7F if fp8 else float("nan")
        if fp8:
            c.scale[at] = float("inf")
    dirty = time_of(call)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert dirty <= 1.15 * clean, f"{dirty:.3f} ms, {clean:.3f} without"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,n", [([200], 3000), ([130], 140), ([3], 700)])
@pytest.mark.parametrize("window,first", [(0, 0), (400, 70)])
def test_values_of_several_edges_reach_their_rows(new, n, window, first, fp8):
    """NaN in a key of the first keys, one that some windows have left, one beside a page outside the cache, and one that only
    the last rows see; garbage where no row looks."""
    page, H, D = 16, 2, 64
    T, held = new[0], (n + page - 1) // page
    k, v = caches(220, (held + 1) * page, H, D, BF16, fp8)
    pages = np.random.default_rng(221).permutation(held).astype(np.int32) + 1
    pages[held // 2] = 2 ** 30
    q = torch.randn((T, 16, D), generator=torch.Generator().manual_seed(222)).to(BF16).cuda()
    call = lambda: idx.idx_paged_attn(q, k, v, gpu(pages[None]), gpu([0, T]), gpu([n]), 0.1, page=page, window=window, first=first)
    want = call()
    bad = {1: 5, max(n - T - window + 20, 20) if window else n // 2 - 20: 11, n - 2: 40}   # key: dim
    for key, dim in bad.items():
        slot = pages[key // page] * page + key % page
        v.data[slot, 1, dim] = 0xFF if fp8 else float("nan")
    for c in (k, v):
        c.data[:page] = 0x7F if fp8 else float("inf")
        c.data[pages[-1] * page + (n - 1) % page + 1:(pages[-1] + 1) * page] = 0x7F if fp8 else float("nan")
    out, lse = call()
    assert torch.equal(lse, want[1])
    pos = n - T + np.arange(T)
    nan = torch.zeros((T, 16, D), dtype=torch.bool)
    for key, dim in bad.items():
        if pages[key // page] <= held:
            sees = (key <= pos) & ((key > pos - window) | (key < first)) if window else key <= pos
            nan[torch.from_numpy(sees), 8:, dim] = True
    assert nan.any() and torch.equal(torch.isnan(out.cpu()), nan)
    assert torch.equal(out.cpu()[~nan], want[0].cpu()[~nan])
