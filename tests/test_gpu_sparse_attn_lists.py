"""Attention over selected keys: long lists in every form that serves a prompt, long caches, and one row in calls of
any size."""
import numpy as np
import pytest
import torch

import mqa_logits_top_amd as idx
from around_ref import attend, keys_of, read_e4m3

pytestmark = pytest.mark.gpu

FP8 = idx.IDX_K_FP8_E4M3
VALUE = {torch.bfloat16: idx.IDX_K_BF16, torch.float16: idx.IDX_K_F16}


def _caches(seed, rows, H, D, dtype, fp8):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        c = idx.Cache.empty(rows, H, D, FP8 if fp8 else VALUE[dtype])
        idx.idx_cache_write([idx.Write(torch.randn((rows, H, D), generator=g).to(dtype).cuda(), c)])
        out.append(c)
    return out


def _values(c, at):
    data = c.data[at].cpu()
    return read_e4m3(data.numpy(), c.scale[at].cpu().numpy()) if c.fmt == FP8 else data.double().numpy()


def _q(seed, T, Hq, D, dtype):
    return (torch.randn((T, Hq, D), generator=torch.Generator().manual_seed(seed)) * 2.0).to(dtype)


def _compare(take, out, lse, q, k, v, sel, scale, pool=1, ks=None, ke=None, table=None):
    """Rows `take` of a call's outputs against 64 bits on the cache rows that they name."""
    sub = lambda a: None if a is None else a[take]
    rows = keys_of(sel[take], sub(ks), sub(ke), pool, k.rows if table is None else len(table), table, k.rows)
    named = np.unique(np.concatenate([*rows, np.zeros(1, np.int64)]))
    at = torch.from_numpy(named).cuda()
    near = [np.searchsorted(named, r) for r in rows]
    step = 2.0 ** -16 if k.fmt == FP8 else 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -11
    want, wl, bo, bl = attend(q[take].double().numpy(), _values(k, at), _values(v, at), near, scale, step, q.dtype)
    got, gl = out.cpu()[take].double().numpy(), lse.cpu()[take].double().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
    err = np.abs(got - want)
    assert (err <= bo).all(), f"{(err > bo).sum()} off, worst {np.max(err / bo):.2f} of the bound"
    fin = np.isfinite(wl)
    assert (np.abs(gl[fin] - wl[fin]) <= bl[fin]).all(), "lse"


def _lists(rng, T, n, most, pool=1):
    """Ascending ids below `most`, one in ten missing, and in some rows runs of 256 entries and more; one row of nothing
    and one of a single id behind them all."""
    s = np.sort(rng.integers(0, most, (T, n)), 1).astype(np.int32)
    s[rng.random((T, n)) < 0.1] = -1
    s[0, : n // 2] = -1
    if T > 4:
        s[1, 256 // pool:768 // pool] = -1
        s[2] = -1
        s[3] = -1
        s[3, -1] = most - 1
        s[T - 1, 300 // pool:] = -1
    return s


@pytest.mark.parametrize("form", ["ids", "window and table", "blocks", "blocks and table"])
@pytest.mark.parametrize("dtype,fp8", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True),
                                       (torch.float16, True)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(800, 32, 1), (401, 96, 2), (1601, 16, 1), (820, 24, 3), (300, 16, 1), (30, 16, 2)])
def test_streamed_lists(form, dtype, fp8, D, T, Hq, Hkv):
    """Lists of more entries than a wave's queue holds, in waves of 32 heads, lone waves of 16, and waves that divide a
    list: ids in flight over several rounds, the queue round its end, whole rounds that add nothing."""
    rng = np.random.default_rng(T + D)
    L, slots, pool = 6000, 6500, 8 if "blocks" in form else 1
    k, v = _caches(T, slots if "table" in form else L, Hkv, D, dtype, fp8)
    ks = ke = table = None
    n = 1111 if pool == 1 else 139
    s = _lists(rng, T, n, L // pool, pool)
    if form != "ids":
        ks = rng.integers(0, 700, T).astype(np.int32)
        ke = (L - rng.integers(0, 700, T)).astype(np.int32)
    if "table" in form:
        table = rng.permutation(slots)[:L].astype(np.int32)
        table[rng.integers(0, L, 300)] = -1
    q = _q(T, T, Hq, D, dtype)
    cu = lambda a: None if a is None else torch.from_numpy(a).cuda()
    out, lse = idx.idx_sparse_attn(q.cuda(), k, v, cu(s), D ** -0.5, pool=pool, ks=cu(ks), ke=cu(ke),
                                   slot_of_key=cu(table))
    _compare(np.array([0, 1, 2, 3, T // 2, T - 1]), out, lse, q, k, v, s, D ** -0.5, pool, ks, ke, table)


@pytest.mark.parametrize("dtype,fp8", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True),
                                       (torch.float16, True)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(2, 8), (60, 16), (100, 32), (330, 4)])
def test_long_lists_on_long_caches(dtype, fp8, D, T, G):
    """Lists of many tiles over caches past 2^32 bytes: the bits of the same call on a compacted copy."""
    H, n, used = 8, 555, 3000
    rows = (2 ** 32 + 2 ** 28) // (H * D * (1 if fp8 else 2))
    rng = np.random.default_rng(T + D)
    at = np.unique(np.concatenate([rng.integers(0, rows, used), [0, rows - 1, rows - 2]]))
    near, _ = _caches(7, len(at), H, D, dtype, fp8)
    data = torch.zeros((rows, H, D), dtype=near.data.dtype, device="cuda")
    scale = torch.zeros((rows, H), device="cuda") if fp8 else None
    where = torch.from_numpy(at).cuda()
    data[where] = near.data
    if fp8:
        scale[where] = near.scale
    far = idx.Cache(data, scale, fmt=near.fmt)
    s = _lists(rng, T, n, len(at))
    big = np.where(s >= 0, at[np.maximum(s, 0)], -1).astype(np.int32)
    q = _q(3, T, H * G, D, dtype).cuda()
    a = idx.idx_sparse_attn(q, far, far, torch.from_numpy(big).cuda(), 0.1)
    b = idx.idx_sparse_attn(q, near, near, torch.from_numpy(s).cuda(), 0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    take = np.array([0, 1, T - 1])
    _compare(take, *a, q.cpu(), near, near, s, 0.1)


@pytest.mark.parametrize("dtype,fp8", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True),
                                       (torch.float16, True)])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 1), (64, 64, 1), (128, 16, 4)])
def test_a_row_in_calls_of_any_size(dtype, fp8, D, Hq, Hkv):
    """A row keeps its bound whatever rows are beside it, and its bits whatever these hold."""
    rng = np.random.default_rng(D)
    k, v = _caches(5, 4000, Hkv, D, dtype, fp8)
    q = _q(9, 1, Hq, D, dtype)
    s = np.sort(rng.choice(4000, 1500, replace=False)).astype(np.int32)[None]
    for T in (1, 2, 9, 40, 130, 270, 400, 800, 1300):
        at, results = T // 3, []
        for other in range(2):
            qs = _q(T + other, T, Hq, D, dtype)
            ids = np.sort(rng.integers(-1000, 4000, (T, 1500)), 1).astype(np.int32)
            qs[at], ids[at] = q[0], s[0]
            results.append(idx.idx_sparse_attn(qs.cuda(), k, v, torch.from_numpy(ids).cuda(), 0.1))
            out, lse = results[-1]
            _compare(np.array([0]), out[at:at + 1], lse[at:at + 1], q, k, v, s, 0.1)
        for a, b in zip(*results):
            assert torch.equal(a[at], b[at])
