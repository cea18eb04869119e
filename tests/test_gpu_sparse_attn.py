"""Attention over selected keys and blocks against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import mqa_logits_top_amd as idx
from around_ref import attend, keys_of, read_e4m3

pytestmark = pytest.mark.gpu

FP8 = idx.IDX_K_FP8_E4M3
VALUE = {torch.bfloat16: idx.IDX_K_BF16, torch.float16: idx.IDX_K_F16}


def _caches(seed, rows, H, D, dtype, fp8, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        x = (torch.randn((rows, H, D), generator=g) * gain).to(dtype)
        c = idx.Cache.empty(rows, H, D, FP8 if fp8 else VALUE[dtype])
        idx.idx_cache_write([idx.Write(x.cuda(), c)])
        out.append(c)
    return out


def _values(c):
    if c.fmt == FP8:
        return read_e4m3(c.data.cpu().numpy(), c.scale.cpu().numpy())
    return c.data.cpu().double().numpy()


def _check(q, k, v, sel, scale, pool=1, ks=None, ke=None, table=None, **kw):
    cu = lambda a: None if a is None else torch.as_tensor(a, dtype=torch.int32).cuda()
    out, lse = idx.idx_sparse_attn(q.cuda(), k, v, cu(sel), scale, pool=pool, ks=cu(ks), ke=cu(ke),
                                   slot_of_key=cu(table), **kw)
    _compare(out, lse, q, k, v, sel, scale, pool, ks, ke, table)
    return out, lse


def _compare(out, lse, q, k, v, sel, scale, pool=1, ks=None, ke=None, table=None):
    rows = keys_of(np.asarray(sel), ks, ke, pool, k.rows if table is None else len(table), table, k.rows)
    # fp16 with E4M3 caches: weights in two bf16 parts, the second's half step of what the first left
    step = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -16 if k.fmt == FP8 else 2.0 ** -11
    want, wl, bo, bl = attend(q.double().numpy(), _values(k), _values(v), rows, scale, step, q.dtype)
    got, gl = out.cpu().double().numpy(), lse.cpu().double().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
    err = np.abs(got - want)
    assert (err <= bo).all(), f"out: {(err > bo).sum()} off, worst {np.max(err / bo):.2f} of the bound"
    fin = np.isfinite(wl)
    assert (np.abs(gl[fin] - wl[fin]) <= bl[fin]).all(), "lse"


def _sel(rng, T, n, L, holes=0.0):
    s = np.stack([np.sort(rng.choice(L, min(n, L), replace=False)) for _ in range(T)]).astype(np.int32)
    s = np.concatenate([s, np.full((T, n - s.shape[1]), -1, np.int32)], 1)
    s[rng.random(s.shape) < holes] = -1
    return s


def _q(seed, T, Hq, D, dtype, gain=2.0):
    return (torch.randn((T, Hq, D), generator=torch.Generator().manual_seed(seed)) * gain).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (16, 1), (32, 1), (64, 1), (80, 1), (128, 1), (24, 8), (6, 6), (51, 3)])
def test_head_layouts(dtype, fp8, D, Hq, Hkv):
    rng = np.random.default_rng(Hq * D)
    k, v = _caches(1, 500, Hkv, D, dtype, fp8)
    _check(_q(2, 3, Hq, D, dtype), k, v, _sel(rng, 3, 100, 500), D ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,n", [(1, 1), (1, 2), (2, 31), (1, 32), (3, 33), (1, 127), (1, 129), (5, 300), (1, 2048),
                                 (700, 40), (1100, 1)])
def test_list_lengths(T, n, fp8):
    """From one key of one row to many rows and long lists: split and unsplit forms, tiles that end anywhere."""
    rng = np.random.default_rng(n)
    k, v = _caches(3, 3000, 1, 128, torch.bfloat16, fp8)
    _check(_q(4, T, 8, 128, torch.bfloat16), k, v, _sel(rng, T, n, 3000), 0.1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq,n", [(1030, 32, 70), (600, 50, 33), (512, 64, 100), (385, 40, 65)])
def test_many_rows_of_many_heads(dtype, fp8, D, T, Hq, n):
    """Rows that fill the machine take 32 heads to a wave."""
    rng = np.random.default_rng(T)
    k, v = _caches(21, 400, 1, D, dtype, fp8)
    s = _sel(rng, T, n, 400, holes=0.1)
    s[3] = -1
    s[7, :] = -1
    s[7, 5] = 11
    _check(_q(22, T, Hq, D, dtype), k, v, s, D ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,Hkv,n", [(300, 1, 700), (33, 8, 900), (2, 2, 3000), (130, 1, 300),
                                     (900, 1, 200), (128, 1, 1100), (16, 8, 1100)])
def test_divided_lists(T, Hkv, n, fp8):
    """Lists divided over workgroups, over waves, and over both; holes and an empty row among them."""
    rng = np.random.default_rng(n)
    k, v = _caches(23, 4000, Hkv, 64, torch.bfloat16, fp8)
    s = _sel(rng, T, n, 4000, holes=0.2)
    s[1] = -1
    s[0, : n // 2] = -1
    _check(_q(24, T, 4 * Hkv, 64, torch.bfloat16), k, v, s, 0.15)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30])
@pytest.mark.parametrize("fp8", [False, True])
def test_scales_of_any_sign(scale, fp8):
    rng = np.random.default_rng(3)
    k, v = _caches(25, 300, 2, 64, torch.float16, fp8)
    _check(_q(26, 5, 32, 64, torch.float16), k, v, _sel(rng, 5, 200, 300), scale)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,n", [(6, 70), (40, 515)])
def test_holes_and_empty_rows(T, n, fp8):
    """-1 anywhere in a list, whole tiles of it, lists of nothing, one key, ids outside the cache and repeats."""
    rng = np.random.default_rng(n)
    k, v = _caches(5, 600, 2, 64, torch.bfloat16, fp8)
    s = _sel(rng, T, n, 600, holes=0.4)
    s[0] = -1
    s[1] = -1
    s[1, n - 1] = 599
    s[2, :64] = -1
    s[3, 3:9] = 17
    s[4, 0], s[4, 1], s[4, 2] = 600, 2 ** 31 - 1, -2 ** 31
    out, lse = _check(_q(6, T, 32, 64, torch.bfloat16), k, v, s, 0.125)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    none, l0 = idx.idx_sparse_attn(_q(6, T, 32, 64, torch.bfloat16).cuda(), k, v,
                                   torch.empty((T, 0), dtype=torch.int32, device="cuda"), 0.125)
    assert (none == 0).all() and torch.isneginf(l0).all()


@pytest.mark.parametrize("T", [1, 9])
def test_windows_and_table(T):
    """Ids outside their row's window do not count; keys go through the slot table, whose own holes do not count
    either."""
    rng = np.random.default_rng(T)
    L, rows = 900, 1300
    k, v = _caches(7, rows, 2, 128, torch.float16, False)
    table = rng.permutation(rows)[:L].astype(np.int32)
    table[rng.integers(0, L, 40)] = -1
    table[5], table[6] = rows, 2 ** 31 - 1
    ks = rng.integers(0, 300, T).astype(np.int32)
    ke = (ks + rng.integers(0, 600, T)).astype(np.int32)
    ke[0] = ks[0]
    _check(_q(8, T, 8, 128, torch.float16), k, v, _sel(rng, T, 400, L, holes=0.05), 0.08, ks=ks, ke=ke, table=table)


@pytest.mark.parametrize("pool", [2, 8, 64])
@pytest.mark.parametrize("table", [False, True])
@pytest.mark.parametrize("T", [1, 12])
def test_blocks(pool, table, T):
    """Block lists: blocks count from the row's window, the last one may be partial, ids past it hold nothing."""
    rng = np.random.default_rng(pool + T)
    L = 1111
    k, v = _caches(9, 1500 if table else L, 2, 64, torch.bfloat16, True)
    ks = rng.integers(0, 500, T).astype(np.int32)
    ke = np.minimum(ks + rng.integers(1, 700, T), L).astype(np.int32)
    n = 40
    s = np.full((T, n), -1, np.int32)
    for t in range(T):
        nb = -(-int(ke[t] - ks[t]) // pool)
        pick = np.sort(rng.choice(nb, min(n - 3, nb), replace=False))
        s[t, :len(pick)] = pick
        s[t, 0] = nb - 1
    s[:, n - 2] = 2 ** 31 - 1
    tab = rng.permutation(1500)[:L].astype(np.int32) if table else None
    _check(_q(10, T, 16, 64, torch.bfloat16), k, v, s, 0.2, pool=pool, ks=ks, ke=ke, table=tab)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_that_do_not_count_are_not_seen(fp8):
    """NaN and infinities in every cache row that no entry names, in the row before and behind, and under masked
    entries: the outputs do not change."""
    rng = np.random.default_rng(0)
    k, v = _caches(11, 400, 2, 128, torch.bfloat16, fp8)
    used = np.sort(rng.choice(400, 90, replace=False))
    used = used[(used != 0) & (used != 399)]
    s = np.full((3, 130), -1, np.int32)
    for t in range(3):
        pick = rng.choice(used, 45, replace=False)
        s[t, rng.permutation(130)[:45]] = pick
    q = _q(12, 3, 16, 128, torch.bfloat16)
    a = _check(q, k, v, s, 0.09)
    unused = torch.from_numpy(np.setdiff1d(np.arange(400), s[s >= 0])).cuda()
    for c in (k, v):
        if fp8:
            c.data[unused] = 0x7F
            c.scale[unused] = float("inf")
        else:
            c.data[unused] = float("nan")
    b = idx.idx_sparse_attn(q.cuda(), k, v, torch.from_numpy(s).cuda(), 0.09)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_not_finite_rows_that_count():
    """A NaN in a value reaches its own dims only; one in a key reaches the whole row; others stay."""
    k, v = _caches(13, 64, 1, 64, torch.bfloat16, False)
    s = np.tile(np.arange(40, dtype=np.int32), (2, 1))
    s[1] += 20
    q = _q(14, 2, 16, 64, torch.bfloat16)
    clean = idx.idx_sparse_attn(q.cuda(), k, v, torch.from_numpy(s).cuda(), 0.1)
    v.data[7, 0, 5] = float("nan")
    out, lse = idx.idx_sparse_attn(q.cuda(), k, v, torch.from_numpy(s).cuda(), 0.1)
    assert out[0, :, 5].isnan().all() and out[0].isnan().sum() == 16
    assert torch.equal(out[1], clean[0][1]) and torch.equal(lse, clean[1])
    k.data[3] = float("nan")
    out, lse = idx.idx_sparse_attn(q.cuda(), k, v, torch.from_numpy(s).cuda(), 0.1)
    assert out[0].isnan().all() and lse[0].isnan().all() and torch.equal(out[1], clean[0][1])


@pytest.mark.parametrize("gain", [1e-3, 30.0])
@pytest.mark.parametrize("fp8", [False, True])
def test_flat_and_peaked(gain, fp8):
    """Scores that are all alike, and scores hundreds apart (weights that vanish)."""
    rng = np.random.default_rng(1)
    k, v = _caches(15, 800, 1, 128, torch.bfloat16, fp8)
    _check(_q(16, 4, 32, 128, torch.bfloat16, gain), k, v, _sel(rng, 4, 500, 800), 0.3)


@pytest.mark.parametrize("gain", [1e-20, 1e15])
def test_e4m3_scales_far_from_one(gain):
    """Scales far outside fp16's range: weights times scales keep bf16's."""
    rng = np.random.default_rng(2)
    x = torch.randn((300, 1, 64), generator=torch.Generator().manual_seed(3))
    k, v = idx.Cache.empty(300, 1, 64, FP8), idx.Cache.empty(300, 1, 64, FP8)
    idx.idx_cache_write([idx.Write(x.cuda(), k), idx.Write((x.flip(0) * gain).cuda(), v)])
    _check(_q(17, 3, 16, 64, torch.bfloat16), k, v, _sel(rng, 3, 200, 300), 0.1)


def test_strides():
    """q and out as slices of wider buffers and head by head, caches interleaved in one buffer, lists with a
    pitch: the same bits as rows of their own, nothing beside them touched."""
    rng = np.random.default_rng(4)
    T, Hq, Hkv, D, rows = 7, 12, 2, 64, 200
    both = torch.randn((rows, 2 * Hkv, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    k, v = idx.Cache(both[:, :Hkv], fmt=idx.IDX_K_BF16), idx.Cache(both[:, Hkv:], fmt=idx.IDX_K_BF16)
    kc = idx.Cache(both[:, :Hkv].contiguous(), fmt=idx.IDX_K_BF16)
    vc = idx.Cache(both[:, Hkv:].contiguous(), fmt=idx.IDX_K_BF16)
    wide = _q(5, T, 2 * Hq, D, torch.bfloat16).cuda()
    sel = torch.from_numpy(_sel(rng, T, 90, rows)).cuda()
    pitched = torch.full((T, 120), 3, dtype=torch.int32, device="cuda")
    pitched[:, 11:101] = sel
    want, wl = idx.idx_sparse_attn(wide[:, Hq:].contiguous(), kc, vc, sel, 0.1)
    out = torch.full((Hq + 2, T + 1, D), 9.0, dtype=torch.bfloat16, device="cuda")
    idx.idx_sparse_attn(wide[:, Hq:], k, v, pitched[:, 11:101], 0.1, out=out[1:-1, :T].transpose(0, 1))
    assert torch.equal(out[1:-1, :T].transpose(0, 1), want)
    assert (out[0] == 9).all() and (out[-1] == 9).all() and (out[:, T] == 9).all()


def test_long_cache_offsets():
    """Cache rows whose bytes lie past 2^32."""
    rows, H, D = 3_000_000, 8, 128
    data = torch.zeros((rows, H, D), dtype=torch.bfloat16, device="cuda")      # 6.1 GB
    at = torch.tensor([5, 2_097_151, 2_097_152 + 77, rows - 1], dtype=torch.int32)
    small = (torch.randn((4, H, D), generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).cuda()
    data[at.long().cuda()] = small
    big, near = idx.Cache(data, fmt=idx.IDX_K_BF16), idx.Cache(small, fmt=idx.IDX_K_BF16)
    q = _q(3, 2, 16, D, torch.bfloat16).cuda()
    a = idx.idx_sparse_attn(q, big, big, at.cuda().expand(2, 4).contiguous(), 0.1)
    b = idx.idx_sparse_attn(q, near, near, torch.arange(4, dtype=torch.int32, device="cuda").expand(2, 4).contiguous(),
                            0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T,Hq,fp8", [(1100, 32, False), (1100, 32, True), (2, 16, True)])
def test_long_cache_offsets_of_one_head(T, Hq, fp8):
    """The same with many rows of many heads, and with E4M3 codes."""
    rows, D = (40_000_000 if fp8 else 20_000_000), 128                         # 5.1 GB
    at = torch.tensor([9, rows // 2, rows // 3, rows - 1], dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    small = idx.Cache.empty(4, 1, D, FP8 if fp8 else idx.IDX_K_BF16)
    idx.idx_cache_write([idx.Write(torch.randn((4, 1, D), generator=g).to(torch.bfloat16).cuda(), small)])
    data = torch.zeros((rows, 1, D), dtype=small.data.dtype, device="cuda")
    scale = torch.zeros((rows, 1), device="cuda") if fp8 else None
    big = idx.Cache(data, scale, fmt=small.fmt)
    data[at.long().cuda()] = small.data
    if fp8:
        scale[at.long().cuda()] = small.scale
    q = _q(3, T, Hq, D, torch.bfloat16).cuda()
    sel = torch.arange(4, dtype=torch.int32).expand(T, 4).contiguous()
    a = idx.idx_sparse_attn(q, big, big, at.expand(T, 4).contiguous().cuda(), 0.1)
    b = idx.idx_sparse_attn(q, small, small, sel.cuda(), 0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals():
    """What the binding and the C entry point refuse."""
    k, v = _caches(1, 20, 2, 64, torch.bfloat16, False)
    q, s = _q(1, 3, 4, 64, torch.bfloat16).cuda(), torch.zeros((3, 5), dtype=torch.int32, device="cuda")
    w = torch.zeros(3, dtype=torch.int32, device="cuda")
    f8 = idx.Cache.empty(20, 2, 64)
    for bad in (lambda: idx.idx_sparse_attn(q, k, v, s.long(), 0.1), lambda: idx.idx_sparse_attn(q, k, v, s[:2], 0.1),
                lambda: idx.idx_sparse_attn(q, k, v, s.cpu(), 0.1), lambda: idx.idx_sparse_attn(q.cpu(), k, v, s, 0.1),
                lambda: idx.idx_sparse_attn(q, k, v, s, 0.1, ks=w), lambda: idx.idx_sparse_attn(q, k, v, s.t(), 0.1),
                lambda: idx.idx_sparse_attn(q, k, v, s, 0.1, ks=w, ke=w[:2]),
                lambda: idx.idx_sparse_attn(q, k, v, s, 0.1, slot_of_key=w.long()),
                lambda: idx.idx_sparse_attn(q, k, v, s, 0.1, lse=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: idx.idx_sparse_attn(q[:, :3], k, v, s, 0.1), lambda: idx.idx_sparse_attn(q.half(), k, v, s, 0.1),
                lambda: idx.idx_sparse_attn(q, k, f8, s, 0.1), lambda: idx.idx_sparse_attn(q, k, v, s, 0.1, pool=8),
                lambda: idx.idx_sparse_attn(q.float(), k, v, s, 0.1),
                lambda: idx.idx_sparse_attn(q, k, v, s, float("nan"))):
        with pytest.raises(idx.IdxError):
            bad()


def test_debug_mode_checks_windows(monkeypatch):
    k, v = _caches(1, 20, 1, 64, torch.bfloat16, False)
    q, s = _q(1, 2, 4, 64, torch.bfloat16).cuda(), torch.zeros((2, 5), dtype=torch.int32, device="cuda")
    w = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    monkeypatch.setenv("IDX_DEBUG", "1")
    idx.idx_sparse_attn(q, k, v, s, 0.1, ks=w(0, 3), ke=w(20, 3))
    with pytest.raises(idx.IdxError) as e:
        idx.idx_sparse_attn(q, k, v, s, 0.1, ks=w(0, 4), ke=w(21, 5))
    assert e.value.status == 9


def test_two_graphs_beside_each_other():
    """Two captured calls with workspaces of their own, replayed in turn and between eager calls."""
    rng = np.random.default_rng(8)
    k, v = _caches(27, 5000, 1, 128, torch.bfloat16, True)
    calls = []
    for i in range(2):
        q, s = _q(30 + i, 1, 16, 128, torch.bfloat16).cuda(), torch.from_numpy(_sel(rng, 1, 2048, 5000)).cuda()
        want = [x.clone() for x in idx.idx_sparse_attn(q, k, v, s, 0.09)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = idx.idx_sparse_attn(q, k, v, s, 0.09)
        calls.append((g, out, want, q, s))
    for turn in range(4):
        for g, out, want, _, _ in calls:
            out[0].fill_(3)
            g.replay()
        idx.idx_sparse_attn(calls[0][3], k, v, calls[1][4], 0.3)
        torch.cuda.synchronize()
        for g, out, want, _, _ in calls:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_large_cache_of_many_heads(fp8):
    """Rows of a cache that no on-chip memory holds are divided over workgroups of one wave."""
    rng = np.random.default_rng(12)
    H, rows = 8, 140_000 if fp8 else 70_000                                     # 143 MB both
    k, v = _caches(41, rows, H, 64, torch.bfloat16, fp8)
    q, s = _q(42, 40, 4 * H, 64, torch.bfloat16), _sel(rng, 40, 2 * rows // 40, rows)
    take = slice(17, 20)                                                        # three rows against 64 bits
    out, lse = idx.idx_sparse_attn(q.cuda(), k, v, torch.from_numpy(s).cuda(), 0.12)
    at = [np.unique(s[take]), None]
    at[1] = np.searchsorted(at[0], s[take]).astype(np.int32)
    few = torch.from_numpy(at[0]).long().cuda()
    small = [idx.Cache(c.data[few], None if c.scale is None else c.scale[few], fmt=c.fmt) for c in (k, v)]
    _compare(out[take], lse[take], q[take], *small, at[1], 0.12)


@pytest.mark.parametrize("fp8", [False, True])
def test_nothing_to_attend_to(fp8):
    """No rows, no entries, no keys, a cache without slots."""
    k, v = _caches(1, 20, 2, 64, torch.bfloat16, fp8)
    e = [idx.Cache.empty(0, 2, 64, k.fmt) for _ in range(2)]
    q = _q(1, 3, 4, 64, torch.bfloat16).cuda()
    ids = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
    out, lse = idx.idx_sparse_attn(q[:0], k, v, ids(0, 5), 0.1)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    for c, s, kw in ((k, v), ids(3, 0), {}), (e, ids(3, 5), {}), (e, ids(3, 2000), {}), ((k, v), ids(3, 5), dict(
            slot_of_key=ids(0))), ((k, v), ids(3, 5), dict(ks=ids(3), ke=ids(3))), (e, ids(3, 5), dict(
            slot_of_key=ids(9))):
        out, lse = idx.idx_sparse_attn(q, *c, s, 0.1, **kw)
        assert not out.any() and torch.isneginf(lse).all()


def test_two_threads():
    """Two host threads, each with its stream."""
    import threading
    rng = np.random.default_rng(13)
    k, v = _caches(43, 3000, 1, 128, torch.bfloat16, True)
    q = [_q(44 + i, 3, 32, 128, torch.bfloat16).cuda() for i in range(2)]
    s = [torch.from_numpy(_sel(rng, 3, 1500, 3000)).cuda() for _ in range(2)]
    want = [idx.idx_sparse_attn(q[i], k, v, s[i], 0.1) for i in range(2)]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        side = torch.cuda.Stream()
        for _ in range(20):
            got[i].append(idx.idx_sparse_attn(q[i], k, v, s[i], 0.1, stream=side))
        side.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 20
        assert all(torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]) for o, l in got[i])


def test_repeatable_and_other_streams():
    """The same bits on every call, on another stream, and with a workspace full of NaN."""
    rng = np.random.default_rng(6)
    k, v = _caches(18, 5000, 1, 128, torch.bfloat16, True)
    q, sel = _q(19, 2, 64, 128, torch.bfloat16).cuda(), torch.from_numpy(_sel(rng, 2, 2000, 5000)).cuda()
    want = idx.idx_sparse_attn(q, k, v, sel, 0.09)
    for _ in range(5):
        got = idx.idx_sparse_attn(q, k, v, sel, 0.09)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = idx.idx_sparse_attn(q, k, v, sel, 0.09, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    got = idx.idx_sparse_attn(q, k, v, sel, 0.09, ws=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_layer_around_the_indexer():
    """The operators in the order a layer uses them: rotate and quantise q, keys and values into caches, select
    through the slot table, attend to what was selected; against the same steps in 64 bits on the codes the
    caches hold.  Then the layer captured in a graph and replayed between eager work."""
    T, L, H, Hq, Hkv, D, K = 24, 1200, 32, 16, 2, 128, 128
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
    plan = idx.Rotary.make(64)
    xq, xk, aq, ak, av = n(T, H, 128), n(L, 1, 128), n(T, Hq, D), n(L, Hkv, D), n(L, Hkv, D)
    w = torch.rand((T, H), generator=g).cuda()
    pos_k = torch.arange(L, dtype=torch.int32, device="cuda")
    pos_q = pos_k[L - T:].contiguous()
    table = torch.randperm(L, generator=g).to(torch.int32).cuda()
    ks, ke = torch.zeros(T, dtype=torch.int32, device="cuda"), pos_q + 1
    iq, ik = idx.Cache.empty(T, H, 128), idx.Cache.empty(L, 1, 128)
    ck, cv = idx.Cache.empty(L, Hkv, D), idx.Cache.empty(L, Hkv, D)
    d = idx.Inputs(q=iq.data, q_scale=iq.scale, k=ik.data.view(L, 128), k_scale=ik.scale.view(L), w=w, ks=ks, ke=ke)
    ws = torch.empty(idx.idx_workspace_size(idx.IDX_OP_LOGITS_TOPK_FUSED, d, K=K, block_k=512), dtype=torch.uint8,
                     device="cuda")

    def layer():
        idx.idx_cache_write([idx.Write(xq, iq, rotary=plan, pos=pos_q), idx.Write(xk, ik, rotary=plan, pos=pos_k),
                             idx.Write(ak, ck, slot=table, rotary=plan, pos=pos_k), idx.Write(av, cv, slot=table)])
        q = idx.idx_rope(aq, pos_q, plan)
        sel, _ = idx.idx_logits_topk_fused(d, K, block_k=512, ws=ws)
        out, lse = idx.idx_sparse_attn(q, ck, cv, sel, D ** -0.5, ks=ks, ke=ke, slot_of_key=table)
        return q, sel, out, lse

    q, sel, out, lse = layer()
    rows = keys_of(sel.cpu().numpy(), ks.cpu().numpy(), ke.cpu().numpy(), 1, L, table.cpu().numpy(), L)
    assert all(len(r) == K for r in rows)
    want, wl, bo, bl = attend(q.cpu().double().numpy(), _values(ck), _values(cv), rows, D ** -0.5, 2.0 ** -8,
                              torch.bfloat16)
    assert (np.abs(out.cpu().double().numpy() - want) <= bo).all()
    assert (np.abs(lse.cpu().double().numpy() - wl) <= bl).all()
    eager = [x.clone() for x in (q, sel, out, lse)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for _ in range(4):
        for c in (iq, ik, ck, cv):
            c.data.zero_()
        for x in held:
            x.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        idx.idx_sparse_attn(q, ck, cv, sel, 0.5)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager))
