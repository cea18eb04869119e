"""Attention over every key, or a window, of a paged cache against its formula in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import mqa_logits_top_amd as idx
from around_ref import attend, read_e4m3
from dense_ref import slots_seen, weight_step

pytestmark = pytest.mark.gpu

FP8 = idx.IDX_K_FP8_E4M3
VALUE = {torch.bfloat16: idx.IDX_K_BF16, torch.float16: idx.IDX_K_F16}
BF16, F16 = torch.bfloat16, torch.float16


def caches(seed, rows, H, D, dtype, fp8, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        x = (torch.randn((rows, H, D), generator=g) * gain).to(dtype)
        c = idx.Cache.empty(rows, H, D, FP8 if fp8 else VALUE[dtype])
        idx.idx_cache_write([idx.Write(x.cuda(), c)])
        out.append(c)
    return out


def values(c):
    if c.fmt == FP8:
        return read_e4m3(c.data.cpu().numpy(), c.scale.cpu().numpy())
    return c.data.cpu().double().numpy()


def batch(seed, new, lens, page, spare=0, holes=0):
    """cu_q, len_k and a table of pages in any order: (cu_q, len_k, pages, slots)."""
    rng = np.random.default_rng(seed)
    held = [-(-max(x, 0) // page) for x in lens]
    total = sum(held) + 2
    order = rng.permutation(total).astype(np.int32)
    table = rng.integers(-5, total + 5, (len(lens), max(held + [0]) + spare)).astype(np.int32)
    at = 0
    for b, p in enumerate(held):
        table[b, :p] = order[at:at + p]
        at += p
    for _ in range(holes):
        b = int(rng.integers(len(lens)))
        if held[b]:
            table[b, int(rng.integers(held[b]))] = rng.choice([-1, -2 ** 31, total, 2 ** 31 - 1])
    return np.cumsum([0] + list(new)).astype(np.int32), np.asarray(lens, np.int32), table, total * page


def queries(seed, T, Hq, D, dtype, gain=2.0):
    return (torch.randn((T, Hq, D), generator=torch.Generator().manual_seed(seed)) * gain).to(dtype)


def gpu(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def compare(out, lse, q, k, v, pages, page, cu, lens, scale, window=0, first=0, rows=None):
    """rows: those to compare (all)."""
    seen = slots_seen(q.shape[0], pages, page, cu, lens, k.rows, window, first)
    pick = [t for t in (range(q.shape[0]) if rows is None else rows) if seen[t] is not None]
    got, gl = out[pick].cpu().double().numpy(), lse[pick].cpu().double().numpy()
    want, wl, bo, bl = attend(q[pick].double().numpy(), values(k), values(v), [seen[t] for t in pick], scale,
                              weight_step(q.dtype == BF16, k.fmt == FP8), q.dtype)
    assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
    err = np.abs(got - want)
    assert (err <= bo).all(), f"out: {(~(err <= bo)).sum()} off, worst {np.nanmax(err / bo):.2f} of the bound"
    fin = np.isfinite(wl)
    assert (np.abs(gl[fin] - wl[fin]) <= bl[fin]).all(), "lse"


def check(q, k, v, b, page, scale, window=0, first=0, rows=None, **kw):
    cu, lens, pages, _ = b
    out, lse = idx.idx_paged_attn(q.cuda(), k, v, gpu(pages), gpu(cu), gpu(lens), scale, page=page, window=window,
                                  first=first, **kw)
    compare(out, lse, q, k, v, pages, page, cu, lens, scale, window, first, rows)
    return out, lse


HEADS = [(1, 1), (8, 1), (16, 1), (32, 1), (64, 1), (80, 1), (128, 1), (24, 8), (32, 8), (6, 6), (51, 3), (28, 4)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_head_layouts(dtype, fp8, D, Hq, Hkv):
    """Single rows, a few rows and a chunk beside each other."""
    b = batch(1, [1, 5, 20, 1], [70, 5, 131, 1], 16)
    k, v = caches(1, b[3], Hkv, D, dtype, fp8)
    check(queries(2, 27, Hq, D, dtype), k, v, b, 16, D ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (32, 8), (5, 5), (64, 2), (21, 3)])
def test_chunks(dtype, fp8, D, Hq, Hkv):
    """Rows enough for the widest tiles, on prefixes of odd lengths."""
    b = batch(3, [150, 33, 259], [150, 700, 1003], 64)
    k, v = caches(4, b[3], Hkv, D, dtype, fp8)
    check(queries(5, 442, Hq, D, dtype), k, v, b, 64, D ** -0.5, rows=[0, 1, 31, 63, 64, 148, 149, 150, 182, 183, 300, 440, 441])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 128, 4096])
@pytest.mark.parametrize("new", [[1, 1, 1], [90, 3, 40]])
def test_pages(page, new, fp8):
    """Pages that end inside a tile, that hold several, ids of any kind behind the last, a strided table."""
    b = batch(6, new, [new[0], 333, 257], page, spare=3)
    k, v = caches(7, b[3], 2, 128, BF16, fp8)
    check(queries(8, sum(new), 8, 128, BF16), k, v, b, page, 0.09)
    wide = torch.zeros((3, b[2].shape[1] + 5), dtype=torch.int32, device="cuda")
    wide[:, :b[2].shape[1]] = gpu(b[2])
    q = queries(8, sum(new), 8, 128, BF16).cuda()
    args = (gpu(b[0]), gpu(b[1]), 0.09)
    one = idx.idx_paged_attn(q, k, v, gpu(b[2]), *args, page=page)
    two = idx.idx_paged_attn(q, k, v, wide[:, :b[2].shape[1]], *args, page=page)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,n", [(1, 1), (1, 2), (1, 31), (1, 32), (1, 33), (1, 64), (1, 65), (1, 127), (1, 1025), (1, 20000),
                                 (2, 20000), (9, 9000), (70, 9000), (300, 5000)])
def test_lengths_of_one_request(T, n, fp8):
    """From one key of one token to long prefixes, whose keys are divided."""
    b = batch(9, [T], [max(n, T)], 32)
    k, v = caches(10, b[3], 1, 128, BF16, fp8)
    check(queries(11, T, 8, 128, BF16), k, v, b, 32, 0.1, rows=sorted({0, T // 2, T - 1}))


@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (5, 0), (64, 0), (64, 4), (100, 64), (77, 65), (1000, 3), (10 ** 9, 5),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (130, 2 ** 31 - 1), (3, 200)])
@pytest.mark.parametrize("fp8,D", [(False, 128), (True, 64)])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [150, 2, 47, 1]])
def test_windows(window, first, fp8, D, new):
    b = batch(12, new, [new[0], 700, 333, 64], 16)
    k, v = caches(13, b[3], 2, D, F16, fp8)
    check(queries(14, sum(new), 8, D, F16), k, v, b, 16, D ** -0.5, window=window, first=first)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,lens", [([0, 3, 0, 0, 1, 0], [5, 9, 0, 77, 100, 0]), ([4, 2], [2, 0]), ([40, 1], [10, 0]),
                                      ([0, 0], [5, 5]), ([1] * 70, list(range(1, 71))), ([2] * 130, [3 * i % 97 for i in range(130)])])
@pytest.mark.parametrize("window", [0, 20])
def test_requests_of_any_kind(new, lens, window, fp8):
    """Requests without rows or keys, rows without keys, more requests than lanes."""
    b = batch(15, new, lens, 8, spare=2)
    k, v = caches(16, b[3], 2, 64, BF16, fp8)
    if sum(new):
        check(queries(17, sum(new), 8, 64, BF16), k, v, b, 8, 0.125, window=window, first=2)


@pytest.mark.parametrize("new,lens", [([1, 1, 1], [100, 300, 40]), ([60, 5], [60, 290])])
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_of_no_request_stay(new, lens, fp8):
    """Rows before the first request and behind the last keep what out and lse held."""
    cu, lens, pages, slots = batch(18, new, lens, 16)
    T = sum(new) + 7
    k, v = caches(19, slots, 1, 128, BF16, fp8)
    q = queries(20, T, 16, 128, BF16)
    for cu in (cu, cu + 3):
        out = torch.full((T, 16, 128), 7.0, dtype=BF16, device="cuda")
        lse = torch.full((T, 16), 9.0, device="cuda")
        check(q, k, v, (cu, lens, pages, slots), 16, 0.1, out=out, lse=lse)
        none = [t for t in range(T) if t < cu[0] or t >= cu[-1]]
        assert (out[none] == 7).all() and (lse[none] == 9).all()


def test_lengths_past_the_table_end_with_it():
    cu, lens, pages, slots = batch(21, [3, 1], [64, 48], 16)
    k, v = caches(22, slots, 1, 64, BF16, False)
    q = queries(23, 4, 4, 64, BF16)
    pages[1, 3] = pages[0, 0]
    check(q, k, v, (cu, np.array([2 ** 31 - 1, 10 ** 6], np.int32), pages, slots), 16, 0.2)
    check(q, k, v, (cu, np.array([-5, -2 ** 31], np.int32), pages, slots), 16, 0.2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 1, 2], [130, 1, 20]])
def test_pages_outside_the_cache_do_not_count(new, fp8):
    b = batch(24, new, [300, 200, 250], 16, holes=12)
    k, v = caches(25, b[3], 2, 64, BF16, fp8)
    check(queries(26, sum(new), 8, 64, BF16), k, v, b, 16, 0.1)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 1], [100, 3]])
def test_slots_no_row_sees_may_hold_anything(new, fp8):
    """NaN and infinities behind the last key of a page, in other pages, and before the window."""
    cu, lens, pages, slots = batch(27, new, [213, 70], 16)
    k, v = caches(28, slots, 2, 64, BF16, fp8)
    q = queries(29, sum(new), 8, 64, BF16)
    for window, first in ((0, 0), (30, 3)):
        clean = idx.idx_paged_attn(q.cuda(), k, v, gpu(pages), gpu(cu), gpu(lens), 0.1, page=16, window=window, first=first)
        seen = np.unique(np.concatenate(slots_seen(sum(new), pages, 16, cu, lens, slots, window, first)))
        rest = torch.ones(slots, dtype=torch.bool)
        rest[seen] = False
        keep = [c.data.clone() for c in (k, v)]
        for c, bad in ((k, float("nan")), (v, float("inf"))):
            if fp8:
                c.data[rest.cuda()] = 0x7F
            else:
                c.data[rest.cuda()] = bad
        dirty = idx.idx_paged_attn(q.cuda(), k, v, gpu(pages), gpu(cu), gpu(lens), 0.1, page=16, window=window, first=first)
        assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])
        compare(*dirty, q, k, v, pages, 16, cu, lens, 0.1, window, first)
        for c, was in zip((k, v), keep):
            c.data.copy_(was)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4)])
@pytest.mark.parametrize("window", [0, 50])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(bad, where, Hq, Hkv, window):
    """A new token's key or value that is not finite: rows before it, and rows whose window has left it, keep their
    results; rows that see it show it."""
    new, lens = [130], [200]
    cu, lens, pages, slots = batch(30, new, lens, 16)
    k, v = caches(31, slots, Hkv, 128, BF16, False)
    q = queries(32, 130, Hq, 128, BF16)
    run = lambda: idx.idx_paged_attn(q.cuda(), k, v, gpu(pages), gpu(cu), gpu(lens), 0.1, page=16, window=window)
    clean = run()
    key = 133                                     # of row 63, in the last cache head, one dim
    slot = int(pages[0, key // 16]) * 16 + key % 16
    (k if where == "k" else v).data[slot, Hkv - 1, 5] = bad
    dirty = run()
    G = Hq // Hkv
    sees = torch.zeros((130, Hq), dtype=torch.bool)
    sees[63:(63 + window if window else 130), Hq - G:] = True
    assert torch.equal(clean[0].cpu()[~sees], dirty[0].cpu()[~sees])
    assert torch.equal(clean[1].cpu()[~sees], dirty[1].cpu()[~sees])
    got = dirty[0].cpu()[sees].float()
    if where == "v":
        assert not torch.isfinite(got[:, 5]).any()
        other = [d for d in range(128) if d != 5]
        assert torch.equal(got[:, other], clean[0].cpu()[sees].float()[:, other])
        assert torch.equal(clean[1].cpu(), dirty[1].cpu())
    elif bad != bad:
        assert torch.isnan(got).all() and torch.isnan(dirty[1].cpu()[sees]).all()


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 2], [100, 5]])
def test_scales_of_any_sign(scale, fp8, new):
    b = batch(33, new, [110, 200], 16)
    k, v = caches(34, b[3], 2, 64, F16, fp8)
    check(queries(35, sum(new), 16, 64, F16), k, v, b, 16, scale)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [[1, 1], [70, 2]])
def test_scores_of_any_size(D, new):
    """Scores past 2^31 and steep ones: a row is its largest key's value."""
    b = batch(36, new, [100, 300], 16)
    k, v = caches(37, b[3], 1, D, BF16, False)
    for scale in (30.0, 1e12):
        q = queries(38, sum(new), 8, D, BF16)
        out, lse = idx.idx_paged_attn(q.cuda(), k, v, gpu(b[2]), gpu(b[0]), gpu(b[1]), scale, page=16)
        seen = slots_seen(sum(new), b[2], 16, b[0], b[1], k.rows)
        kk, vv = values(k), values(v)
        for t in (0, sum(new) // 2, sum(new) - 1):
            s = np.einsum("hd,nd->hn", q[t].double().numpy(), kk[seen[t], 0])
            best = s.argmax(1)
            gap = np.sort(s, 1)[:, -2:] if s.shape[1] > 1 else None
            for h in range(8):
                # the next key's score is so far below that it has no weight
                if gap is None or (gap[h, 1] - gap[h, 0]) * scale > 40 + 2.0 ** -16 * abs(gap[h, 1]) * scale:
                    assert np.array_equal(out[t, h].cpu().double().numpy(), vv[seen[t][best[h]], 0])


def test_strides_and_given_arrays():
    b = batch(39, [3, 40], [50, 90], 16)
    k, v = caches(40, b[3], 2, 64, BF16, False)
    wide = queries(41, 43 * 2, 12, 64, BF16).view(43, 2, 12, 64)[:, 0].cuda()
    q = wide[:, 2:10]
    out = torch.zeros((8, 43, 64), dtype=BF16, device="cuda").transpose(0, 1)
    lse = torch.zeros((43, 8), device="cuda")
    got = idx.idx_paged_attn(q, k, v, gpu(b[2]), gpu(b[0]), gpu(b[1]), 0.1, page=16, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    compare(out, lse, q.cpu(), k, v, b[2], 16, b[0], b[1], 0.1)
    plain = idx.idx_paged_attn(q.contiguous(), k, v, gpu(b[2]), gpu(b[0]), gpu(b[1]), 0.1, page=16, with_lse=False)
    assert plain[1] is None and torch.equal(plain[0], out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 1], [80, 2]])
def test_slots_further_apart(new, fp8):
    """K and V as the halves of one array of slots."""
    b = batch(42, new, [100, 300], 32)
    H, D = 2, 64
    both = torch.zeros((b[3], 2, H, D), dtype=torch.uint8 if fp8 else BF16, device="cuda")
    scales = torch.ones((b[3], 2, H), device="cuda") if fp8 else None
    k, v = (idx.Cache(both[:, i], None if scales is None else scales[:, i], fmt=FP8 if fp8 else idx.IDX_K_BF16)
            for i in range(2))
    g = torch.Generator().manual_seed(43)
    for c in (k, v):
        idx.idx_cache_write([idx.Write(torch.randn((b[3], H, D), generator=g).to(BF16).cuda(), c)])
    check(queries(44, sum(new), 8, D, BF16), k, v, b, 32, 0.125)


@pytest.mark.parametrize("fp8", [False, True])
def test_caches_past_32_bits(fp8):
    """Slots whose bytes lie past 2^32, for single rows and for a chunk."""
    H, D, page = 8, 128, 64
    rows = (1 << 32) // (H * D * (1 if fp8 else 2)) + 4096
    k, v = (idx.Cache.empty(rows, H, D, FP8 if fp8 else idx.IDX_K_BF16) for _ in range(2))
    n = 500
    for new in ([1], [130]):
        top = np.arange(rows // page - 8, rows // page, dtype=np.int32)[None, ::-1].copy()
        at = (torch.from_numpy(np.ascontiguousarray(top[0])).long()[:, None] * page + torch.arange(page)).flatten()[:n]
        g = torch.Generator().manual_seed(45)
        x = [torch.randn((n, H, D), generator=g).to(BF16) for _ in range(2)]
        idx.idx_cache_write([idx.Write(a.cuda(), c, slot=at.to(torch.int32).cuda()) for a, c in zip(x, (k, v))])
        q = queries(46, sum(new), 16, D, BF16)
        out, lse = idx.idx_paged_attn(q.cuda(), k, v, gpu(top), gpu([0, new[0]]), gpu([n]), 0.1, page=page)
        small = [idx.Cache.empty(512, H, D, FP8 if fp8 else idx.IDX_K_BF16) for _ in range(2)]
        idx.idx_cache_write([idx.Write(a.cuda(), c) for a, c in zip(x, small)])
        same = idx.idx_paged_attn(q.cuda(), *small, gpu([list(range(8))]), gpu([0, new[0]]), gpu([n]), 0.1, page=page)
        assert torch.equal(out, same[0]) and torch.equal(lse, same[1])
    del k, v


def test_repeatable_and_independent_of_other_rows():
    b = batch(47, [1, 1, 64], [3000, 500, 900], 16)
    k, v = caches(48, b[3], 2, 128, BF16, False)
    q = queries(49, 66, 16, 128, BF16)
    run = lambda q: idx.idx_paged_attn(q.cuda(), k, v, gpu(b[2]), gpu(b[0]), gpu(b[1]), 0.1, page=16)
    one, two = run(q), run(q)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    q2 = q.clone()
    q2[:40] = float("nan")
    three = run(q2)
    assert torch.equal(one[0][40:], three[0][40:]) and torch.equal(one[1][40:], three[1][40:])


@pytest.mark.parametrize("fp8", [False, True])
def test_a_request_alone_and_among_others(fp8):
    """The same request in calls of any size keeps its result within the bound."""
    k, v = caches(50, 16 * 512, 2, 128, BF16, fp8)
    q = queries(51, 700, 8, 128, BF16)
    pages = np.random.default_rng(52).permutation(512).astype(np.int32).reshape(2, 256)
    check(q[:1], k, v, (np.array([0, 1]), np.array([2500]), pages[:1], 0), 16, 0.1)
    for n in (3, 200, 699):
        cu, lens = np.array([0, 1, 1 + n]), np.array([2500, 3000])
        check(q[:1 + n], k, v, (cu, lens, pages, 0), 16, 0.1, rows=[0, 1, n])


def test_a_captured_call_takes_new_lengths():
    """cu_q, len_k, pages, q and the caches change between the replays; two graphs share a workspace, one after the other."""
    k, v = caches(53, 64 * 40, 2, 64, BF16, False)
    T, B, page = 48, 6, 16
    q = queries(54, T, 8, 64, BF16).cuda()
    cu, lens = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    pages = torch.zeros((B, 26), dtype=torch.int32, device="cuda")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    outs = [(torch.zeros_like(q), torch.zeros((T, 8), device="cuda")) for _ in range(2)]
    call = lambda i, w: idx.idx_paged_attn(q, k, v, pages, cu, lens, 0.1, page=page, window=w, first=2, out=outs[i][0],
                                           lse=outs[i][1], ws=ws)
    call(0, 0), call(1, 33)
    torch.cuda.synchronize()
    graphs = []
    for i, w in ((0, 0), (1, 33)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, w)
        graphs.append(g)
    for r, (new, ln) in enumerate([([1] * 6, [300, 1, 50, 400, 16, 17]), ([40, 0, 3, 1, 0, 4], [40, 9, 400, 8, 0, 30]),
                                   ([8] * 6, [8, 100, 200, 300, 416, 64]), ([0, 0, 0, 0, 0, 2], [0, 0, 0, 0, 0, 5])]):
        c, n, p, _ = batch(60 + r, new, ln, page)
        p = np.pad(p % 160, ((0, 0), (0, 26 - p.shape[1])))
        cu.copy_(gpu(c)), lens.copy_(gpu(n)), pages.copy_(gpu(p))
        q.copy_(queries(70 + r, T, 8, 64, BF16))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i, w in ((0, 0), (1, 33)):
            compare(*outs[i], q.cpu(), k, v, p, page, c, n, 0.1, w, 2)


def test_streams_and_two_calls_at_once():
    b = batch(80, [1, 60], [2000, 700], 16)
    k, v = caches(81, b[3], 2, 128, BF16, False)
    q = queries(82, 61, 8, 128, BF16)
    args = (q.cuda(), k, v, gpu(b[2]), gpu(b[0]), gpu(b[1]), 0.1)
    want = idx.idx_paged_attn(*args, page=16)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [idx.idx_paged_attn(*args, page=16, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_debug_checks(monkeypatch):
    monkeypatch.setenv("IDX_DEBUG", "1")
    cu, lens, pages, slots = batch(83, [2, 3], [30, 50], 16)
    k, v = caches(84, slots, 1, 64, BF16, False)
    q = queries(85, 5, 4, 64, BF16).cuda()
    run = lambda cu, lens, pages, **kw: idx.idx_paged_attn(q, k, v, gpu(pages), gpu(cu), gpu(lens), 0.1, page=16, **kw)
    run(cu, lens, pages)
    run(cu, [1, 50], pages)                              # rows without a key are no mistake
    for bad in (([0, 3, 2], lens, pages), ([0, 2, 6], lens, pages), ([-1, 2, 5], lens, pages), (cu, [30, -1], pages),
                (cu, [30, 65], pages)):
        with pytest.raises(idx.IdxError) as e:
            run(*bad)
        assert e.value.status == 9
    worse = pages.copy()
    worse[1, 0] = slots // 16
    with pytest.raises(idx.IdxError) as e:
        run(cu, lens, worse)
    assert e.value.status == 9
    run(cu, lens, worse, window=10)                      # no row sees that page
    with pytest.raises(idx.IdxError):
        run(cu, lens, worse, window=10, first=1)


def test_nothing_to_do():
    k, v = caches(86, 64, 2, 64, BF16, False)
    for T, B in ((0, 0), (0, 3), (5, 0)):
        q = queries(87, T, 4, 64, BF16).cuda()
        out = torch.full_like(q, 3.0)
        idx.idx_paged_attn(q, k, v, torch.zeros((B, 2), dtype=torch.int32, device="cuda"), gpu([0] * (B + 1)), gpu([0] * B),
                           0.1, page=16, out=out)
        assert (out == 3).all()
    # a table without pages: rows that see nothing
    q = queries(88, 2, 4, 64, BF16).cuda()
    out, lse = idx.idx_paged_attn(q, k, v, torch.zeros((1, 0), dtype=torch.int32, device="cuda"), gpu([0, 2]), gpu([7]), 0.1,
                                  page=16)
    assert (out == 0).all() and torch.isneginf(lse).all()
    # a cache without slots
    e = [idx.Cache.empty(0, 2, 64, idx.IDX_K_BF16) for _ in range(2)]
    out, lse = idx.idx_paged_attn(q, *e, gpu([[0]]), gpu([0, 2]), gpu([7]), 0.1, page=16)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_refusals():
    k, v = caches(90, 64, 2, 64, BF16, False)
    q = queries(91, 2, 4, 64, BF16).cuda()
    good = dict(q=q, k=k, v=v, pages=gpu([[0, 1], [2, 3]]), cu_q=gpu([0, 1, 2]), len_k=gpu([7, 9]), scale=0.1, page=16)
    idx.idx_paged_attn(**good)
    small = torch.empty(8, dtype=torch.uint8, device="cuda")
    for kw in (dict(pages=gpu([0, 1])), dict(pages=gpu([[0, 1], [2, 3]]).long()), dict(pages=gpu([[0, 1], [2, 3]]).cpu()),
               dict(pages=gpu([[0, 1], [2, 3]]).t().contiguous().t()), dict(cu_q=gpu([0, 2])), dict(cu_q=gpu([0, 1, 2]).long()),
               dict(len_k=gpu([7])), dict(len_k=gpu([7, 1, 9, 1])[::2]), dict(len_k=torch.tensor([7, 9], dtype=torch.int32)),
               dict(q=q.float().requires_grad_()), dict(q=q.cpu()), dict(lse=torch.zeros((2, 3), device="cuda")),
               dict(lse=torch.zeros((2, 4), device="cuda", dtype=BF16)), dict(out=torch.zeros_like(q).cpu()),
               dict(ws=small.float())):
        with pytest.raises(ValueError):
            idx.idx_paged_attn(**(good | kw))
    for kw in (dict(window=-1), dict(first=-1), dict(page=-16), dict(window=2 ** 32 + 5)):
        with pytest.raises(ValueError):
            idx.idx_paged_attn(**(good | kw))
    for kw, status in ((dict(page=3), 6), (dict(page=0), 6), (dict(q=q[:, :3]), 2),
                       (dict(v=caches(92, 64, 2, 64, F16, False)[0]), 4), (dict(scale=float("nan")), 3)):
        with pytest.raises(idx.IdxError) as e:
            idx.idx_paged_attn(**(good | kw))
        assert e.value.status == status


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("where", ["codes", "scale"])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("T", [2, 150])
def test_quantised_values_that_are_not_finite(where, which, T, fp8):
    """The same of E4M3 codes and scales (of a value in 16 bits where there are none), for few rows and for many."""
    if where == "scale" and not fp8:
        pytest.skip("no scales")
    n = 200
    cu, lens, pages, slots = batch(100, [T], [n], 16)
    k, v = caches(101, slots, 2, 64, F16, fp8)
    q = queries(102, T, 8, 64, F16)
    run = lambda: idx.idx_paged_attn(q.cuda(), k, v, gpu(pages), gpu(cu), gpu(lens), 0.1, page=16)
    clean = run()
    key = n - T + T // 2                          # of row T // 2
    slot = int(pages[0, key // 16]) * 16 + key % 16
    c = k if which == "k" else v
    if where == "scale":
        c.scale[slot, 1] = float("inf")
    elif fp8:
        c.data[slot, 1, 7] = 0xFF
    else:
        c.data[slot, 1, 7] = float("nan")
    dirty = run()
    sees = torch.zeros((T, 8), dtype=torch.bool)
    sees[T // 2:, 4:] = True
    assert torch.equal(clean[0].cpu()[~sees], dirty[0].cpu()[~sees])
    assert torch.equal(clean[1].cpu()[~sees], dirty[1].cpu()[~sees])
    got = dirty[0].cpu()[sees].float()
    if which == "v":
        wrong = ~torch.isfinite(got)
        if where == "scale":
            # every dim whose code is not zero, and NaN where it is
            assert wrong.all()
        else:
            assert wrong[:, 7].all() and wrong.sum() == wrong[:, 7].sum()
        assert torch.equal(clean[1].cpu(), dirty[1].cpu())
    elif where == "codes":
        assert torch.isnan(got).all()


def test_more_requests_than_are_divided():
    """5000 single rows and small chunks; rows of no request between none."""
    rng = np.random.default_rng(103)
    new = rng.integers(0, 4, 5000)
    lens = new + rng.integers(0, 40, 5000)
    b = batch(104, new, lens, 8)
    k, v = caches(105, b[3], 1, 64, BF16, False)
    T = int(new.sum())
    check(queries(106, T, 4, 64, BF16), k, v, b, 8, 0.125, rows=sorted(rng.choice(T, 300, replace=False)))


@pytest.mark.parametrize("new", [[3, 1], [20, 2]])
def test_more_heads_than_a_tile_has_rows(new):
    b = batch(107, new, [100, 333], 16)
    k, v = caches(108, b[3], 1, 64, BF16, False)
    check(queries(109, sum(new), 300, 64, BF16), k, v, b, 16, 0.125)


@pytest.mark.parametrize("new", [[1], [70]])
def test_slots_past_32_bits_apart(new):
    """16 slots of a page spread over more than 2^32 bytes."""
    ld = (1 << 28) + 1024                         # bytes, E4M3
    n, rows = 30, 32
    flat = torch.empty(rows * ld, dtype=torch.uint8, device="cuda")
    small, wide = [], []
    for i in range(2):
        c = idx.Cache.empty(rows, 2, 64)
        x = (torch.randn((rows, 2, 64), generator=torch.Generator().manual_seed(110 + i))).to(BF16)
        idx.idx_cache_write([idx.Write(x.cuda(), c)])
        d = flat.as_strided((rows, 2, 64), (ld, 64, 1), 512 * i)
        d.copy_(c.data)
        small.append(c)
        wide.append(idx.Cache(d, c.scale))
    q = queries(112, sum(new), 8, 64, BF16).cuda()
    args = (gpu([[1, 0]]), gpu([0, new[0]]), gpu([n]), 0.1)
    a, b = (idx.idx_paged_attn(q, *c, *args, page=16) for c in (small, wide))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_layer_of_a_chunk_and_a_step():
    """Norm with the residual, projections, rotation into the caches, attention over everything and over a window, the
    next norm: a chunk of two requests, then a token of each, against the same in 64 bits."""
    torch.manual_seed(0)
    N, Hq, Hkv, D, page = 512, 8, 2, 64, 16
    g = torch.Generator().manual_seed(113)
    w = {n: (torch.randn(s, generator=g) * s[0] ** -0.5).cuda() for n, s in
         (("q", (N, Hq * D)), ("k", (N, Hkv * D)), ("v", (N, Hkv * D)), ("o", (Hq * D, N)))}
    gain = (1 + 0.1 * torch.randn(N, generator=g)).cuda()
    plan = idx.Rotary.make(D)
    k, v = (idx.Cache.empty(16 * 8, Hkv, D, idx.IDX_K_BF16) for _ in range(2))
    pages = gpu([[5, 2, 7], [0, 3, 6]])
    held, x_all = [0, 0], [[], []]
    freq = plan.freq.cpu().numpy()

    def turn(x, pos):                            # [n, H, D] fp64
        a = np.asarray(pos)[:, None, None] * freq
        lo, hi = x[..., :D // 2], x[..., D // 2:]
        return np.concatenate([lo * np.cos(a) - hi * np.sin(a), hi * np.cos(a) + lo * np.sin(a)], -1)

    for new in ([30, 9], [1, 1], [1, 1]):
        T = sum(new)
        x = torch.randn((T, N), generator=g).to(BF16).cuda()
        residual = torch.randn((T, N), generator=g).to(BF16).cuda()
        total = torch.empty_like(residual)
        to = idx.Cache.empty(T, N // 128, 128)
        y = idx.idx_rms_norm(x, gain, residual=residual, total=total, to=to)
        h = x.double() + residual.double()
        want = (h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gain.double())
        assert ((y.double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 1e-30).all()
        back = idx.idx_cache_read(to, dtype=torch.float32).view(T, N).double()
        amax = want.view(T, -1, 128).abs().amax(-1, keepdim=True).expand(-1, -1, 128).reshape(T, N)
        assert ((back - want).abs() <= 2.0 ** -4 * 1.01 * want.abs() + 2.0 ** -10 / 448 * 1.01 * amax).all()
        pos = np.concatenate([np.arange(held[b], held[b] + n) for b, n in enumerate(new)])
        slot = np.concatenate([pages[b].cpu().numpy()[np.arange(held[b], held[b] + n) // page] * page
                               + np.arange(held[b], held[b] + n) % page for b, n in enumerate(new)])
        proj = {n: (y.float() @ w[n]).to(BF16).view(T, -1, D) for n in "qkv"}
        idx.idx_cache_write([idx.Write(proj["k"], k, slot=gpu(slot), rotary=plan, pos=gpu(pos)),
                             idx.Write(proj["v"], v, slot=gpu(slot))])
        q = idx.idx_rope(proj["q"], gpu(pos), plan)
        held = [a + n for a, n in zip(held, new)]
        cu = np.cumsum([0] + new)
        for window, first in ((0, 0), (12, 2)):
            out, lse = idx.idx_paged_attn(q, k, v, pages, gpu(cu), gpu(held), D ** -0.5, page=page, window=window, first=first)
            compare(out, lse, q.cpu(), k, v, pages.cpu().numpy(), page, cu, held, D ** -0.5, window, first)
        for b in range(2):
            x_all[b].append(proj["k"][cu[b]:cu[b + 1]].double().cpu().numpy())
        x2 = (out.reshape(T, Hq * D).float() @ w["o"]).to(BF16)
        y2 = idx.idx_rms_norm(x2, gain, residual=total)        # in place: the stream of the layers
        assert torch.isfinite(y2).all()
    # what the cache holds is each key turned to its place
    for b in range(2):
        keys = np.concatenate(x_all[b])
        at = pages[b].cpu().numpy()[np.arange(held[b]) // page] * page + np.arange(held[b]) % page
        want = turn(keys, np.arange(held[b]))
        assert (np.abs(k.data.cpu().double().numpy()[at] - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + 2.0 ** -20).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [24, 1500])
def test_bounds_that_go_back_stay_inside_the_workspace(fp8, T):
    """cu_q that is not ascending counts its rows several times over: results mean nothing, but bytes behind the workspace,
    and rows of no request, are left alone."""
    B, Hq, Hkv, page = 40, 24, 3, 16
    k, v = caches(120, 64 * page, Hkv, 64, BF16, fp8)
    q = queries(121, T, Hq, 64, BF16).cuda()
    pages = torch.arange(64, dtype=torch.int32, device="cuda").repeat(B, 1)
    cu = gpu([(T - 4 if b % 2 else 0) for b in range(B + 1)])
    lens = gpu([64 * page] * B)
    need = ctypes.c_size_t()
    out, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device="cuda")
    a = idx.idx_paged(idx._rows(q, "q"), idx._rows(out, "out"), k._struct, v._struct, pages.data_ptr(), 64, 64, page,
                      cu.data_ptr(), lens.data_ptr(), B, 0, 0, 0.125, lse.data_ptr())
    lib = idx.load_library()
    assert lib.idx_paged_attn_workspace(a, need) == 0 and need.value > 0
    ws = torch.full((need.value + (64 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    assert lib.idx_paged_attn(a, ws.data_ptr(), need.value, None) == 0
    torch.cuda.synchronize()
    assert (ws[need.value:] == 0xA5).all()
    assert (out[T - 4:] == 7.0).all() and (lse[T - 4:] == 7.0).all()
