"""Rotary positions, quantised cache writes and cache reads against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import mqa_logits_top_amd as idx
from around_ref import (HALF_STEP, SMALLEST, quantise_e4m3, quantise_mxfp4, read_e4m3, read_mxfp4, rotate,
                        rotate_bound)

pytestmark = pytest.mark.gpu

FP8, FP4, BF16, F16, F32 = (idx.IDX_K_FP8_E4M3, idx.IDX_K_MXFP4, idx.IDX_K_BF16, idx.IDX_K_F16, idx.IDX_K_F32)
BITS16 = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}


def _x(seed, *shape, dtype=torch.bfloat16, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(dtype)


def _pos(seed, T, lo=-1000, hi=500000):
    return torch.randint(lo, hi, (T,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)


def _rope_ok(got, x, pos, plan, inverse=False):
    want, mag = rotate(x.double().numpy(), pos.numpy(), plan.freq.cpu().numpy(), plan.rot0,
                       plan.layout == idx.IDX_ROPE_HALF, plan.mscale, inverse)
    err = np.abs(got.cpu().double().numpy() - want)
    lim = rotate_bound(want, mag, x.dtype)
    assert (err <= lim).all(), f"{(err > lim).sum()} off, worst {np.max(err / lim):.2f} of the bound"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", [idx.IDX_ROPE_HALF, idx.IDX_ROPE_INTERLEAVED])
@pytest.mark.parametrize("T,H,D,rot,rot0", [(1, 1, 8, 8, 0), (1, 32, 128, 64, 0), (5, 3, 128, 64, 64),
                                            (33, 9, 64, 24, 40), (2, 65, 256, 256, 0), (7, 5, 80, 40, 8),
                                            (3, 2, 512, 64, 448), (300, 1, 96, 96, 0)])
def test_rope(dtype, layout, T, H, D, rot, rot0):
    plan = idx.Rotary.make(rot, rot0=rot0, layout=layout)
    x, pos = _x(T + D, T, H, D, dtype=dtype), _pos(T, T)
    got = idx.idx_rope(x.cuda(), pos.cuda(), plan)
    _rope_ok(got, x, pos, plan)
    back = idx.idx_rope(x.cuda(), pos.cuda(), plan, inverse=True)
    _rope_ok(back, x, pos, plan, inverse=True)


@pytest.mark.parametrize("scaling", [dict(), dict(scaling=idx.IDX_ROPE_LINEAR, factor=8.0),
                                     dict(scaling=idx.IDX_ROPE_BASE, factor=8.0),
                                     dict(scaling=idx.IDX_ROPE_PARTS, factor=16.0, original=32768.0)])
def test_rope_far_positions_and_scaling(scaling):
    """Positions up to the int32 range: the angle's fraction of a turn survives."""
    plan = idx.Rotary.make(64, **scaling)
    pos = torch.tensor([0, 1, -1, 65535, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    x = _x(3, len(pos), 4, 128, dtype=torch.float32)
    _rope_ok(idx.idx_rope(x.cuda(), pos.cuda(), plan), x, pos, plan)


@pytest.mark.parametrize("layout", [idx.IDX_ROPE_HALF, idx.IDX_ROPE_INTERLEAVED])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_in_place_and_strided(layout, dtype):
    """In place, in a slice of a wider projection, and to an output laid out head by head: the same bits as
    rows of their own, the neighbours untouched."""
    T, H, D = 37, 6, 128
    plan = idx.Rotary.make(64, rot0=32, layout=layout)
    wide, pos = _x(4, T, 2 * H, D, dtype=dtype).cuda(), _pos(5, T).cuda()
    want = idx.idx_rope(wide[:, H:].contiguous(), pos, plan)
    heads = torch.empty((H, T, D), dtype=dtype, device="cuda")
    idx.idx_rope(wide[:, H:], pos, plan, out=heads.transpose(0, 1))
    assert torch.equal(heads.transpose(0, 1), want)
    before = wide[:, :H].clone()
    assert idx.idx_rope(wide[:, H:], pos, plan, out=wide[:, H:]).data_ptr() == wide[:, H:].data_ptr()
    assert torch.equal(wide[:, H:], want) and torch.equal(wide[:, :H], before)
    one = _x(6, T, 1, D, dtype=dtype).cuda()
    assert torch.equal(idx.idx_rope(one.expand(T, H, D), pos, plan), idx.idx_rope(one, pos, plan).expand(T, H, D))


def test_rope_gradient_is_its_inverse():
    """The gradient of <g, rope(x)> in x is the inverse rotation of g: against the formula's transpose and
    central differences of the rotation in fp32 (linear, so a difference of step 1 is exact but for the
    roundings of the two values it subtracts)."""
    plan = idx.Rotary.make(32)
    T, H, D = 3, 2, 32
    x, g = _x(7, T, H, D, dtype=torch.float32), _x(8, T, H, D, dtype=torch.float32)
    pos = torch.tensor([3, -70, 90001], dtype=torch.int32)
    grad = idx.idx_rope(g.cuda(), pos.cuda(), plan, inverse=True).cpu().double()
    _rope_ok(grad, g, pos, plan, inverse=True)
    for t, h, d in [(0, 0, 0), (1, 1, 17), (2, 0, 31), (2, 1, 15)]:
        e = torch.zeros_like(x)
        e[t, h, d] = 1.0
        up = idx.idx_rope((x + e).cuda(), pos.cuda(), plan).cpu().double()
        down = idx.idx_rope((x - e).cuda(), pos.cuda(), plan).cpu().double()
        slope = (g.double() * (up - down)).sum() / 2
        # each rotated value is off by at most 2^-23 of its magnitudes (|x| + 1 in each of two terms)
        lim = 2.0 ** -21 * (g.double().abs() * (x.double().abs().max() + 1)).sum()
        assert abs(slope - grad[t, h, d]) <= lim




@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt,D", [(FP8, 8), (FP8, 16), (FP8, 24), (FP8, 64), (FP8, 72), (FP8, 128), (FP8, 512), (FP4, 32), (FP4, 96),
                                   (FP4, 128), (FP4, 512)])
@pytest.mark.parametrize("T,H", [(1, 1), (17, 5)])
def test_quantised_codes(dtype, fmt, D, T, H):
    """Codes and scales are those of the definition, bit for bit, over a wide range of magnitudes, zero rows
    and blocks among them; the values read back are their products, rounded once."""
    x = _x(T * D + H, T, H, D, dtype=torch.float32)
    x *= torch.exp2(torch.randint(-12, 13, (T, H, 1), generator=torch.Generator().manual_seed(D)).float())
    x[0, 0] = 0.0
    if T > 1:
        x[3, 2, : D // 2] = 0.0
        x[4, 1, -1] = -x[4, 1].abs().max() * 0.5
    x = x.to(dtype)
    c = idx.Cache.empty(T, H, D, fmt)
    idx.idx_cache_write([idx.Write(x.cuda(), c)])
    xf = x.float().numpy()
    codes, scale = quantise_e4m3(xf) if fmt == FP8 else quantise_mxfp4(xf)
    value = (read_e4m3 if fmt == FP8 else read_mxfp4)(codes, scale)
    got = c.data.cpu().numpy()
    # a zero's sign is free
    same = got == codes if fmt == FP8 else np.ones_like(got, bool)
    assert (same | ((got | codes) == 0x80)).all()
    assert np.array_equal(c.scale.cpu().numpy(), scale)
    for out in (torch.bfloat16, torch.float16, torch.float32):
        back = idx.idx_cache_read(c, dtype=out).cpu().double().numpy()
        with np.errstate(over="ignore"):
            want = torch.from_numpy(value.astype(np.float32)).to(out).double().numpy()
        assert np.array_equal(back, want)


@pytest.mark.parametrize("layout", [idx.IDX_ROPE_HALF, idx.IDX_ROPE_INTERLEAVED])
@pytest.mark.parametrize("fmt", [FP8, FP4, BF16, F16, F32])
@pytest.mark.parametrize("D,rot,rot0", [(128, 64, 0), (128, 64, 64), (128, 128, 0), (96, 40, 8), (64, 8, 56)])
def test_rotated_write(layout, fmt, D, rot, rot0):
    """Rotation and storage in one pass: each value within half a step of the rotated one."""
    T, H = 21, 3
    plan = idx.Rotary.make(rot, rot0=rot0, layout=layout)
    x, pos = _x(11, T, H, D), _pos(12, T)
    c = idx.Cache.empty(T, H, D, fmt)
    idx.idx_cache_write([idx.Write(x.cuda(), c, rotary=plan, pos=pos.cuda())])
    want, mag = rotate(x.double().numpy(), pos.numpy(), plan.freq.cpu().numpy(), rot0, layout == idx.IDX_ROPE_HALF)
    got = idx.idx_cache_read(c, dtype=torch.float32).cpu().double().numpy()
    slack = 2.0 ** -22 * (np.abs(want) + mag)          # the fp32 rotation, and the scale's roundings
    if fmt == FP8:
        amax = np.abs(want).max(-1, keepdims=True)
        # half a step: 2^-4 of the value, or half of the smallest code (2^-10) times the scale
        lim = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * amax / 448) * (1 + 2.0 ** -20) + slack
    elif fmt == FP4:
        b = want.reshape(T, H, -1, 32)
        unit = 2.0 ** (np.floor(np.log2(np.abs(b).max(-1, keepdims=True) * (1 + 2.0 ** -22))) - 2)
        # half a step of E2M1 is 1/4 below 2, 1/2 below 4, 1 above; past 6 the codes saturate (values below 8)
        y = np.abs(b) / unit
        lim = (np.where(y <= 2, 0.25, np.where(y <= 4, 0.5, np.where(y <= 6, 1.0, y - 6))) * unit).reshape(want.shape)
        lim = lim * (1 + 2.0 ** -20) + slack
    else:
        lim = rotate_bound(want, mag, BITS16[fmt])
    err = np.abs(got - want)
    assert (err <= lim).all(), f"{(err > lim).sum()} off, worst {np.max(err / lim):.3f} of the bound"


@pytest.mark.parametrize("fmt", [FP8, FP4, BF16])
def test_slots_and_untouched_rows(fmt):
    """Rows go to their slots; -1 and slots past the cache are dropped; every other slot, and the bytes between
    slots of a wider buffer, stay as they were.  Reads take any slot list, zeros where there is none."""
    T, H, D, rows = 50, 2, 64, 300
    wide = torch.randint(0, 100, (rows, 3 * H, D // 2 if fmt == FP4 else D),
                         generator=torch.Generator().manual_seed(1)).cuda()
    wide = wide.to(torch.uint8) if fmt != BF16 else wide.to(torch.bfloat16)
    scales = None
    if fmt == FP8:
        scales = torch.rand((rows, 2 * H)).cuda()
    elif fmt == FP4:
        scales = torch.randint(100, 140, (rows, 2 * H, D // 32)).to(torch.uint8).cuda()
    c = idx.Cache(wide[:, H:2 * H], None if scales is None else scales[:, H:], D=D, fmt=fmt)
    before, before_s = wide.clone(), None if scales is None else scales.clone()
    x = _x(2, T, H, D)
    slot = torch.randperm(rows, generator=torch.Generator().manual_seed(3))[:T].to(torch.int32)
    slot[5], slot[9], slot[49] = -1, rows, 2 ** 31 - 1
    idx.idx_cache_write([idx.Write(x.cuda(), c, slot=slot.cuda())])
    own = idx.Cache.empty(T, H, D, fmt)
    idx.idx_cache_write([idx.Write(x.cuda(), own)])
    kept = [i for i in range(T) if 0 <= slot[i] < rows]
    at = slot[kept].long().cuda()
    before[at, H:2 * H] = own.data[kept]
    assert torch.equal(wide, before)
    if scales is not None:
        before_s[at, H:] = own.scale[kept]
        assert torch.equal(scales, before_s)
    got = idx.idx_cache_read(c, slot.cuda(), dtype=torch.float32)
    want = idx.idx_cache_read(own, dtype=torch.float32)
    drop = [i for i in range(T) if i not in kept]
    want[drop] = 0.0
    assert torch.equal(got, want)
    twice = torch.tensor([slot[0], slot[0], -7, slot[1]], dtype=torch.int32, device="cuda")
    assert torch.equal(idx.idx_cache_read(c, twice, dtype=torch.float32), want[[0, 0, drop[0], 1]])


def test_not_finite_stays_visible():
    """A NaN or an infinity makes its E4M3 row, and its MXFP4 block, NaN; other rows and blocks keep theirs."""
    x = _x(9, 4, 2, 64, dtype=torch.float32)
    clean = x.clone()
    x[1, 0, 40], x[2, 1, 3] = float("inf"), float("nan")
    for fmt in (FP8, FP4):
        a, b = idx.Cache.empty(4, 2, 64, fmt), idx.Cache.empty(4, 2, 64, fmt)
        idx.idx_cache_write([idx.Write(x.cuda(), a), idx.Write(clean.cuda(), b)])
        got, want = (idx.idx_cache_read(c, dtype=torch.float32).cpu() for c in (a, b))
        bad = torch.zeros(4, 2, 64, dtype=torch.bool)
        if fmt == FP8:
            bad[1, 0] = bad[2, 1] = True
        else:
            bad[1, 0, 32:] = bad[2, 1, :32] = True
        assert got[bad].isnan().all() and torch.equal(got[~bad], want[~bad])


def test_every_mxfp4_code():
    """Reading back every code under every E8M0 scale: 2^-127 (a subnormal) and NaN among them."""
    e8 = torch.arange(256, dtype=torch.uint8).view(256, 1, 1)
    data = (torch.arange(16) | (torch.arange(16).flip(0) << 4)).to(torch.uint8).expand(256, 1, 16).contiguous()
    c = idx.Cache(data.cuda(), e8.cuda(), D=32, fmt=FP4)
    got = idx.idx_cache_read(c, dtype=torch.float32).cpu().double().numpy()
    with np.errstate(over="ignore"):
        want = read_mxfp4(data.numpy(), e8.numpy()).astype(np.float32).astype(np.float64)
    assert np.array_equal(got, want, equal_nan=True)


def test_smallest_values():
    """Rows and blocks below 2^-100 become zeros; the largest fp32 values survive."""
    x = torch.zeros((3, 1, 64))
    x[0, 0, :] = 2.0 ** -101
    x[1, 0, 3] = 2.0 ** -100
    x[2, 0, 5], x[2, 0, 40] = 3.0e38, -1.0e38
    for fmt in (FP8, FP4):
        c = idx.Cache.empty(3, 1, 64, fmt)
        idx.idx_cache_write([idx.Write(x.cuda(), c)])
        got = idx.idx_cache_read(c, dtype=torch.float32).cpu()
        assert (got[0] == 0).all() and got[1, 0, 3] > 0 and (got[1, 0, :3] == 0).all()
        assert abs(got[2, 0, 5] / 3.0e38 - 1) <= (2.0 ** -4 if fmt == FP8 else 0.25) and got[2, 0, 40] < 0


def test_several_arrays_in_a_call():
    """A step's four arrays in one launch: what each gives on its own."""
    plan = idx.Rotary.make(64)
    T, rows = 11, 64
    pos = _pos(1, T).cuda()
    slot = torch.randperm(rows)[:T].to(torch.int32).cuda()
    arrays = [(_x(1, T, 64, 128).cuda(), FP8, T, None, plan), (_x(2, T, 1, 128).cuda(), FP4, rows, slot, plan),
              (_x(3, T, 8, 64, dtype=torch.float16).cuda(), FP8, rows, slot, None),
              (_x(4, T, 8, 64, dtype=torch.float16).cuda(), F16, rows, slot, plan),
              (_x(5, 0, 8, 64).cuda(), FP8, rows, None, None)]
    made = []
    for together in (True, False):
        caches = [idx.Cache.empty(r, x.shape[1], x.shape[2], f) for x, f, r, _, _ in arrays]
        w = [idx.Write(x, c, slot=s, rotary=p, pos=pos if p else None)
             for (x, _, _, s, p), c in zip(arrays, caches)]
        if together:
            idx.idx_cache_write(w)
        else:
            for one in w:
                idx.idx_cache_write([one])
        made.append(caches)
    for a, b in zip(*made):
        assert torch.equal(a.data, b.data)
        assert a.scale is None or torch.equal(a.scale, b.scale)


def test_long_cache_offsets():
    """Slots whose bytes lie past 2^32."""
    rows, H, D = 5_000_000, 8, 128            # 5.1 GB of codes
    c = idx.Cache(torch.empty((rows, H, D), dtype=torch.uint8, device="cuda"),
                  torch.empty((rows, H), dtype=torch.float32, device="cuda"), fmt=FP8)
    x = _x(1, 3, H, D)
    slot = torch.tensor([rows - 1, 4_194_303, 4_194_304 + 9], dtype=torch.int32)
    idx.idx_cache_write([idx.Write(x.cuda(), c, slot=slot.cuda())])
    got = idx.idx_cache_read(c, slot.cuda(), dtype=torch.float32).cpu().double().numpy()
    assert np.array_equal(got, read_e4m3(*quantise_e4m3(x.float().numpy())).astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("fmt", [FP8, FP4])
def test_indexer_inputs(fmt):
    """The caches are the indexer's own inputs: codes and scales of q and keys written here give the top-K of
    the same arrays made on the host."""
    import oracle
    import synth
    from checks import topk_ok
    T, H, L, K = 20, 32, 700, 64
    xq, xk = _x(1, T, H, 128, dtype=torch.float32), _x(2, L, 1, 128, dtype=torch.float32)
    q, k = idx.Cache.empty(T, H, 128, FP8), idx.Cache.empty(L, 1, 128, fmt)
    idx.idx_cache_write([idx.Write(xq.cuda(), q), idx.Write(xk.cuda(), k)])
    w = torch.rand((T, H), generator=torch.Generator().manual_seed(4))
    ke = torch.arange(L - T + 1, L + 1, dtype=torch.int32)
    d = idx.Inputs(q=q.data, q_scale=q.scale, k=k.data.view(L, -1),
                   k_scale=k.scale.view(L) if fmt == FP8 else k.scale.view(L, -1), w=w.cuda(),
                   ks=torch.zeros(T, dtype=torch.int32, device="cuda"), ke=ke.cuda(), k_fmt=fmt)
    gi, gv = idx.idx_logits_topk_fused(d, K, block_k=512)
    p = synth.make_problem(T, L, H, k_fmt=fmt, seed=1)
    qc, qs = quantise_e4m3(xq.numpy())
    kc, kscale = (quantise_e4m3 if fmt == FP8 else quantise_mxfp4)(xk.numpy())
    p.q, p.q_scale, p.k, p.w = qc, qs, kc.reshape(L, -1), w.numpy()
    p.k_scale = kscale.reshape(L) if fmt == FP8 else kscale.reshape(L, -1)
    dq = oracle.Dequantised(p)
    topk_ok(gi.cpu().numpy(), gv.cpu().numpy(), oracle.rows_logits(dq, range(T)), dq.ks, K)


def test_debug_mode_finds_a_slot_named_twice(monkeypatch):
    """IDX_DEBUG: a slot of one array named twice is reported before anything is written; slots outside the
    cache may repeat."""
    x, c = _x(1, 5, 1, 64).cuda(), idx.Cache.empty(10, 1, 64)
    monkeypatch.setenv("IDX_DEBUG", "1")
    ok = torch.tensor([-1, 3, -1, 99, 99], dtype=torch.int32, device="cuda")
    idx.idx_cache_write([idx.Write(x, c, slot=ok)])
    before = c.data.clone()
    twice = torch.tensor([0, 3, 1, 3, 9], dtype=torch.int32, device="cuda")
    with pytest.raises(idx.IdxError) as e:
        idx.idx_cache_write([idx.Write(x, c, slot=ok), idx.Write(x, c, slot=twice)])
    assert e.value.status == 9
    assert torch.equal(c.data, before)


def test_binding_refusals():
    """What the binding refuses before the C entry points: shapes, types, devices and leftovers."""
    plan, c = idx.Rotary.make(64), idx.Cache.empty(8, 2, 128)
    x, pos = _x(1, 4, 2, 128).cuda(), torch.zeros(4, dtype=torch.int32, device="cuda")
    bad = [lambda: idx.idx_rope(x, pos.long(), plan), lambda: idx.idx_rope(x, pos[:3], plan),
           lambda: idx.idx_rope(x, pos.cpu(), plan), lambda: idx.idx_rope(x.cpu(), pos, plan),
           lambda: idx.idx_rope(x.transpose(1, 2), pos, plan), lambda: idx.idx_rope(x[0], pos, plan),
           lambda: idx.idx_cache_write([idx.Write(x, c, pos=pos)]),
           lambda: idx.idx_cache_write([idx.Write(x, c, slot=pos[:2])]),
           lambda: idx.idx_cache_write([idx.Write(x, c, rotary=plan)]),
           lambda: idx.idx_cache_read(c, pos.long()), lambda: idx.idx_cache_read(c, pos, out=x[:3]),
           lambda: idx.Cache(c.data, c.scale[:7]), lambda: idx.Cache(c.data.float(), c.scale),
           lambda: idx.Cache(c.data.transpose(0, 1), c.scale.transpose(0, 1))]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(idx.IdxError):                     # a cache of other heads
        idx.idx_cache_write([idx.Write(x[:, :1], c)])
    with pytest.raises(AttributeError):
        c.data = x


@pytest.mark.parametrize("fmt", [FP8, FP4, idx.IDX_K_BF16, idx.IDX_K_F32])
def test_nothing_to_do(fmt):
    """No rows, a cache without slots, an empty list: nothing is written, reads outside are zeros."""
    plan = idx.Rotary.make(32)
    none, pos = _x(1, 0, 3, 64).cuda(), torch.zeros(0, dtype=torch.int32, device="cuda")
    assert idx.idx_rope(none, pos, plan).shape == (0, 3, 64)
    c, empty = idx.Cache.empty(4, 3, 64, fmt), idx.Cache.empty(0, 3, 64, fmt)
    before = c.data.clone()
    idx.idx_cache_write([])
    idx.idx_cache_write([idx.Write(none, c, rotary=plan, pos=pos), idx.Write(none, empty)])
    far = torch.tensor([0, 5, -1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    idx.idx_cache_write([idx.Write(_x(2, 5, 3, 64).cuda(), empty, slot=far)])
    assert torch.equal(c.data, before)
    assert idx.idx_cache_read(c, pos).shape == (0, 3, 64) and idx.idx_cache_read(empty).shape == (0, 3, 64)
    assert not idx.idx_cache_read(empty, far).any()


def test_graph_and_streams():
    """Captured calls take what their inputs hold at each replay; calls on another stream give the same."""
    plan = idx.Rotary.make(64, layout=1)
    x, pos = _x(3, 9, 4, 128).cuda(), torch.arange(9, dtype=torch.int32, device="cuda")
    slot = torch.arange(9, dtype=torch.int32, device="cuda") * 2
    caches = [idx.Cache.empty(40, 4, 128, f) for f in (FP8, FP4, idx.IDX_K_BF16)]

    def run(stream=None):
        y = idx.idx_rope(x, pos, plan, stream=stream)
        idx.idx_cache_write([idx.Write(x, c, slot=slot, rotary=plan, pos=pos) for c in caches], stream=stream)
        return [y] + [idx.idx_cache_read(c, slot, stream=stream) for c in caches]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for turn in range(4):
        x.copy_(_x(10 + turn, 9, 4, 128))
        pos.add_(1000)
        slot.add_(1)
        want = [y.clone() for y in run()]
        for c in caches:
            c.data.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        side = torch.cuda.Stream()
        got = run(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,D", [(1, 1, 32), (17, 5, 96), (40, 3, 128), (3, 2, 512)])
def test_mxfp4_codes(dtype, T, H, D):
    """Nibble by nibble: the even value in the low one, codes to nearest even and saturating, on values half way between
    two codes and on borders of the exponent too.  A zero's sign is free."""
    g = torch.Generator().manual_seed(T * D)
    x = torch.randn((T, H, D), generator=g) * torch.exp2(torch.randint(-9, 10, (T, H, 1), generator=g).float())
    ties = torch.tensor([0.25, -0.75, 1.25, -1.75, 2.5, -3.5, 5.0, 7.0])
    x[-1, -1, :8] = ties * 4.0                 # amax 28: unit 4
    x[-1, -1, 8:32] = 0.0
    x = x.to(dtype)
    c = idx.Cache.empty(T, H, D, FP4)
    idx.idx_cache_write([idx.Write(x.cuda(), c)])
    packed, e8 = quantise_mxfp4(x.float().numpy())
    assert np.array_equal(c.scale.cpu().numpy(), e8)
    got = c.data.cpu().numpy()
    for shift in (0, 4):
        a, b = (got >> shift) & 15, (packed >> shift) & 15
        assert ((a == b) | ((a | b) == 8)).all()
