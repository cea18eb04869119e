"""The operators around the indexer, as workloads: rotary positions, quantised cache writes, reading a cache back, and
attention over selected keys.

`run` computes a case in plain torch operations, or, with `own` set, through libidx's entry points on the same inputs.
The shapes are those of the indexer's own workloads (chunks of 2048 and 16384 rows, prefixes of 65536, 102400 and 487936
keys, 32 and 64 heads of 128, top-512 and top-2048, 8-key blocks) and serving steps beside them.

Every case is a dict: `op` says which operator, the rest its sizes.  Rows belong to `R` requests of nearly equal length,
the new rows of a request being the last of its keys.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -100          # a quantised row whose largest value is below it is stored as zeros
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token of one request: its attention queries are rotated; only the call's latency counts
        {"name": "rope_token", "op": "rope", "T": 1, "H": 32, "D": 128, "rot": 64, "rot0": 0, "layout": "half",
         "scaling": "none", "first": 65535, "dtype": "bf16"},
        # the last chunk of a 487936-token prompt: q of every head, a slice of a wider projection, frequencies scaled
        # by parts for the long context, rotated part behind the unrotated one
        {"name": "rope_chunk", "op": "rope", "T": 16384, "H": 64, "D": 128, "rot": 64, "rot0": 64,
         "layout": "interleaved", "scaling": "parts", "first": 471552, "dtype": "bf16"},
        # one decode step of 24 requests: the indexer's q and key are rotated and quantised, the keys go to their slots
        {"name": "index_step", "op": "index", "T": 24, "H": 64, "D": 128, "rows": 65536, "fmt": "fp8", "rot": 64,
         "layout": "half", "first": 60000, "dtype": "bf16"},
        # a prefill chunk of 2048 rows against a 102400-key MXFP4 prefix; the chunk's keys are read back after it
        {"name": "index_chunk", "op": "index", "T": 2048, "H": 64, "D": 128, "rows": 102400, "fmt": "mxfp4", "rot": 64,
         "layout": "half", "first": 100352, "dtype": "bf16"},
        # the attention's keys and values of a ragged batch (4 x 7168 fresh rows and 2048 on a prefix), grouped heads,
        # some rows padding
        {"name": "kv_batch", "op": "kv", "T": 30720, "H": 8, "D": 128, "rows": 180720, "fmt": "fp8", "rot": 128,
         "layout": "half", "first": 0, "pad": 0.02, "dtype": "bf16"},
        # an MXFP4 prefix of indexer keys read back whole, in order
        {"name": "read_keys", "op": "read", "N": 102400, "H": 1, "D": 128, "rows": 102400, "fmt": "mxfp4",
         "order": "straight", "dtype": "bf16"},
        # one request's cached keys gathered from pages in any order, a length that fills no tile
        {"name": "read_kv", "op": "read", "N": 7167, "H": 8, "D": 128, "rows": 180720, "fmt": "fp8", "order": "paged",
         "dtype": "bf16"},
        # one token of one request on the longest prefix, every head sharing one kv head
        {"name": "attend_token", "op": "attend", "T": 1, "R": 1, "L": 487936, "Hq": 64, "Hkv": 1, "D": 128, "K": 512,
         "pool": 1, "fmt": "bf16", "slots": False, "dtype": "bf16"},
        # a decode step of 40 requests on 4000 keys each, grouped heads, quantised paged cache
        {"name": "attend_batch", "op": "attend", "T": 40, "R": 40, "L": 160000, "Hq": 32, "Hkv": 8, "D": 128, "K": 2048,
         "pool": 1, "fmt": "fp8", "slots": True, "dtype": "bf16"},
        # the 2048-row chunk on 65536 keys, top-2048, 32 heads sharing one kv head
        {"name": "attend_chunk", "op": "attend", "T": 2048, "R": 1, "L": 65536, "Hq": 32, "Hkv": 1, "D": 128, "K": 2048,
         "pool": 1, "fmt": "bf16", "slots": False, "dtype": "bf16"},
        # the 2048-row chunk on 102400 keys, top-512, 64 heads, quantised cache
        {"name": "attend_chunk_fp8", "op": "attend", "T": 2048, "R": 1, "L": 102400, "Hq": 64, "Hkv": 1, "D": 128,
         "K": 512, "pool": 1, "fmt": "fp8", "slots": False, "dtype": "bf16"},
        # a ragged batch whose rows attend inside 8-key candidate blocks, small heads, odd sizes
        {"name": "attend_blocks", "op": "attend", "T": 1023, "R": 5, "L": 20001, "Hq": 16, "Hkv": 2, "D": 64, "K": 96,
         "pool": 8, "fmt": "fp16", "slots": False, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "index", "kv", "read", "attend", "attend"])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        D = rng.choice([64, 128, 256])
        rot = 8 * rng.randint(1, D // 8)
        return {"op": op, "T": _log(rng, 1, 4096), "H": rng.randint(1, 64), "D": D, "rot": rot,
                "rot0": 8 * rng.randint(0, (D - rot) // 8), "layout": layout,
                "scaling": rng.choice(["none", "linear", "base", "parts"]), "first": _log(rng, 1, 1 << 20),
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "index":
        T = _log(rng, 1, 2048)
        return {"op": op, "T": T, "H": rng.choice([32, 64]), "D": 128, "rows": T + _log(rng, 1, 131072),
                "fmt": rng.choice(["fp8", "mxfp4"]), "rot": 16 * rng.randint(1, 8), "layout": layout,
                "first": _log(rng, 1, 1 << 20), "dtype": rng.choice(["bf16", "fp16"])}
    if op == "kv":
        T, D = _log(rng, 1, 15000), rng.choice([64, 128])
        return {"op": op, "T": T, "H": rng.randint(1, 16), "D": D, "rows": T + _log(rng, 1, 65536), "fmt": "fp8",
                "rot": 8 * rng.randint(1, D // 8), "layout": layout, "first": _log(rng, 1, 1 << 20),
                "pad": rng.choice([0.0, 0.1]), "dtype": rng.choice(["bf16", "fp16"])}
    if op == "read":
        rows = _log(rng, 64, 200000)
        return {"op": op, "N": _log(rng, 1, 50000), "H": rng.randint(1, 8), "D": rng.choice([64, 128]), "rows": rows,
                "fmt": rng.choice(["fp8", "mxfp4"]), "order": "paged", "dtype": rng.choice(["bf16", "fp16"])}
    Hkv = rng.choice([1, 1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 3, 4, 8] if Hkv > 1 else [8, 16, 32, 64])
    R = _log(rng, 1, 64)
    T = R if rng.random() < 0.5 else R * rng.randint(1, 14) + rng.randint(0, R)
    pool = rng.choice([1, 1, 8])
    K = _log(rng, 16, 2048) if pool == 1 else _log(rng, 2, 128)
    dtype = rng.choice(["bf16", "fp16"])
    return {"op": op, "T": T, "R": R, "L": R * _log(rng, 64, 16384) + rng.randint(0, 7), "Hq": Hq, "Hkv": Hkv,
            "D": rng.choice([64, 128]), "K": K, "pool": pool, "fmt": rng.choice([dtype, "fp8"]),
            "slots": rng.random() < 0.5, "dtype": dtype}


# ------------------------------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)


def _frequencies(rot, scaling):
    """Radians a position of every pair, base 10000, and the gain on the rotated values: a context of 32768 positions
    stretched 16 times."""
    base, factor, original = 10000.0, 16.0, 32768.0
    if scaling == "base":
        base *= factor ** (rot / max(rot - 2, 1))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling != "parts":
        return f, 1.0
    where = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(where(32.0)), 0), min(math.ceil(where(1.0)), rot - 1)
    ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
    return [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


def _rotary(case, scaling="none"):
    """The rotary plan a program keeps: frequencies on the device, which part of the head, the layout."""
    f, gain = _frequencies(case["rot"], scaling)
    s = {"freq": torch.tensor(f, dtype=torch.float64, device="cuda"), "gain": gain, "rot": case["rot"],
         "rot0": case.get("rot0", 0), "half": case["layout"] == "half"}
    if own:
        import mqa_logits_top_amd as idx
        s["plan"] = idx.Rotary(s["freq"], rot0=s["rot0"], layout=idx.IDX_ROPE_HALF if s["half"] else
                               idx.IDX_ROPE_INTERLEAVED, mscale=gain)
    return s


def _cache(g, rows, H, D, fmt):
    """A cache of `rows` slots with contents of its own, and one slot more that no call may name."""
    if fmt in DTYPES:
        c = {"data": _normal(g, (rows + 1, H, D), DTYPES[fmt]), "scale": None}
    else:
        x = torch.randn((rows + 1, H, D), generator=g, device="cuda")
        codes, scale = _to_fp8(x) if fmt == "fp8" else _to_mxfp4(x)
        c = {"data": codes, "scale": scale}
    c |= {"fmt": fmt, "rows": rows}
    if own:
        import mqa_logits_top_amd as idx
        c["handle"] = idx.Cache(c["data"][:rows], None if c["scale"] is None else c["scale"][:rows], D=D,
                                fmt={"fp8": idx.IDX_K_FP8_E4M3, "mxfp4": idx.IDX_K_MXFP4, "bf16": idx.IDX_K_BF16,
                                     "fp16": idx.IDX_K_F16}[fmt])
    return c


def _windows(case):
    """First and one past the last key of every row: request r of R owns keys [r L / R, (r + 1) L / R)."""
    T, R, L = case["T"], case["R"], case["L"]
    t = torch.arange(T, device="cuda", dtype=torch.int64)
    r = t * R // T
    ks, end = r * L // R, (r + 1) * L // R
    last = ((r + 1) * T + R - 1) // R - 1          # the request's last row
    return ks.to(torch.int32), torch.maximum(ks, end - (last - t)).to(torch.int32)


def _selection(g, case, ks, ke):
    """What the indexer would have selected: each row's best keys (or blocks of `pool` keys) by a score that rows of a
    request share in part; ascending ids, -1 behind them.  Keys are absolute, blocks count from ks."""
    K, pool, R = case["K"], case["pool"], case["R"]
    n = (ke - ks + pool - 1) // pool
    W = (-(-case["L"] // R) + pool - 1) // pool + 1
    r = torch.arange(case["T"], device="cuda") * R // case["T"]
    score = torch.randn((case["T"], W), generator=g, device="cuda")
    score += torch.randn((R, W), generator=g, device="cuda")[r]
    j = torch.arange(W, device="cuda")
    score.masked_fill_(j >= n[:, None], -math.inf)
    top = torch.topk(score, min(K, W), dim=1, sorted=False)
    ids = torch.where(top.values > -math.inf, top.indices, 1 << 40).sort(dim=1).values
    ids = torch.where(ids < (1 << 40), ids + (ks[:, None] if pool == 1 else 0), -1)
    return torch.nn.functional.pad(ids, (0, K - ids.shape[1]), value=-1).to(torch.int32).contiguous()


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"op": op, "case": case}
    dtype = DTYPES[case["dtype"]]
    if op == "attend":
        T, Hq, Hkv, D, L = case["T"], case["Hq"], case["Hkv"], case["D"], case["L"]
        s["q"] = _normal(g, (T, Hq, D), dtype, 2.5)       # scores spread enough for a softmax with few large terms
        s["k"], s["v"] = _cache(g, L, Hkv, D, case["fmt"]), _cache(g, L, Hkv, D, case["fmt"])
        s["ks"], s["ke"] = _windows(case)
        s["sel"] = _selection(g, case, s["ks"], s["ke"])
        s["table"] = torch.randperm(L, generator=g, device="cuda").to(torch.int32) if case["slots"] else None
        return s
    H, D, rows = case["H"], case["D"], case.get("rows", 0)
    if op == "read":
        s["cache"] = _cache(g, rows, H, D, case["fmt"])
        at = torch.arange(case["N"], device="cuda") % rows
        s["at"] = (at if case["order"] == "straight" else
                   torch.randint(-1, rows, (case["N"],), generator=g, device="cuda")).to(torch.int32)
        return s
    T = case["T"]
    s["pos"] = torch.arange(T, device="cuda", dtype=torch.int32) + case["first"]
    if op == "rope":
        s["x"] = _normal(g, (T, H + 2, D), dtype)[:, :H]  # a slice of a wider projection
        s["rotary"] = _rotary(case, case["scaling"])
        return s
    s["rotary"] = _rotary(case)
    slots = torch.randperm(rows, generator=g, device="cuda")[:T]
    pad = torch.rand(T, generator=g, device="cuda") < case.get("pad", 0.0)
    s["slot"] = torch.where(pad, -1, slots).to(torch.int32)
    if op == "index":
        s["xq"], s["xk"] = _normal(g, (T, H, D), dtype), _normal(g, (T, 1, D), dtype)
        s["q"], s["k"] = _cache(g, T, H, D, "fp8"), _cache(g, rows, 1, D, case["fmt"])
    else:
        s["xk"], s["xv"] = _normal(g, (T, H, D), dtype), _normal(g, (T, H, D), dtype)
        s["k"], s["v"] = _cache(g, rows, H, D, case["fmt"]), _cache(g, rows, H, D, case["fmt"])
    return s


# ------------------------------------------------------------------------------------------------ the plain forms
def _rotate(x, pos, r):
    """float32 [T, H, D]: pairs turned by pos * freq.  Angles, and the two products of a turn, in 64 bits: a position
    times a frequency loses its fraction in 32, and a value next to a border of the quantisers may not move."""
    angle = pos.double()[:, None, None] * r["freq"]
    c, s = (angle.cos() * r["gain"]).float().double(), (angle.sin() * r["gain"]).float().double()
    lo, hi = r["rot0"], r["rot0"] + r["rot"]
    part = x[..., lo:hi].double()
    if r["half"]:
        a, b = part[..., :r["rot"] // 2], part[..., r["rot"] // 2:]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([x[..., :lo].float(), turned.float(), x[..., hi:].float()], -1)


def _to_fp8(x):
    """E4M3 codes and one scale a row of the last dimension."""
    amax = x.abs().amax(-1)
    some = amax >= TINY
    scale = torch.where(some, amax / E4M3_MAX, 1.0)
    inverse = torch.where(some, E4M3_MAX / amax, 0.0)
    return (x * inverse[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _to_mxfp4(x):
    """E2M1 codes, two a byte, and one E8M0 scale for 32 values."""
    blocks = x.unflatten(-1, (-1, 32))
    amax = blocks.abs().amax(-1)
    exponent = torch.frexp(amax).exponent - 1 - 2
    e8 = torch.where(amax >= TINY, exponent + 127, 0).clamp(0, 254)
    a = (blocks * torch.ldexp(torch.ones_like(amax), 127 - e8)[..., None]).abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int() + 8 * (blocks < 0).int()).flatten(-2)
    code = torch.where((amax < TINY).repeat_interleave(32, -1), 0, code)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), e8.to(torch.uint8)


def _values(data, scale, fmt):
    """float32 values of cache rows."""
    if fmt == "fp8":
        return data.view(torch.float8_e4m3fn).float() * scale[..., None]
    if fmt == "mxfp4":
        code = torch.stack([data & 15, data >> 4], -1).flatten(-2).long()
        grid = torch.tensor(E2M1, device=data.device)
        x = torch.where(code >= 8, -grid[code & 7], grid[code & 7])
        return x * torch.exp2(scale.float() - 127).repeat_interleave(32, -1)
    return data.float()


def _store(cache, slot, x):
    """Rows of x to their slots; row -1 to the slot that no call may name."""
    data, scale = _to_fp8(x) if cache["fmt"] == "fp8" else _to_mxfp4(x)
    at = torch.where(slot >= 0, slot, cache["rows"]).long()
    cache["data"][at], cache["scale"][at] = data, scale


def _contents(cache, n=None):
    """A cache's first n slots, as the tensors it is held in."""
    n = cache["rows"] if n is None else n
    return [cache["data"][:n].view(torch.float8_e4m3fn), cache["scale"][:n]]


def _load(cache, at, dtype):
    rows = torch.where(at >= 0, at, cache["rows"]).long()
    scale = None if cache["scale"] is None else cache["scale"][rows]
    return torch.where((at >= 0)[:, None, None], _values(cache["data"][rows], scale, cache["fmt"]), 0.0).to(dtype)


def _keys(s):
    """Cache row of every entry of the selection, and whether it counts: [T, K pool]."""
    pool, L = s["case"]["pool"], s["case"]["L"]
    sel, ks, ke = s["sel"].long(), s["ks"].long()[:, None], s["ke"].long()[:, None]
    key = sel
    if pool > 1:
        key = (ks[..., None] + sel[..., None] * pool + torch.arange(pool, device=sel.device)).flatten(1)
        sel = sel.repeat_interleave(pool, 1)
    counts = (sel >= 0) & (key >= ks) & (key < ke)
    row = key.clamp(0, L - 1)
    return (row if s["table"] is None else s["table"].long()[row]), counts


def _attend(s):
    c = s["case"]
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    row, counts = _keys(s)
    pick = lambda x: _values(x["data"][row], None if x["scale"] is None else x["scale"][row], x["fmt"])
    q = s["q"].float().view(T, Hkv, Hq // Hkv, D)
    score = torch.matmul(q, pick(s["k"]).permute(0, 2, 3, 1).contiguous()) * D ** -0.5
    score.masked_fill_(~counts[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, pick(s["v"]).permute(0, 2, 1, 3).contiguous()) / torch.where(total > 0, total, 1.0)
    return [out.view(T, Hq, D).to(s["q"].dtype), (top + torch.log(total)).view(T, Hq)]


def _plain(s):
    op, case = s["op"], s["case"]
    if op == "attend":
        return _attend(s)
    if op == "read":
        return _load(s["cache"], s["at"], DTYPES[case["dtype"]])
    if op == "rope":
        return _rotate(s["x"], s["pos"], s["rotary"]).to(s["x"].dtype)
    _store(s["k"], s["slot"], _rotate(s["xk"], s["pos"], s["rotary"]))
    if op == "kv":
        _store(s["v"], s["slot"], s["xv"].float())
        return _contents(s["k"]) + _contents(s["v"])
    codes, scale = _to_fp8(_rotate(s["xq"], s["pos"], s["rotary"]))
    q = [codes.view(torch.float8_e4m3fn), scale]
    return q + (_contents(s["k"]) if case["fmt"] == "fp8" else [_load(s["k"], s["slot"], s["xk"].dtype)])


# ------------------------------------------------------------------------------------------------ libidx
def _libidx(s):
    import mqa_logits_top_amd as idx
    op, case = s["op"], s["case"]
    if op == "attend":
        return idx.idx_sparse_attn(s["q"], s["k"]["handle"], s["v"]["handle"], s["sel"], scale=case["D"] ** -0.5,
                                   pool=case["pool"], ks=s["ks"], ke=s["ke"], slot_of_key=s["table"])
    if op == "read":
        return idx.idx_cache_read(s["cache"]["handle"], s["at"], dtype=DTYPES[case["dtype"]])
    plan = s["rotary"]["plan"]
    if op == "rope":
        return idx.idx_rope(s["x"], s["pos"], plan)
    if op == "kv":
        idx.idx_cache_write([idx.Write(s["xk"], s["k"]["handle"], slot=s["slot"], rotary=plan, pos=s["pos"]),
                             idx.Write(s["xv"], s["v"]["handle"], slot=s["slot"])])
        return _contents(s["k"]) + _contents(s["v"])
    idx.idx_cache_write([idx.Write(s["xq"], s["q"]["handle"], rotary=plan, pos=s["pos"]),
                         idx.Write(s["xk"], s["k"]["handle"], slot=s["slot"], rotary=plan, pos=s["pos"])])
    if case["fmt"] == "fp8":
        return _contents(s["q"]) + _contents(s["k"])
    return _contents(s["q"]) + [idx.idx_cache_read(s["k"]["handle"], s["slot"], dtype=s["xk"].dtype)]


def run(state):
    return _libidx(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ what a pass needs
def _row_bytes(H, D, fmt):
    return H * {"fp8": D + 4, "mxfp4": D // 2 + D // 32, "bf16": 2 * D, "fp16": 2 * D}[fmt]


def work(case):
    op, D = case["op"], case["D"]
    if op == "attend":
        T, keys = case["T"], case["K"] * case["pool"]
        seen = min(keys, -(-case["L"] // case["R"]))       # a row sees no more than its request's keys
        touched = min(case["L"], T * seen)
        return {"bytes": 2 * touched * _row_bytes(case["Hkv"], D, case["fmt"]) + T * case["Hq"] * (4 * D + 4)
                + 4 * T * case["K"] + 8 * T, "flops": 4 * T * case["Hq"] * seen * D}
    H = case["H"]
    if op == "read":
        return {"bytes": case["N"] * (_row_bytes(H, D, case["fmt"]) + 2 * H * D + 4), "flops": case["N"] * H * D}
    T, size = case["T"], 4 if case["dtype"] == "fp32" else 2
    if op == "rope":
        return {"bytes": 2 * T * H * D * size + 4 * T, "flops": 3 * T * H * case["rot"]}
    if op == "kv":
        return {"bytes": 2 * T * (H * D * size + _row_bytes(H, D, case["fmt"])) + 8 * T,
                "flops": 2 * T * H * (3 * D + case["rot"])}
    again = _row_bytes(1, D, "mxfp4") + D * size + 4 if case["fmt"] == "mxfp4" else 0
    return {"bytes": T * ((H + 1) * D * size + _row_bytes(H, D, "fp8") + _row_bytes(1, D, case["fmt"]) + 8 + again),
            "flops": T * (H + 1) * 3 * (D + case["rot"])}


# ------------------------------------------------------------------------------------------------ from the definition
def _exact_turn(x, pos, r):
    """Complex numbers turned by e^(i pos freq)."""
    part = x.double()[..., r["rot0"]:r["rot0"] + r["rot"]]
    pairs = part.unflatten(-1, (2, -1)).movedim(-2, -1) if r["half"] else part.unflatten(-1, (-1, 2))
    unit = torch.polar(torch.full_like(r["freq"], r["gain"]).expand(len(pos), -1), pos.double()[:, None] * r["freq"])
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit[:, None])
    out = x.double().clone()
    out[..., r["rot0"]:r["rot0"] + r["rot"]] = z.movedim(-1, -2).flatten(-2) if r["half"] else z.flatten(-2)
    return out


def _nearest(x, grid):
    """The nearest value of an ascending grid, ties to the even place (as E4M3's and E2M1's codes are ordered)."""
    a = x.abs()
    up = torch.searchsorted(grid, a.contiguous()).clamp(1, len(grid) - 1)
    below, above = grid[up - 1], grid[up]
    lower = (a - below < above - a) | ((a - below == above - a) & ((up - 1) % 2 == 0))
    return torch.copysign(torch.where(lower, below, above), x)


def _exact_fp8(x):
    grid = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    scale = x.abs().amax(-1) / E4M3_MAX
    return _nearest(x / scale[..., None], grid), scale


def _exact_stored(cache, slot, x):
    codes, scale = _exact_fp8(x)
    data = cache["data"][:cache["rows"]].view(torch.float8_e4m3fn).double()
    scales, real = cache["scale"][:cache["rows"]].double(), slot >= 0
    data[slot[real].long()], scales[slot[real].long()] = codes[real], scale[real]
    return [data, scales]


def _exact_rows(cache, rows):
    """Values of cache rows in 64 bits."""
    data = cache["data"][rows]
    if cache["fmt"] == "fp8":
        return data.view(torch.float8_e4m3fn).double() * cache["scale"][rows].double()[..., None]
    if cache["fmt"] == "mxfp4":
        grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
        nibbles = torch.empty(data.shape[:-1] + (2 * data.shape[-1],), dtype=torch.int64, device="cuda")
        nibbles[..., 0::2], nibbles[..., 1::2] = data % 16, data // 16
        x = grid[nibbles].unflatten(-1, (-1, 32))
        return (x * 2.0 ** (cache["scale"][rows].double() - 127)[..., None]).flatten(-2)
    return data.double()


def _exact_attend(s):
    c = s["case"]
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    row, counts = _keys(s)
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 28) // (row.shape[1] * Hkv * D))
    for a in range(0, T, step):
        b = min(a + step, T)
        k, v = (_exact_rows(x, row[a:b]).transpose(1, 2).repeat_interleave(Hq // Hkv, 1) if Hkv > 1 else
                _exact_rows(x, row[a:b]).transpose(1, 2) for x in (s["k"], s["v"]))
        q = s["q"][a:b].double()
        score = ((q[:, :, None] * k).sum(-1) if Hkv > 1 else q @ k[:, 0].mT.contiguous()) / math.sqrt(D)
        score = torch.where(counts[a:b, None], score, -math.inf)
        lse[a:b] = torch.logsumexp(score, -1)
        p = torch.where(counts[a:b, None], torch.softmax(score, -1), 0.0)
        out[a:b] = (p[..., None] * v).sum(2) if Hkv > 1 else p @ v[:, 0].contiguous()
    return [out, lse]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attend":
        return _exact_attend(s)
    if op == "read":
        x = _exact_rows(s["cache"], s["at"].long().clamp(min=0))
        x[s["at"] < 0] = 0.0
        return x
    if op == "rope":
        return _exact_turn(s["x"], s["pos"], s["rotary"])
    k = _exact_turn(s["xk"], s["pos"], s["rotary"])
    if op == "kv":
        return _exact_stored(s["k"], s["slot"], k) + _exact_stored(s["v"], s["slot"], s["xv"].double())
    q = list(_exact_fp8(_exact_turn(s["xq"], s["pos"], s["rotary"])))
    if case["fmt"] == "fp8":
        return q + _exact_stored(s["k"], s["slot"], k)
    blocks = k.unflatten(-1, (-1, 32))
    unit = 2.0 ** (torch.floor(torch.log2(blocks.abs().amax(-1, keepdim=True))) - 2)
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    return q + [(_nearest(blocks / unit, grid) * unit).flatten(-2)]
