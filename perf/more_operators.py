"""Attention over every key of a paged cache, attention with a sliding window, and the norm in front of the projections, as
workloads.

`run` computes a case in plain torch operations, or, with `own` set, through libidx's entry points on the same inputs.
The shapes are those of the indexer's own workloads (chunks of 2048 rows, a prefix of 65536 keys, batches of 4 fresh
requests, 32 and 64 heads of 128) and serving steps beside them.

Every case is a dict: `op` says which operator, the rest its sizes.  In the attention cases T new rows belong to B
requests of nearly equal shares, the new rows of a request being the last of its keys; request b has about
L (1 - spread * frac(0.618 b)) keys, or its new rows alone where L is 0.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -100          # a quantised row whose largest value is below it is stored as zeros
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------ the cases
def _attention(name, op, T, B, L, spread, Hq, Hkv, D, page, fmt, dtype, window=0, first=0, spare=0):
    """spare: pages of a request's row in the table behind its longest length, as a table of fixed width has."""
    c = {"op": op, "T": T, "B": B, "L": L, "spread": spread, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "fmt": fmt,
         "dtype": dtype, "window": window, "first": first, "spare": spare}
    return {"name": name, **c} if name else c


def _norm(name, T, H, D, heads, dtype, residual, out, quant, wide=0):
    """heads: each head's D values have a norm of their own, else all H D of a row; residual: its type or ""; quant:
    values that share an E4M3 scale (0: no codes); wide: heads more that the rows' projection holds."""
    c = {"op": "norm", "T": T, "H": H, "D": D, "heads": heads, "dtype": dtype, "residual": residual, "out": out,
         "quant": quant, "wide": wide}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one new token of one request: only the call's latency counts
        _attention("chunk_token", "chunk", 1, 1, 4000, 0.0, 32, 8, 128, 64, "bf16", "bf16", spare=32),
        # a decode step of 32 requests of very different lengths, quantised cache, small pages, a wide table
        _attention("chunk_step", "chunk", 32, 32, 16384, 0.9, 32, 8, 128, 16, "fp8", "bf16", spare=512),
        # the 2048-row chunk of one request on 65536 keys
        _attention("chunk_prefix", "chunk", 2048, 1, 65536, 0.0, 32, 8, 128, 64, "bf16", "bf16"),
        # a ragged batch on prefixes of odd lengths, small heads, seven groups of eight
        _attention("chunk_ragged", "chunk", 3333, 7, 9001, 0.9, 16, 2, 64, 128, "fp16", "fp16"),
        # three requests' chunks of 333 and 334 rows on quantised prefixes, 64 heads
        _attention("chunk_fp8", "chunk", 1000, 3, 30001, 0.5, 64, 8, 128, 16, "fp8", "bf16", spare=3),
        # a decode step of 64 requests in a layer that sees the last 4096 keys and the first 4
        _attention("window_step", "window", 64, 64, 30000, 0.5, 32, 8, 128, 64, "bf16", "bf16", window=4096, first=4),
        # four fresh prompts of 2048 tokens in a layer with a window of 1024
        _attention("window_prompts", "window", 8192, 4, 0, 0.0, 32, 8, 128, 64, "bf16", "bf16", window=1024, first=4),
        # 500-odd rows on a quantised prefix, a window that fills no tile, 65 first keys, one head for all
        _attention("window_odd", "window", 511, 2, 12345, 0.3, 32, 1, 64, 1, "fp8", "fp16", window=777, first=65),
        # one token's hidden row: residual added, E4M3 with a scale for each 128 values, for the next projection
        _norm("norm_token", 1, 64, 128, False, "bf16", "bf16", False, 128),
        # a chunk of 16384 hidden rows, the same
        _norm("norm_chunk", 16384, 64, 128, False, "bf16", "bf16", False, 128),
        # a chunk's queries, each head normed before its rotation; a slice of a wider projection
        _norm("norm_heads", 2048, 64, 128, True, "bf16", "", True, 0, wide=2),
        # odd sizes, a residual kept in 32 bits, values and E4M3 codes with one scale a row
        _norm("norm_odd", 1023, 1, 5000, False, "fp16", "fp32", True, 5000),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "window", "norm"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "norm":
        heads = rng.random() < 0.4
        if heads:
            H, D = rng.randint(1, 64), rng.choice([64, 96, 128, 256])
            quant = rng.choice([0, D])
        else:
            quant = rng.choice([0, 64, 128, -1])
            D = max(quant, 8)
            H = _log(rng, 1, 8192 // D)
            if quant == -1:
                H, D, quant = 1, H * D, H * D
        return _norm("", _log(rng, 1, 8192), H, D, heads, rng.choice([dtype, dtype, "fp32"]),
                     rng.choice(["", dtype, "fp32"]), quant == 0 or rng.random() < 0.5, quant, rng.randint(0, 2) if heads else 0)
    Hkv = rng.choice([1, 2, 4, 8])
    Hq, D = Hkv * rng.choice([1, 3, 4, 7, 8]) if Hkv > 1 else rng.choice([8, 16, 32, 64]), rng.choice([64, 128])
    B = _log(rng, 1, 64)
    n = 1 if rng.random() < 0.4 else _log(rng, 2, 1200)
    T = B * n + (rng.randint(0, B - 1) if n > 1 else 0)
    fresh = n > 1 and rng.random() < 0.3
    # the padded scores of the plain form, and its padded keys, stay within 4 GB each
    most = min((1 << 30) // (B * Hq * (n + 1)), (1 << 30) // (B * Hkv * D), 65536)
    if most < n + 1 or (fresh and B * n * n * Hq > 1 << 30):
        T, n, fresh = B, 1, False
        most = min((1 << 30) // (B * Hq * 2), (1 << 30) // (B * Hkv * D), 65536)
    L = 0 if fresh else _log(rng, n + 1, most)
    window = _log(rng, 16, 4096) if op == "window" else 0
    return _attention("", op, T, B, L, rng.choice([0.0, 0.5, 0.9]), Hq, Hkv, D, rng.choice([1, 16, 64, 256]),
                      rng.choice([dtype, "fp8"]), dtype, window, rng.choice([0, 1, 4, 100]) if window else 0,
                      rng.choice([0, 0, 40]))


def _requests(case):
    """New rows and keys of every request."""
    T, B, L = case["T"], case["B"], case["L"]
    n = [(b + 1) * T // B - b * T // B for b in range(B)]
    keys = [max(x, round(L * (1.0 - case["spread"] * ((0.6180339887 * b) % 1.0)))) for b, x in enumerate(n)]
    return n, keys


# ------------------------------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)


def _cache(g, rows, H, D, fmt):
    """A cache with contents of its own in every slot."""
    if fmt == "fp8":
        x = torch.randn((rows, H, D), generator=g, device="cuda")
        codes, scale = _to_fp8(x)
        c = {"data": codes.view(torch.uint8), "scale": scale}
    else:
        c = {"data": _normal(g, (rows, H, D), DTYPES[fmt]), "scale": None}
    if own:
        import mqa_logits_top_amd as idx
        c["handle"] = idx.Cache(c["data"], c["scale"], D=D, fmt={"fp8": idx.IDX_K_FP8_E4M3, "bf16": idx.IDX_K_BF16,
                                                                   "fp16": idx.IDX_K_F16}[fmt])
    return c


def _prepare_norm(case, seed):
    g, dtype = _generator(seed), DTYPES[case["dtype"]]
    T, H, D = case["T"], case["H"], case["D"]
    # a row's size is its own, and few channels carry large values, as hidden states have them
    gain = torch.exp(torch.randn((T, 1, 1), generator=g, device="cuda"))
    gain = gain * torch.where(torch.rand((1, H, D), generator=g, device="cuda") < 0.01, 20.0, 1.0)
    x = (torch.randn((T, H, D), generator=g, device="cuda") * gain).to(dtype)
    if case["wide"]:
        wider = torch.zeros((T, H + case["wide"], D), dtype=dtype, device="cuda")
        wider[:, :H] = x
        x = wider[:, :H]
    width = D if case["heads"] else H * D
    s = {"case": case, "x": x if case["heads"] else x.flatten(1), "residual": None, "total": None, "to": None,
         "weight": (1.0 + 0.2 * torch.randn(width, generator=g, device="cuda")).to(dtype)}
    if case["residual"]:
        s["residual"] = _normal(g, s["x"].shape, DTYPES[case["residual"]], 2.0)
        s["total"] = torch.empty_like(s["residual"])
    if case["quant"]:
        q = case["quant"]
        s["codes"] = torch.zeros((T, H * D // q, q), dtype=torch.uint8, device="cuda")
        s["scale"] = torch.ones((T, H * D // q), dtype=torch.float32, device="cuda")
        if own:
            import mqa_logits_top_amd as idx
            s["to"] = idx.Cache(s["codes"], s["scale"], D=q, fmt=idx.IDX_K_FP8_E4M3)
    return s


def prepare(case, seed):
    if case["op"] == "norm":
        return _prepare_norm(case, seed)
    g = _generator(seed)
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    n, keys = _requests(case)
    held = [-(-x // page) for x in keys]                       # pages of a request
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((B, max(held) + case["spare"]), dtype=torch.int32, device="cuda")
    at = 0
    for b, p in enumerate(held):
        table[b, :p] = order[at:at + p]
        at += p
    s = {"case": case, "pages": table}
    s["q"] = _normal(g, (case["T"], case["Hq"], D), DTYPES[case["dtype"]], 2.5)  # a softmax with few large terms
    s["k"], s["v"] = _cache(g, pages * page, Hkv, D, case["fmt"]), _cache(g, pages * page, Hkv, D, case["fmt"])
    s["cu_q"] = torch.tensor([sum(n[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    s["len_k"] = torch.tensor(keys, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ the plain forms
def _to_fp8(x):
    """E4M3 codes and one scale a row of the last dimension."""
    amax = x.abs().amax(-1)
    some = amax >= TINY
    scale = torch.where(some, amax / E4M3_MAX, 1.0)
    inverse = torch.where(some, E4M3_MAX / amax, 0.0)
    return (x * inverse[..., None]).to(torch.float8_e4m3fn), scale


def _plain_norm(s):
    case, x = s["case"], s["x"].float()
    out = []
    if s["residual"] is not None:
        x = x + s["residual"].float()
        out.append(x.to(s["residual"].dtype))
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if case["out"]:
        out.append(y.to(s["x"].dtype))
    if case["quant"]:
        out += _to_fp8(y.reshape(case["T"], -1, case["quant"]))
    return out


def _plain_attention(s):
    c = s["case"]
    T, B, Hq, Hkv, D = c["T"], c["B"], c["Hq"], c["Hkv"], c["D"]
    G, dev = Hq // Hkv, s["q"].device
    n = -(-T // B)                                             # rows and keys of the padded batch
    longest = max(_requests(c)[1])
    cu, keys = s["cu_q"].long(), s["len_k"].long()
    held = cu[1:] - cu[:-1]
    i, j = torch.arange(n, device=dev), torch.arange(longest, device=dev)
    slot = s["pages"].long()[:, j // c["page"]] * c["page"] + j % c["page"]          # [B, keys]

    def pick(x):
        v = x["data"][slot]
        v = v.view(torch.float8_e4m3fn).float() * x["scale"][slot][..., None] if x["scale"] is not None else v.float()
        return v.permute(0, 2, 1, 3)                           # [B, Hkv, keys, D]

    row = (cu[:-1, None] + i).clamp(max=T - 1)                 # [B, n]
    q = s["q"][row].float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    score = torch.matmul(q, pick(s["k"]).mT.contiguous()).mul_(D ** -0.5).view(B, Hkv, n, G, longest)
    pos = (keys - held)[:, None, None] + i[:, None]            # [B, n, 1]
    seen = j <= pos
    if c["window"]:
        seen &= (j > pos - c["window"]) | (j < c["first"])
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, Hkv, n * G, longest), pick(s["v"]).contiguous()).view(B, Hkv, n, G, D)
    out = (out / torch.where(total > 0, total, 1.0)).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(B, n, Hq)
    real = i < held[:, None]
    return [out[real].to(s["q"].dtype), lse[real]]


# ------------------------------------------------------------------------------------------------ libidx
def _libidx(s):
    import mqa_logits_top_amd as idx
    c = s["case"]
    if c["op"] == "norm":
        y = idx.idx_rms_norm(s["x"], s["weight"], eps=EPS, residual=s["residual"], total=s["total"], to=s["to"],
                             with_out=c["out"])
        return (([] if s["total"] is None else [s["total"]]) + ([y] if c["out"] else [])
                + ([s["codes"].view(torch.float8_e4m3fn), s["scale"]] if c["quant"] else []))
    return idx.idx_paged_attn(s["q"], s["k"]["handle"], s["v"]["handle"], s["pages"], s["cu_q"], s["len_k"],
                              scale=c["D"] ** -0.5, page=c["page"], window=c["window"], first=c["first"])


def run(state):
    if own:
        return list(_libidx(state))
    return _plain_norm(state) if state["case"]["op"] == "norm" else _plain_attention(state)


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    size = lambda t: 4 if t == "fp32" else 2
    if case["op"] == "norm":
        n = case["T"] * case["H"] * case["D"]
        width = case["D"] if case["heads"] else case["H"] * case["D"]
        bytes_ = n * size(case["dtype"]) * (2 if case["out"] else 1) + width * size(case["dtype"])
        if case["residual"]:
            bytes_ += 2 * n * size(case["residual"])
        if case["quant"]:
            bytes_ += n + 4 * (n // case["quant"])
        return {"bytes": bytes_, "flops": 6 * n}
    Hq, Hkv, D, T = case["Hq"], case["Hkv"], case["D"], case["T"]
    row = Hkv * (D + 4 if case["fmt"] == "fp8" else 2 * D)
    window, first = case["window"], case["first"]
    pairs = touched = 0
    for n, keys in zip(*_requests(case)):
        start = keys - n
        if not window:
            touched += keys
            pairs += n * start + n * (n + 1) // 2
            continue
        low = max(0, start - window + 1)                       # the first row's window
        touched += keys - low + min(first, low)
        for pos in range(start, keys):
            a = max(0, pos - window + 1)
            pairs += pos + 1 - a + min(first, a)
    return {"bytes": 2 * touched * row + T * Hq * (4 * D + 4) + 4 * (touched // case["page"]) + 8 * case["B"],
            "flops": 4 * Hq * D * pairs}


# ------------------------------------------------------------------------------------------------ from the definition
def _nearest(x):
    """The nearest E4M3 value, ties to the even code."""
    grid = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    a = x.abs()
    up = torch.searchsorted(grid, a.contiguous()).clamp(1, len(grid) - 1)
    below, above = grid[up - 1], grid[up]
    lower = (a - below < above - a) | ((a - below == above - a) & ((up - 1) % 2 == 0))
    return torch.copysign(torch.where(lower, below, above), x)


def _exact_norm(s):
    case, h = s["case"], s["x"].double()
    out = []
    if s["residual"] is not None:
        h = h + s["residual"].double()
        out.append(h)
    y = h / torch.sqrt(h.square().sum(-1, keepdim=True) / h.shape[-1] + EPS) * s["weight"].double()
    if case["out"]:
        out.append(y)
    if case["quant"]:
        groups = y.reshape(case["T"], -1, case["quant"])
        scale = groups.abs().amax(-1) / E4M3_MAX
        out += [_nearest(groups / scale[..., None]), scale]
    return out


def _exact_attention(s):
    """Request by request, cache head by cache head, at most 2^27 scores at a time."""
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    G, dev = Hq // Hkv, s["q"].device
    out = torch.zeros((c["T"], Hq, D), dtype=torch.float64, device=dev)
    lse = torch.full((c["T"], Hq), -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for b, (n, keys) in enumerate(zip(*_requests(c))):
        key = torch.arange(keys, device=dev)
        slot = s["pages"][b][key // page].long() * page + key % page
        step = max(1, (1 << 27) // (G * keys))
        for h in range(Hkv):
            kv = []
            for x in (s["k"], s["v"]):
                rows = x["data"][slot, h]
                kv.append(rows.double() if x["scale"] is None else
                          rows.view(torch.float8_e4m3fn).double() * x["scale"][slot, h].double()[:, None])
            for a in range(0, n, step):
                e = min(a + step, n)
                q = s["q"][at + a:at + e, h * G:(h + 1) * G].double().reshape(-1, D)
                pos = (torch.arange(a, e, device=dev) + keys - n).repeat_interleave(G)[:, None]
                hidden = key > pos
                if c["window"]:
                    hidden |= (pos - key >= c["window"]) & (key >= c["first"])
                score = (q @ kv[0].T.contiguous() / math.sqrt(D)).masked_fill(hidden, -math.inf)
                lse[at + a:at + e, h * G:(h + 1) * G] = torch.logsumexp(score, -1).view(e - a, G)
                out[at + a:at + e, h * G:(h + 1) * G] = (torch.softmax(score, -1) @ kv[1]).view(e - a, G, D)
        at += n
    return [out, lse]


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "norm" else _exact_attention(s)
