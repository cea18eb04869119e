"""Plain 64-bit forms of the operators around the indexer, and bounds on what the kernels may be off.

Everything here is numpy / torch on the CPU, written from the definitions in include/idx.h."""
from __future__ import annotations

import numpy as np
import torch

import synth

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float64)
E4M3 = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SMALLEST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def rotate(x: np.ndarray, pos: np.ndarray, freq: np.ndarray, rot0: int, half: bool, mscale=1.0, inverse=False):
    """x [T, H, D] fp64 -> (rotated fp64, sum of the magnitudes that enter each value)."""
    n = len(freq)
    ang = pos.astype(np.float64)[:, None, None] * freq * (-1.0 if inverse else 1.0)
    c, s = np.cos(ang) * mscale, np.sin(ang) * mscale
    ia = rot0 + (np.arange(n) if half else 2 * np.arange(n))
    ib = ia + (n if half else 1)
    out, mag = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (np.abs(a) + np.abs(b)) * abs(mscale)
    return out, mag


def rotate_bound(want: np.ndarray, mag: np.ndarray, dtype) -> np.ndarray:
    """The angle and its cosine and sine, in fp64, are off by less than 2^-23 on the pair's magnitudes; the sum is
    rounded to fp32 (2^-24) and to the output's type (half a step)."""
    return (HALF_STEP[dtype] + 2.0 ** -23) * np.abs(want) + 2.0 ** -23 * mag + SMALLEST[dtype]


def quantise_e4m3(x: np.ndarray):
    """x fp32 [..., D] -> (codes, scale fp32 [...]) in the arithmetic of the definition."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(-1)
    some = amax >= np.float32(2.0 ** -100)
    scale = np.where(some, amax / np.float32(448), np.float32(1)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        y = x.astype(np.float64) * 448 / np.where(some, amax, np.inf)[..., None].astype(np.float64)
    y = y.astype(np.float32)
    return synth.encode_e4m3(y.astype(np.float64)), scale


def quantise_mxfp4(x: np.ndarray):
    """x fp32 [..., D] -> (packed uint8 [..., D / 2], E8M0 uint8 [..., D / 32])."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(b).max(-1)
    some = amax >= 2.0 ** -100
    e = np.where(some, np.floor(np.log2(np.where(some, amax, 1.0))) - 2, -127)
    y = np.where(some[..., None], b * 2.0 ** -e[..., None], 0.0)
    codes = synth.encode_e2m1(y).reshape(x.shape)
    codes = np.where(np.repeat(some, 32, -1), codes, 0).astype(np.uint8)
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8), (e + 127).astype(np.uint8)


def read_e4m3(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    return E4M3[codes] * scale.astype(np.float64)[..., None]


def read_mxfp4(packed: np.ndarray, e8: np.ndarray) -> np.ndarray:
    code = np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(e8 == 255, np.nan, 2.0 ** (e8.astype(np.float64) - 127))
    return v * np.repeat(s, 32, -1)


def keys_of(sel, ks, ke, pool, L, table, rows):
    """Per row of the list the cache rows of the entries that count, in order (an int64 array a row)."""
    out = []
    for t in range(len(sel)):
        ids = sel[t].astype(np.int64)
        ids = ids[ids >= 0]
        if pool > 1:
            ids = (ks[t] + ids[:, None] * pool + np.arange(pool)).reshape(-1)
        lo, hi = (0, L) if ks is None else (max(int(ks[t]), 0), min(int(ke[t]), L))
        ids = ids[(ids >= lo) & (ids < hi)]
        r = ids if table is None else table[ids].astype(np.int64)
        out.append(r[(r >= 0) & (r < rows)])
    return out


def attend(q, k, v, rows, scale, weight_step, dtype):
    """q [T, Hq, D], k and v [slots, Hkv, D] fp64, rows from keys_of: (out, lse, bound of out, bound of lse).

    The bounds: a score is a sum of D exact products in fp32 (D + 2 roundings of 2^-24 of the products'
    magnitudes, once more for the scales), off by ds; weights are exp of it, off by 2 ds where the
    normalisation moves with them, plus 2^-21 for the exponential, its argument's rounding (2^-23 of the
    largest score's distance, within ds) and the reciprocal; each weight is rounded
    (weight_step: half a step; fp16 weights below its smallest normal lose up to 2^-25 of the largest);
    sums over n keys add n 2^-23; the result is rounded to the output's type."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    bo, bl = np.full((T, Hq, D), SMALLEST[dtype]), np.zeros((T, Hq))
    for t in range(T):
        r = rows[t]
        if not len(r):
            continue
        kk, vv = np.repeat(k[r], G, 1), np.repeat(v[r], G, 1)          # [n, Hq, D]
        s = np.einsum("hd,nhd->hn", q[t], kk) * scale
        mag = np.einsum("hd,nhd->hn", np.abs(q[t]), np.abs(kk)) * abs(scale)
        ds = ((D + 6) * 2.0 ** -24 * mag).max(1) + 2.0 ** -22 * np.abs(s).max(1)
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        total = p.sum(1)
        lse[t] = top[:, 0] + np.log(total)
        out[t] = np.einsum("hn,nhd->hd", p, vv) / total[:, None]
        pv = np.einsum("hn,nhd->hd", p, np.abs(vv)) / total[:, None]
        n = len(r)
        rel = np.expm1(4 * ds) + weight_step + 2.0 ** -21 + n * 2.0 ** -23
        bo[t] += rel[:, None] * pv + (HALF_STEP[dtype] + 2.0 ** -22) * np.abs(out[t])
        if weight_step < 2.0 ** -9:
            bo[t] += 2.0 ** -25 * np.abs(vv).sum(0) / total[:, None]
        bl[t] = 2 * ds + 2.0 ** -21 + n * 2.0 ** -23 + 2.0 ** -22 * np.abs(lse[t])
    return out, lse, bo, bl
