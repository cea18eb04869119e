"""Plain 64-bit forms of attention over a paged cache and of the RMS norm, from the definitions in include/idx.h."""
from __future__ import annotations

import numpy as np

from around_ref import HALF_STEP, SMALLEST, quantise_e4m3


def slots_seen(T, pages, page, cu_q, len_k, rows, window=0, first=0):
    """Per row the slots of the keys it sees, in order (None: the row is in no request)."""
    pages, out = np.asarray(pages, np.int64), [None] * T
    for b in range(len(len_k)):
        n = int(cu_q[b + 1]) - int(cu_q[b])
        length = min(max(int(len_k[b]), 0), pages.shape[1] * page)
        for i in range(n):
            pos = length - n + i
            s = np.arange(pos + 1, dtype=np.int64)
            if window:
                s = s[(s > pos - window) | (s < first)]
            slot = pages[b, s // page] * page + s % page
            out[int(cu_q[b]) + i] = slot[(slot >= 0) & (slot < rows)]
    return out


def weight_step(q_bf16: bool, fp8: bool) -> float:
    """Half a step of a weight of the second product."""
    return 2.0 ** -8 if q_bf16 else 2.0 ** -16 if fp8 else 2.0 ** -11


def rms_norm(x, residual, weight, eps):
    """x [..., D] fp64 and the rest likewise or None: (sum, y)."""
    h = x if residual is None else x + residual
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h, y if weight is None else y * weight


def norm_bound(h, y, D, residual):
    """What y may be off in fp32 before it is rounded to its type: the sum h of two values is rounded once (2^-24 of h),
    and so is each of the two products and the reciprocal root (its division, root, quotient and sum: 4 roundings, half of
    those under the root), and the squares' sum of D terms moves the root by at most (D / 2 + 2) roundings."""
    return ((D / 2 + 2) + 8) * 2.0 ** -24 * np.abs(y) + (2.0 ** -23 * np.abs(y) if residual else 0.0)


__all__ = ["HALF_STEP", "SMALLEST", "norm_bound", "quantise_e4m3", "rms_norm", "slots_seen", "weight_step"]
