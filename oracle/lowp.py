"""Oracle of the 8-bit block-scaled products and of the routing to experts -- TEST INFRASTRUCTURE ONLY.

Plain definitions in numpy, 64 bits wherever the definition is a real number,
sharing no code with the CUDA path:

* ``e4m3_values``: the 256 code values from the format (sign, 4 exponent bits
  of bias 7, 3 mantissa bits, no infinities, NaN 0x7F and 0xFF).
* ``fp8_pack``: s = max(amax / 448, 2^-126) rounded to fp32, code nearest to
  x * 448 / amax (x * 2^126 for the least scale) rounded to fp32, ties to the
  even code.
* ``fp8_gemm``: products of the real values in float64, and the sum of the
  magnitudes that bounds the rounding of any order of addition.
* ``route``, ``route_plan``, ``route_combine``: token by token.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 128


def e4m3_values() -> np.ndarray:
    v = np.empty(256, dtype=np.float64)
    for c in range(256):
        sign, e, m = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            v[c] = math.nan
        elif e == 0:
            v[c] = sign * m * 2.0 ** -9
        else:
            v[c] = sign * (1 + m / 8) * 2.0 ** (e - 7)
    return v


VALUES = e4m3_values()


def e4m3_nearest(q: np.ndarray) -> np.ndarray:
    """Codes nearest to finite q (|q| <= 464), ties to the even code; the sign of a zero is kept."""
    pos = VALUES[:127]                                  # 0 .. 448, ascending
    a = np.minimum(np.abs(q.astype(np.float64)), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dlo, dhi = a - pos[lo], pos[hi] - a
    pick = np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick | np.where(np.signbit(q), 0x80, 0)).astype(np.uint8)


def fp8_pack(x: np.ndarray, block_rows: int):
    """x float32 [rows, K] -> (codes uint8 [rows, K], scales float32 [blocks of K, row blocks])."""
    x = np.asarray(x, dtype=np.float32)
    rows, K = x.shape
    nb, nr = -(-K // BLOCK), -(-rows // block_rows)
    codes = np.zeros((rows, K), np.uint8)
    scales = np.zeros((nb, nr), np.float32)
    for b in range(nb):
        for i in range(nr):
            t = x[i * block_rows:(i + 1) * block_rows, b * BLOCK:(b + 1) * BLOCK]
            fin = np.abs(t[np.isfinite(t)])
            amax = fin.max() if fin.size else np.float32(0)
            s = np.maximum(np.float32(amax) / np.float32(448.0), np.float32(2.0 ** -126))
            scales[b, i] = s
            with np.errstate(invalid="ignore", over="ignore", under="ignore"):
                least = amax < 448.0 * 2.0 ** -126
                q = t.astype(np.float64) * (2.0 ** 126 if least else 448.0) / (1.0 if least else float(amax))
                q = q.astype(np.float32)
            c = e4m3_nearest(np.where(np.isfinite(t), q, np.float32(0)))
            c = np.where(np.isfinite(t), c, 0x7F)       # the sign of a NaN code says nothing
            codes[i * block_rows:(i + 1) * block_rows, b * BLOCK:(b + 1) * BLOCK] = c
    return codes, scales


def fp8_values(codes: np.ndarray, scales: np.ndarray, K: int, block_rows: int) -> np.ndarray:
    rows = codes.shape[0]
    i, b = np.arange(rows) // block_rows, np.arange(K) // BLOCK
    return VALUES[codes[:, :K]] * scales.astype(np.float64)[b[None, :], i[:, None]]


def fp8_gemm(A, a_scales, W, w_scales, K: int):
    """(C, sum of |products|) in float64."""
    a, w = fp8_values(A, a_scales, K, 1), fp8_values(W, w_scales, K, BLOCK)
    return a @ w.T, np.abs(a) @ np.abs(w).T


def route(logits: np.ndarray, k: int, score: str, bias=None, n_groups: int = 1, kept_groups: int = 1,
          group_top: int = 2, renormalize: bool = True, scale: float = 1.0):
    """(idx int32 [T, k], weights float64 [T, k])."""
    T, E = logits.shape
    idx = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k), np.float64)
    big = float(np.finfo(np.float32).max)
    for t in range(T):
        l = logits[t].astype(np.float64)
        on = ~np.isnan(l) & (l > -math.inf)
        l = np.where(on, np.minimum(l, big), 0.0)
        s = np.zeros(E)
        if on.any():
            with np.errstate(over="ignore", under="ignore"):
                if score == "softmax":
                    ex = np.where(on, np.exp(l - l[on].max()), 0.0)
                    s = ex / ex.sum()
                else:
                    s = np.where(on, 1.0 / (1.0 + np.exp(-l)), 0.0)
        c = s.copy() if bias is None else s + bias.astype(np.float64)
        c = np.where(on & ~np.isnan(c), c, -math.inf)
        if n_groups > 1:
            per = E // n_groups
            gs = []
            for g in range(n_groups):
                top = sorted(c[g * per:(g + 1) * per], reverse=True)
                top = [v for v in top[:group_top] if v > -math.inf]
                gs.append(sum(top) if top else -math.inf)
            keep = sorted(range(n_groups), key=lambda g: (-gs[g], g))[:kept_groups]
            for g in range(n_groups):
                if g not in keep:
                    c[g * per:(g + 1) * per] = -math.inf
        order = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > -math.inf][:k]
        w = np.array([s[e] for e in order])
        if renormalize and len(order):
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        idx[t, :len(order)] = order
        weights[t, :len(order)] = w * scale
    return idx, weights


def route_plan(idx: np.ndarray, E: int):
    """(offsets [E + 1], row_token [T * k], slot_row [T, k])."""
    T, k = idx.shape
    rows = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if idx[t, j] >= 0:
                rows[idx[t, j]].append(t * k + j)
    offsets = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int32)
    row_token = np.full(T * k, -1, np.int32)
    slot_row = np.full(T * k, -1, np.int32)
    for r, s in enumerate(s for part in rows for s in part):
        row_token[r] = s // k
        slot_row[s] = r
    return offsets, row_token, slot_row.reshape(T, k)


def route_combine(Y: np.ndarray, slot_row: np.ndarray, weights: np.ndarray):
    """(out, sum of |terms|) in float64."""
    T, k = slot_row.shape
    out = np.zeros((T, Y.shape[1]))
    mag = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < Y.shape[0]:
                out[t] += float(weights[t, j]) * Y[r].astype(np.float64)
                mag[t] += abs(float(weights[t, j])) * np.abs(Y[r].astype(np.float64))
    return out, mag
