"""8-bit paged key/value cache: append with the position rotation (fp32, in the
written operation order), and attention over it (fp64).

Storage: K codes int8 [page][head][slot][dim], V codes int8 [page][head][dim][slot],
scales fp32 [page][head][2] (K, V); value = scale * code.  A batch is ragged:
sequence b owns tokens offsets[b] .. offsets[b+1]-1, the last of its kv_lens[b].

Append, per page and head (K and V apart): s = max |new| / 127, or the old scale
if the page already holds earlier tokens and it is larger; earlier codes become
rint(q * (s_old * (1/s))) where s grew; new codes clamp(rint(x * (1/s)), +-127).
Scales below 2^-126 (K) or 2^-80 (V) are 0 (codes 0); a value that is not finite makes the scale NaN.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import numpy as np

F = np.float32


def rope_tables(max_pos: int, rot: int, base: float = 10000.0):
    angle = np.arange(max_pos, dtype=np.float64)[:, None] * base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    return np.cos(angle).astype(F), np.sin(angle).astype(F)


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, rot: int, pairs: bool) -> np.ndarray:
    """x fp32 [heads][dim] of one token; cos, sin fp32 [rot / 2] of its position."""
    y = x.astype(F).copy()
    if rot:
        ia = np.arange(0, rot, 2) if pairs else np.arange(rot // 2)
        ib = ia + 1 if pairs else ia + rot // 2
        a, b = x[:, ia].astype(F), x[:, ib].astype(F)
        y[:, ia] = (a * cos) - (b * sin)
        y[:, ib] = (b * cos) + (a * sin)
    return y


def _quantize(x: np.ndarray, inv: np.float32) -> np.ndarray:
    with np.errstate(all="ignore"):
        return np.clip(np.rint(x.astype(F) * inv), F(-127), F(127))


def _store(fresh: np.ndarray, old_codes: np.ndarray, s_old: np.float32, least: float):
    """fresh fp32 [t][dim], old_codes int8 [olds][dim]: (scale, all codes, whether the codes mean anything)."""
    a = np.max(np.abs(fresh)) if np.isfinite(fresh).all() else F(np.nan)
    s = F(a) / F(127)
    if len(old_codes):
        s = F(np.nan) if np.isnan(s) or np.isnan(s_old) else max(s, F(s_old))
    if s < F(least):
        s = F(0)
    if np.isnan(s):
        return s, np.zeros((len(old_codes) + len(fresh), fresh.shape[1]), np.int8), False
    inv = F(1) / s if s > 0 else F(0)
    kept = old_codes.astype(F)
    if len(old_codes) and s != s_old:
        kept = _quantize(kept, F(s_old) * inv)
    return s, np.concatenate([kept, _quantize(fresh, inv)]).astype(np.int8), True


def append(k_codes, v_codes, scales, offsets, kv_lens, table, Q, K, V, cos, sin, rot, pairs):
    """Updates the cache arrays in place; returns the rotated queries (fp32, not rounded).  Q, K, V fp32
    [tokens][heads][dim]."""
    H, P = k_codes.shape[1:3]
    q_out = Q.astype(F).copy()
    for b in range(len(kv_lens)):
        row, n, m = int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(kv_lens[b])
        rotated = []
        for i in range(n):
            at = max(m - n + i, 0)
            c, s = (cos[min(at, len(cos) - 1)], sin[min(at, len(sin) - 1)]) if rot else (None, None)
            q_out[row + i] = rotate(Q[row + i], c, s, rot, pairs)
            rotated.append(rotate(K[row + i], c, s, rot, pairs))
        lo = max(m - n, 0)
        while lo < m:
            p = lo // P
            hi, page, olds = min(m, (p + 1) * P), int(table[b][p]), lo - p * P
            if 0 <= page < len(k_codes):
                t = slice(lo - (m - n), hi - (m - n))
                for h in range(H):
                    fresh_k = np.stack([r[h] for r in rotated[t]])
                    s, codes, _ = _store(fresh_k, k_codes[page, h, :olds], scales[page, h, 0], 2.0 ** -126)
                    scales[page, h, 0] = s
                    k_codes[page, h, :olds + hi - lo] = codes
                    fresh_v = V[row:row + n][t][:, h]
                    s, codes, _ = _store(fresh_v, v_codes[page, h, :, :olds].T, scales[page, h, 1], 2.0 ** -80)
                    scales[page, h, 1] = s
                    v_codes[page, h, :, :olds + hi - lo] = codes.T
            lo = hi
    return q_out


def values(k_codes, v_codes, scales, table_row, length, head):
    """fp64 keys and values [length][dim] of one sequence and head, and which positions are held (NaN elsewhere)."""
    P, D = k_codes.shape[2:]
    k, v, held = np.full((length, D), np.nan), np.full((length, D), np.nan), np.zeros(length, bool)
    for p in range(-(-length // P)):
        page, lo, hi = int(table_row[p]), p * P, min(length, (p + 1) * P)
        if 0 <= page < len(k_codes):
            k[lo:hi] = k_codes[page, head, :hi - lo].astype(np.float64) * np.float64(scales[page, head, 0])
            v[lo:hi] = v_codes[page, head, :, :hi - lo].T.astype(np.float64) * np.float64(scales[page, head, 1])
            held[lo:hi] = True
    return k, v, held


def visible(p: int, length: int, window: int, sinks: int) -> np.ndarray:
    j = np.arange(length)
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    return seen


def attention(k_codes, v_codes, scales, offsets, kv_lens, table, Q, scale, window, sinks):
    """fp64: outputs [tokens][q_heads][dim], the weighted means of |v| in the same layout, and per row the largest
    sum |q k| scale of a visible score and the largest visible |v| (what rounding errors scale with)."""
    T, Hq, D = Q.shape
    Hk = k_codes.shape[1]
    G = Hq // Hk
    Y, A = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    score, peak = np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(kv_lens)):
        row, n, m = int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(kv_lens[b])
        for h in range(Hk):
            k, v, held = values(k_codes, v_codes, scales, table[b], m, h)
            for i in range(n):
                seen = visible(m - n + i, m, window, sinks) & held
                if not seen.any():
                    continue
                ks, vs = k[seen], v[seen]
                for hq in range(h * G, h * G + G):
                    q = Q[row + i, hq].astype(np.float64)
                    x = (ks @ q) * scale
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    Y[row + i, hq], A[row + i, hq] = w @ vs, w @ np.abs(vs)
                    score[row + i, hq] = (np.abs(ks) @ np.abs(q)).max() * scale
                    peak[row + i, hq] = np.abs(vs).max()
    return Y, A, score, peak


def attention_scored(k_codes, v_codes, scales, offsets, kv_lens, table, Q, scale, window, sinks, cap=0.0, slopes=None,
                     prefix_lens=None, starts=None):
    """As attention, with scores capped by cap tanh(x / cap) and lowered by slopes[head] |p - j|, prefixes of sequences
    that all their queries see, and first visible positions of tokens; also per row the largest visible slope |p - j|."""
    T, Hq, D = Q.shape
    Hk = k_codes.shape[1]
    G = Hq // Hk
    Y, A = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    score, peak, far = np.zeros((T, Hq)), np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(kv_lens)):
        row, n, m = int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(kv_lens[b])
        j = np.arange(m)
        for h in range(Hk):
            k, v, held = values(k_codes, v_codes, scales, table[b], m, h)
            for i in range(n):
                p = m - n + i
                start = max(int(starts[row + i]), 0) if starts is not None else 0
                seen = (j <= p) | ((j < int(prefix_lens[b])) if prefix_lens is not None else False)
                if window:
                    seen &= (j > p - window) | (j < start + sinks)
                seen &= held & (j >= start) & (p >= 0)
                if not seen.any():
                    continue
                ks, vs, away = k[seen], v[seen], np.abs(p - j[seen]).astype(np.float64)
                for hq in range(h * G, h * G + G):
                    q = Q[row + i, hq].astype(np.float64)
                    x = (ks @ q) * scale
                    if cap:
                        x = cap * np.tanh(x / cap)
                    if slopes is not None:
                        x = x - float(slopes[hq]) * away
                        far[row + i, hq] = abs(float(slopes[hq])) * away.max()
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    Y[row + i, hq], A[row + i, hq] = w @ vs, w @ np.abs(vs)
                    score[row + i, hq] = (np.abs(ks) @ np.abs(q)).max() * scale
                    peak[row + i, hq] = np.abs(vs).max()
    return Y, A, score, peak, far
