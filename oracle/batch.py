"""Packed batches over the paged cache, plain numpy (test infrastructure only): row maps, bounds of
pages' keys, the blocks that a row picks, and the attention of packed rows in 64 bits."""
from __future__ import annotations

import numpy as np


def batch_rows(table, lens, ps, n_pages, seqs, start, counts, rows):
    """(row_start, row_seq, row_pos, row_slot) one row at a time."""
    max_seqs = len(lens)
    row_start, maps = [0], np.full((3, rows), -1, np.int64)
    at = 0
    for i, c in enumerate(counts):
        c = max(int(c), 0)
        s = i if seqs is None else int(seqs[i])
        named = seqs is not None and s in [int(x) for x in seqs[:i]]
        ok = 0 <= s < max_seqs and not named
        length = min(max(int(lens[s]), 0), table.shape[1] * ps) if ok else 0
        first = length - min(c, rows - at) if start is None else int(start[i])   # of the rows that the arrays hold
        for t in range(c):
            if at >= rows:
                break
            if ok and first >= 0:
                p = first + t
                maps[0, at], maps[1, at] = s, p
                if p < length and 0 <= table[s, p // ps] < n_pages:
                    maps[2, at] = int(table[s, p // ps]) * ps + p % ps
            at += 1
        row_start.append(at)
    return np.array(row_start, np.int32), *maps.astype(np.int32)


def bounds(keys):
    """(codes int8 [2][D], scale) of a page's filled keys [slots][D] in fp32."""
    k = np.asarray(keys, np.float32)
    if not np.isfinite(k).all():
        return np.zeros((2, k.shape[1]), np.int8), np.float32(np.inf)
    lo, hi = k.min(0), k.max(0)
    s = np.float32(np.float32(max(np.abs(lo).max(), np.abs(hi).max())) / np.float32(127))
    if s == 0:
        return np.zeros((2, k.shape[1]), np.int8), s
    c = np.stack([np.floor(lo / s), np.ceil(hi / s)])
    return np.clip(c, -127, 127).astype(np.int8), s


def scores(q, codes, scales):
    """Scores of blocks for the heads q [rep][D] of one group: codes int8 [blocks][2][D], scales [blocks]."""
    best = np.full(len(scales), -np.inf, np.float32)
    for x in np.asarray(q, np.float32):
        top = np.abs(x).max()
        s = np.float32(top / np.float32(127)) if np.isfinite(x).all() else np.float32(np.inf)
        c = np.zeros(x.shape, np.int64)
        if 0 < s < np.inf:
            c = np.clip(np.rint(x / s), -127, 127).astype(np.int64)
        u = np.where(c > 0, c * codes[:, 1].astype(np.int64), c * codes[:, 0].astype(np.int64)).sum(1)
        with np.errstate(invalid="ignore"):
            v = u.astype(np.float32) * scales.astype(np.float32) * s
        best = np.maximum(best, np.where(np.isnan(v), np.float32(np.inf), v))
    return best


def pick(score, keep, first, recent):
    """The blocks that are read, ascending."""
    n = len(score)
    if n <= keep:
        return list(range(n))
    always = sorted(set(range(first)) | set(range(n - recent, n)))
    rest = sorted((b for b in range(n) if b not in always), key=lambda b: (-score[b], b))
    return sorted(always + rest[:keep - len(always)])


def attend(q, k, v, positions, window=0, sinks=0):
    """Rows q [rows][Hq][D] at `positions` over k, v [Hkv][len][D]: (out, lse, sum of weight * |value|)."""
    rows, Hq, D = q.shape
    out, mag, lse = np.zeros((rows, Hq, D)), np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
    p, j = np.asarray(positions)[:, None], np.arange(k.shape[1])[None]
    seen = j <= p
    if window > 0:
        seen &= (j > p - window) | (j < sinks)
    for h in range(Hq):
        kk, vv = k[h // (Hq // k.shape[0])], v[h // (Hq // k.shape[0])]
        kk, vv = np.where(seen.any(0)[:, None], kk, 0.0), np.where(seen.any(0)[:, None], vv, 0.0)
        l = np.where(seen, q[:, h].astype(np.float64) @ kk.T / np.sqrt(D), -np.inf)
        m = l.max(axis=1, initial=-np.inf, keepdims=True)
        w = np.exp(l - np.where(np.isfinite(m), m, 0.0))
        s = w.sum(axis=1, keepdims=True)
        with np.errstate(divide="ignore"):
            lse[:, h] = (m + np.log(s))[:, 0]
        w /= np.where(s > 0, s, 1.0)
        out[:, h], mag[:, h] = w @ vv, w @ np.abs(vv)
    return out, lse, mag


