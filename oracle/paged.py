"""Paged cache and windowed attention, plain numpy in 64 bits (test infrastructure only).

The page operators follow their definition one request and one page at a time: new pages are
the free pages (reference count 0) of lowest number, a fork shares full pages and copies a
partly filled last one, compaction moves the kept slots into new pages.
"""
from __future__ import annotations

import numpy as np


def visible(p, n_keys, window, sinks):
    """Which of n_keys keys a query at position p sees."""
    j = np.arange(n_keys)
    seen = j <= p
    if window > 0:
        seen &= (j > p - window) | (j < sinks)
    return seen


def attend_row(q, k, v, seen):
    """One query over the keys it sees: (out, lse, sum of weight * |value|)."""
    D = q.shape[-1]
    if not seen.any():
        return np.zeros(D), -np.inf, np.zeros(D)
    k, v = k[seen].astype(np.float64), v[seen].astype(np.float64)
    l = k @ q.astype(np.float64) / np.sqrt(D)
    m = l.max()
    w = np.exp(l - m)
    lse = m + np.log(w.sum())
    w /= w.sum()
    return w @ v, lse, w @ np.abs(v)


def window_attention(q, k, v, window, sinks, q_lens=None, k_lens=None):
    """q [B,Hq,Tq,D], k, v [B,Hkv,Tk,D] float arrays; rows at or past q_lens are NaN in the result."""
    B, Hq, Tq, D = q.shape
    Hkv, Tk = k.shape[1], k.shape[2]
    out = np.full((B, Hq, Tq, D), np.nan)
    mag = np.full((B, Hq, Tq, D), np.nan)
    lse = np.full((B, Hq, Tq), np.nan)
    for b in range(B):
        ql = Tq if q_lens is None else min(max(int(q_lens[b]), 0), Tq)
        kl = Tk if k_lens is None else min(max(int(k_lens[b]), 0), Tk)
        p = kl - ql + np.arange(ql)[:, None]
        j = np.arange(kl)[None]
        seen = j <= p
        if window > 0:
            seen &= (j > p - window) | (j < sinks)
        for h in range(Hq):
            kk = k[b, h // (Hq // Hkv), :kl].astype(np.float64)
            vv = v[b, h // (Hq // Hkv), :kl].astype(np.float64)
            l = np.where(seen, q[b, h, :ql].astype(np.float64) @ kk.T / np.sqrt(D), -np.inf)
            m = l.max(axis=1, initial=-np.inf, keepdims=True)
            w = np.exp(l - np.where(np.isfinite(m), m, 0.0))
            s = w.sum(axis=1, keepdims=True)
            with np.errstate(divide="ignore"):
                lse[b, h, :ql] = (m + np.log(s))[:, 0]
            w /= np.where(s > 0, s, 1.0)
            out[b, h, :ql], mag[b, h, :ql] = w @ vv, w @ np.abs(vv)
    return out, lse, mag


class Pages:
    """k, v: stored rows [layers][n_pages][Hkv][ps][...]; any array type."""

    def __init__(self, k, v, table, lens, refs):
        self.k, self.v = k.copy(), v.copy()
        self.table, self.lens, self.refs = table.copy(), lens.copy(), refs.copy()
        self.ps = k.shape[3]

    def pages_of(self, n):
        return -(-int(n) // self.ps)

    def valid(self, s):
        return 0 <= s < len(self.lens)

    def _grant(self, needs):
        """Free pages for each request's need (None: not valid), or None where they do not suffice."""
        free = list(np.flatnonzero(self.refs == 0))
        got, used = [], 0
        for need in needs:
            if need is None:
                got.append(None)
                continue
            used += need
            got.append(free[used - need:used] if need == 0 or used <= len(free) else None)
        return got

    def reserve(self, seqs, add):
        cap = self.table.shape[1] * self.ps
        needs = []
        for i, (s, a) in enumerate(zip(seqs, add)):
            ok = self.valid(s) and s not in seqs[:i] and a >= 0 and self.lens[s] + a <= cap
            needs.append(self.pages_of(self.lens[s] + a) - self.pages_of(self.lens[s]) if ok else None)
        start = []
        for s, a, got in zip(seqs, add, self._grant(needs)):
            start.append(-1 if got is None else int(self.lens[s]))
            if got is not None:
                have = self.pages_of(self.lens[s])
                self.table[s, have:have + len(got)] = got
                self.refs[got] = 1
                self.lens[s] += a
        return np.array(start, np.int32)

    def fork(self, parent, child):
        needs = []
        for i, (s, c) in enumerate(zip(parent, child)):
            ok = self.valid(s) and self.valid(c) and c not in parent and c not in child[:i] and self.lens[c] == 0
            needs.append(int(self.lens[s] % self.ps > 0) if ok else None)
        ok = []
        for s, c, got in zip(parent, child, self._grant(needs)):
            ok.append(int(got is not None))
            if got is None:
                continue
            full, rest = divmod(int(self.lens[s]), self.ps)
            self.table[c, :full] = self.table[s, :full]
            self.refs[self.table[s, :full]] += 1
            if rest:
                self.table[c, full] = got[0]
                self.refs[got[0]] = 1
                for x in (self.k, self.v):
                    x[:, got[0], :, :rest] = x[:, self.table[s, full], :, :rest]
            self.lens[c] = self.lens[s]
        return np.array(ok, np.int32)

    def free(self, seqs):
        ok = []
        for i, s in enumerate(seqs):
            ok.append(int(self.valid(s) and s not in seqs[:i]))
            if ok[-1]:
                mine = self.table[s, :self.pages_of(self.lens[s])]
                self.refs[mine] -= 1
                mine[:] = -1
                self.lens[s] = 0
        return np.array(ok, np.int32)

    def copy(self, src, dst):
        n, ok = len(self.refs), []
        for i, (s, d) in enumerate(zip(src, dst)):
            fine = 0 <= s < n and 0 <= d < n and d not in dst[:i]
            fine = fine and not any(src[j] == d for j in range(len(src)) if j != i)
            ok.append(int(fine))
        for s, d, fine in zip(src, dst, ok):
            if fine:
                self.k[:, d], self.v[:, d] = self.k[:, s], self.v[:, s]
        return np.array(ok, np.int32)

    def compact(self, seqs, keep_pos, keep_n):
        layers, _, Hkv, most = keep_pos.shape
        needs = []
        for i, (s, n) in enumerate(zip(seqs, keep_n)):
            ok = self.valid(s) and s not in seqs[:i] and 0 <= n <= min(most, self.lens[s])
            needs.append(self.pages_of(n) if ok else None)
        ok, todo = [], []
        for i, (s, n, got) in enumerate(zip(seqs, keep_n, self._grant(needs))):
            at = keep_pos[:, i, :, :max(int(n), 0)]
            fine = got is not None and bool(((at >= 0) & (at < self.lens[s])).all())
            ok.append(int(fine))
            if not fine:
                continue
            rows = self.table[s]
            for j in range(n):
                for l in range(layers):
                    for h in range(Hkv):
                        p = at[l, h, j]
                        for x in (self.k, self.v):
                            x[l, got[j // self.ps], h, j % self.ps] = x[l, rows[p // self.ps], h, p % self.ps]
            todo.append((s, n, got))
        for s, n, got in todo:
            mine = self.table[s, :self.pages_of(self.lens[s])]
            np.subtract.at(self.refs, mine, 1)
            mine[:] = -1
            self.table[s, :len(got)] = got
            self.refs[got] = 1
            self.lens[s] = n
        return np.array(ok, np.int32)

    def rows(self, x, layer, s):
        """Sequence s's stored rows in slot order, [len][Hkv][...]."""
        j = np.arange(self.lens[s])
        return x[layer][self.table[s][j // self.ps], :, j % self.ps]
