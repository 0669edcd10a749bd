"""Oracle of attention, the rotary embedding and the pages of a cache (test
infrastructure only; see the package docstring), in float64 from the definition:

  y_i = sum over the keys j <= last_i of p_ij v_j,  p_ij = exp(s_ij) / sum exp(s_ij),
  s_ij = scale q_i . k_j

A query that sees no key, or none with a score above -inf, has y = 0 and a
logarithm of its sum of -inf.  What a query does not see takes no part at all.
"""
from __future__ import annotations

import numpy as np


def attend(q, k, v, last, scale):
    """One sequence: q [n, H, D], k, v [m, Hk, D], last [n] -> a dict of y [n, H, D], lse
    [n, H], `size` (sum p |v|, what errors of the weights scale with) and `score` [n, H]
    (the largest scale * sum |q k|, what errors of the scores scale with)."""
    n, H, D = q.shape
    G = H // k.shape[1] if k.shape[1] else 1
    y, size = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, score = np.full((n, H), -np.inf), np.zeros((n, H))
    with np.errstate(all="ignore"):
        for i in range(n):
            seen = min(int(last[i]) + 1, k.shape[0])
            if seen <= 0:
                continue
            for h in range(H):
                kk, vv = k[:seen, h // G], v[:seen, h // G]
                s = scale * (kk * q[i, h]).sum(1)
                score[i, h] = scale * np.abs(kk * q[i, h]).sum(1).max()
                top = s.max()
                if top == -np.inf:
                    continue
                p = np.exp(s - top)
                lse[i, h] = top + np.log(p.sum())
                p = p / p.sum()
                y[i, h] = (p[:, None] * vv).sum(0)
                size[i, h] = (p[:, None] * np.abs(vv)).sum(0)
    return {"y": y, "lse": lse, "size": size, "score": score}


def rotate(x, positions, inv_freq, interleaved):
    """x [n, heads, D] with its first 2 len(inv_freq) channels turned by positions * inv_freq."""
    half = len(inv_freq)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    at = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    a, b = x[..., at[0]], x[..., at[1]]
    y = np.array(x, np.float64)
    y[..., at[0]], y[..., at[1]] = a * c - b * s, b * c + a * s
    return y


class Pages:
    """Tables, lengths and counts of a cache, and the content of its pages as one number each
    place; the rules one after the other, over Python lists."""

    def __init__(self, tables, lengths, refs, page, pools):
        self.tables, self.lengths, self.refs = [list(r) for r in tables], list(lengths), list(refs)
        self.page, self.pools = page, [np.array(p) for p in pools]

    def count(self, tokens):
        return -(-tokens // self.page)

    def _free(self):
        return [p for p, n in enumerate(self.refs) if n == 0]

    def copy(self, src, dst):
        for p in self.pools:
            p[:, dst] = p[:, src]

    def reserve(self, grow):
        free, used, out = self._free(), 0, []
        for r, more in enumerate(grow):
            have, want = self.count(self.lengths[r]), self.count(self.lengths[r] + more)
            if more < 0 or want > len(self.tables[r]):
                out.append(-1)
                continue
            used += want - have
            if want > have and used > len(free):
                out.append(-2)
                continue
            for c in range(have, want):
                self.tables[r][c] = free[used - want + c]
                self.refs[self.tables[r][c]] = 1
            self.lengths[r] += more
            out.append(want - have)
        return out

    def fork(self, parents):
        free, used, out, lengths = self._free(), 0, [], list(self.lengths)
        for r, parent in enumerate(parents):
            if parent < 0:
                out.append(0)
                continue
            if parent >= len(parents) or lengths[r] or parents[parent] >= 0:
                out.append(-1)
                continue
            n = lengths[parent]
            part = int(n % self.page != 0)
            used += part
            if part and used > len(free):
                out.append(-2)
                continue
            row = self.tables[parent][:self.count(n)]
            if part:
                self.copy(row[-1], free[used - 1])
                row[-1] = free[used - 1]
            for p in row:
                self.refs[p] += 1
            self.tables[r][:len(row)] = row
            self.lengths[r] = n
            out.append(part)
        return out

    def free(self, drop):
        for r, d in enumerate(drop):
            if d:
                for p in self.tables[r][:self.count(self.lengths[r])]:
                    self.refs[p] -= 1
                self.lengths[r] = 0

    def compact(self):
        n = sum(c > 0 for c in self.refs)
        holes = [p for p in range(n) if self.refs[p] <= 0]
        moves = dict(zip([p for p in range(n, len(self.refs)) if self.refs[p] > 0], holes))
        for r, row in enumerate(self.tables):
            held = self.count(self.lengths[r])
            row[:held] = [moves.get(p, p) for p in row[:held]]
        for src, dst in moves.items():
            self.refs[dst], self.refs[src] = self.refs[src], 0
            self.copy(src, dst)
        return n
