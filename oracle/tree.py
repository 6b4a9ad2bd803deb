"""Oracle of the tree-verification operators (test infrastructure only):
attention of drafted tokens over a Q8_0 cache, the acceptance walk, and the
page bookkeeping, written one sequence, token and page at a time in float64
and plain Python integers."""
from __future__ import annotations

import numpy as np


def ancestors(parent) -> list[int]:
    """Mask words of a tree: bit j of word i is set when j is i or an ancestor of i."""
    out = []
    for i, p in enumerate(parent):
        out.append((out[p] if 0 <= p < i else 0) | 1 << i)
    return out


def tree_attention_f64(q, K, V, length, masks, scale):
    """One query head: q [n, D], K, V [length + n, D] (cache values), masks n
    words -> out [n, D], wabs [n, D] = sum w |v| / sum w, smag [n] = the
    largest scale * sum |q k| over the positions that a token sees."""
    n, D = q.shape
    out, wabs, smag = np.zeros((n, D)), np.zeros((n, D)), np.zeros(n)
    for i in range(n):
        see = [j for j in range(length + n) if j < length or masks[i] >> (j - length) & 1]
        if not see:
            continue
        k, v = K[see].astype(np.float64), V[see].astype(np.float64)
        s = scale * (k @ q[i].astype(np.float64))
        w = np.exp(s - s.max())
        w /= w.sum()
        out[i], wabs[i] = w @ v, w @ np.abs(v)
        smag[i] = scale * (np.abs(k) @ np.abs(q[i].astype(np.float64))).max()
    return out, wabs, smag


def verify_tree(logits, tokens, parent, u, draft=None, temperature=1.0):
    """One sequence: logits [n, V]; returns (path, next_token, lse [n])."""
    l64 = np.asarray(logits, np.float64)
    n, vocab = l64.shape
    T = temperature if temperature > 0 else 1.0
    top = l64.max(1)
    lse = top / T + np.log(np.exp((l64 - top[:, None]) / T).sum(1))
    if n == 0:
        return [], -1, lse
    cur, path = 0, [0]
    w = np.exp((l64[0] - top[0]) / T)
    r, R, S = w, w.sum(), 0.0
    for i in range(1, n):
        if parent[i] != cur:
            continue
        x = int(tokens[i])
        if temperature == 0:
            yes = x == int(np.argmax(l64[cur]))
        elif not 0 <= x < vocab:
            yes = False
        else:
            q = 1.0 if draft is None else float(draft[cur][x])
            yes = float(u[i]) * q * R < r[x]
        if yes:
            cur = i
            path.append(i)
            w = np.exp((l64[i] - top[i]) / T)
            r, R, S = w, w.sum(), 0.0
        elif temperature > 0 and draft is not None:
            less = np.maximum(w - (S + R) * np.asarray(draft[cur], np.float64), 0)
            if less.sum() > 0:
                S, r, R = S + R, less, less.sum()
        elif temperature > 0 and 0 <= x < vocab:
            r = r.copy()
            r[x] = 0.0
            R = r.sum()
    upto = np.cumsum(r)
    if temperature == 0 or upto[-1] <= 0:
        return path, int(np.argmax(l64[cur])), lse
    return path, int(np.argmax(upto > float(u[0]) * upto[-1])), lse


class Pages:
    """The page bookkeeping: table (lists of ids), length, refs, and the rows
    as a dictionary (page, slot) -> value."""

    def __init__(self, n_pages, n_seq, max_pages, page_size):
        self.P, self.max_pages = page_size, max_pages
        self.table = [[] for _ in range(n_seq)]
        self.length = [0] * n_seq
        self.refs = [0] * n_pages
        self.rows = {}

    def truncate(self, new_length):
        for s, n in enumerate(new_length):
            if n < 0:
                continue
            self.length[s] = min(self.length[s], n)
            keep = -(-self.length[s] // self.P)
            for page in self.table[s][keep:]:
                self.refs[page] -= 1
            del self.table[s][keep:]

    def fork(self, src, dst):
        status = []
        for i, (a, b) in enumerate(zip(src, dst)):
            n = len(self.table)
            if not (0 <= a < n and 0 <= b < n) or a == b or a in dst or b in dst[:i] or self.table[b] or self.length[b]:
                status.append(1)
                continue
            status.append(0)
            self.length[b] = self.length[a]
            self.table[b] = self.table[a][: -(-self.length[a] // self.P)]
            for page in self.table[b]:
                self.refs[page] += 1
        return status

    def reserve(self, extra):
        status, full = [], False
        for s, n in enumerate(extra):
            if n <= 0:
                status.append(0)
                continue
            first, last = self.length[s] // self.P, -(-(self.length[s] + n) // self.P)
            if last > self.max_pages:
                status.append(2)
                continue
            row = self.table[s]
            copy = self.length[s] % self.P > 0 and self.refs[row[first]] > 1
            need = max(0, last - len(row)) + copy
            free = [p for p, c in enumerate(self.refs) if c == 0]
            full = full or need > len(free)
            status.append(1 if full else 0)
            if full:
                continue
            if copy:
                old, row[first] = row[first], free.pop(0)
                self.refs[old] -= 1
                self.refs[row[first]] = 1
                for slot in range(self.length[s] % self.P):
                    self.rows[row[first], slot] = self.rows.get((old, slot))
            while len(row) < last:
                row.append(free.pop(0))
                self.refs[row[-1]] = 1
        return status

    def compact(self, path, n_keep):
        for s, n in enumerate(n_keep):
            at = lambda pos: (self.table[s][pos // self.P], pos % self.P)  # noqa: E731
            n = min(max(n, 0), len(path[s]))
            moved = {}
            for i in range(n):
                if i < path[s][i] < len(path[s]):
                    moved[at(self.length[s] + i)] = self.rows.get(at(self.length[s] + path[s][i]))
            self.rows.update(moved)
            self.length[s] += n


def sum_bound(T: int) -> float:
    """Relative rounding bound of a float32 sum over T positions that no more
    than T/4 of its terms pass through one accumulator (half a unit, 2^-24,
    an addition), with 32 more for the products, the split of an operand into
    two fp16 parts (2^-22) and the joins."""
    return (32 + T / 4) * 2.0 ** -24


def attention_bound(wabs, smag, T, D):
    """Error bound of tree_attention_f64's out: scores off by ds change every
    weight by a factor within exp(+-2 ds); ds counts D/4 additions of a dot
    product, 32 for the rest, relative to the sum of magnitudes."""
    ds = (32 + D / 4) * 2.0 ** -24 * smag
    return wabs * (np.expm1(2 * ds)[..., None] + 2 * sum_bound(T)) + 1e-30


