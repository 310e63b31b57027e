"""Plain statements of the operators of include/pace_serve.h in 64 bits, written from the header and sharing no code with the CUDA
path."""
from __future__ import annotations

import numpy as np


# ---- the gated delta rule: one sequence and head ---------------------------------------------------------------------------------
def rule(S, k, v, a, beta):
    S = a * S
    return S + np.outer(k, beta * (v - k @ S))


def chunk(S, q, k, v, a, beta):
    """Outputs and last state of tokens [n, d] from S [d, d]."""
    o = np.zeros_like(v)
    for t in range(len(v)):
        S = rule(S, k[t], v[t], a[t], beta[t])
        o[t] = q[t] @ S
    return o, S


def draft(S, q, k, v, a, beta, see):
    """Outputs of a tree: token t after its ancestors see[t] (booleans), in order."""
    o = np.zeros_like(v)
    for t in range(len(v)):
        X = S
        for s in range(t + 1):
            if s == t or see[t, s]:
                X = rule(X, k[s], v[s], a[s], beta[s])
        o[t] = q[t] @ X
    return o


# ---- verification: one sequence --------------------------------------------------------------------------------------------------
def verify(tokens, p, q, u, parents):
    """Kept nodes and the next token. p, q [N, V] (q None), parents [N]."""
    clean = lambda x: np.clip(np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)
    N, V = p.shape
    node, path = 0, [0]
    R, Z = clean(p[0]), 1.0
    for i in range(1, N):
        if parents[i] != node:
            continue
        y = tokens[i]
        if not 0 <= y < V:
            continue
        draw = clean(q[node]) if q is not None else None
        if float(u[i]) * (1.0 if draw is None else draw[y]) * Z < R[y]:
            node, R, Z = i, clean(p[i]), 1.0
            path.append(i)
        elif draw is None:
            Z = max(Z - R[y], 0.0)
            R = R.copy()
            R[y] = 0.0
        else:
            R = np.maximum(R - draw * Z, 0.0)
            Z = R.sum()
    if R.sum() < 2.0 ** -46:
        R = clean(p[node])
    if R.sum() < 2.0 ** -46:
        return path, -1
    cum = np.cumsum(R)
    return path, int(np.argmax(cum > float(u[0]) * cum[-1]))


# ---- pages -------------------------------------------------------------------------------------------------------------------------
class Pages:
    def __init__(self, n_pages, page, table, lens, refs):
        self.n, self.page = n_pages, page
        self.table, self.lens, self.refs = np.array(table), np.array(lens), np.array(refs)
        self.moves = []

    def cover(self, tokens):
        return -(-int(tokens) // self.page)

    def select(self, src=None):
        old, lens = self.table.copy(), self.lens.copy()
        for b in range(len(old)):
            f = b if src is None else int(src[b])
            f = b if f < -1 or f >= len(old) else f
            self.lens[b] = lens[f] if f >= 0 else 0
            for c in range(old.shape[1]):
                x = old[f, c] if f >= 0 and c < self.cover(lens[f]) else -1
                x = x if 0 <= x < self.n else -1
                if 0 <= old[b, c] < self.n:
                    self.refs[old[b, c]] -= 1
                if x >= 0:
                    self.refs[x] += 1
                self.table[b, c] = x

    def take(self, n_new):
        B, C = self.table.shape
        wants, copies, bad = [[] for _ in range(B)], [False] * B, [False] * B
        writers = {}
        for b in range(B):
            n, m = int(self.lens[b]), max(int(n_new[b]), 0)
            if m == 0:
                continue
            if n < 0 or n + m > C * self.page:
                bad[b] = True
                continue
            x = self.table[b, self.cover(n) - 1] if n % self.page else None
            cells = self.table[b, self.cover(n):self.cover(n + m)]
            if (x is not None and (not 0 <= x < self.n or self.refs[x] < 1)) or any(c < -1 or c >= self.n for c in cells):
                bad[b] = True
                continue
            wants[b] = [c for c in range(self.cover(n), self.cover(n + m)) if self.table[b, c] < 0]
            if x is not None and self.refs[x] > 1:
                writers.setdefault(int(x), []).append(b)
        for x, rows in writers.items():
            keeper = max(rows, key=lambda b: (int(self.lens[b]) % self.page, -b))       # (writes behind every other holder's tokens)
            for b in rows:
                if not (len(rows) == self.refs[x] and b == keeper):
                    copies[b] = True
                    wants[b].insert(0, self.cover(self.lens[b]) - 1)
        free = [x for x in range(self.n) if self.refs[x] == 0]
        fits, used, self.moves = [], 0, []
        drop = []
        for b in range(B):
            used += len(wants[b])
            fits.append(not bad[b] and (used <= len(free) or not wants[b]))
            if fits[b] and wants[b]:
                for c, x in zip(wants[b], free[used - len(wants[b]):]):
                    if copies[b] and c == wants[b][0]:
                        self.moves.append((int(self.table[b, c]), x))
                        drop.append(int(self.table[b, c]))
                    self.table[b, c] = x
                    self.refs[x] = 1
        for x in drop:
            self.refs[x] -= 1
        return np.array(fits, int), bad

    def compact(self):
        used = [x for x in range(self.n) if self.refs[x]]
        top = len(used)
        self.moves = list(zip([x for x in used if x >= top], [x for x in range(top) if not self.refs[x]]))
        to = dict(self.moves)
        for s, d in self.moves:
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.table = np.array([[to.get(int(x), int(x)) for x in row] for row in self.table]).reshape(self.table.shape)
