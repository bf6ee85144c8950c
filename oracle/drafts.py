"""Drafted tokens of the hybrid model: conv, delta rule, commit, verification, pages (oracle).

TEST INFRASTRUCTURE (see the package header).

Everything in float64 from the given values, one token after another.  ``delta``
and ``commit`` also return what a result may be off by per unit of relative
rounding error: the same recurrence over absolute values.
"""
from __future__ import annotations

import numpy as np


def parents(n, words=None):
    """Parent of each of a sequence's n tokens (-1: none): the highest bit below i of its mask word."""
    if words is None:
        return [i - 1 for i in range(n)]
    return [(int(words[i]) & ((1 << i) - 1)).bit_length() - 1 for i in range(n)]


def path(up, i):
    """The tokens from the root to i."""
    out = []
    while i >= 0:
        out.insert(0, i)
        i = up[i]
    return out


def conv(x, tail, up, w, n_qk, d, q_heads, eps, q_scale):
    """y [n][channels] of raw inputs x [n][channels], the conv state tail [channels][3] (oldest first) and taps w
    [channels][4]; and the sums of |w x| that its rounding errors are proportional to, through the same norm."""
    y, spread = np.zeros(x.shape), np.zeros(x.shape)
    for i in range(len(x)):
        taps = [x[j] for j in path(up, i)][-4:]
        taps = [tail[:, 3 - (4 - len(taps)) + k] for k in range(4 - len(taps))] + taps
        t = np.stack(taps, axis=1).astype(np.float64)
        u = (t * w).sum(axis=1)
        y[i] = u / (1 + np.exp(-u))
        spread[i] = (np.abs(t) * np.abs(w)).sum(axis=1)
        for h in range(n_qk):
            c = slice(h * d, (h + 1) * d)
            f = (q_scale if h < q_heads else 1.0) / np.sqrt((y[i, c] ** 2).sum() + eps)
            y[i, c] *= f
            spread[i, c] *= abs(f)
    return y, spread


def gates(beta, alpha, A_log, dt_bias):
    u = alpha.astype(np.float64) + dt_bias
    return -np.exp(A_log.astype(np.float64)) * np.logaddexp(0, u), 1 / (1 + np.exp(-beta.astype(np.float64)))


def delta(q, k, v, log_a, b, state, up):
    """One value head: q, k, v [n][d], log_a, b [n], state [dv][dk].  u, o [n][d] and their sums of absolute values."""
    n, d = q.shape
    u, o, eu, eo = (np.zeros((n, d)) for _ in range(4))
    states, spread = [], []
    for i in range(n):
        prev = (states[up[i]] if up[i] >= 0 else state) * np.exp(log_a[i])
        err = (spread[up[i]] if up[i] >= 0 else np.abs(state)) * np.exp(log_a[i])
        u[i] = b[i] * (v[i] - prev @ k[i])
        eu[i] = abs(b[i]) * (np.abs(v[i]) + err @ np.abs(k[i]))
        states.append(prev + np.outer(u[i], k[i]))
        spread.append(err + np.outer(eu[i], np.abs(k[i])))
        o[i] = states[-1] @ q[i]
        eo[i] = spread[-1] @ np.abs(q[i])
    return u, o, eu, eo


def commit(k, u, log_a, state, up, node):
    """The state after token node of one value head, and its sum of absolute values."""
    s, e = state.astype(np.float64), np.abs(state.astype(np.float64))
    for i in path(up, node):
        a = np.exp(log_a[i])
        s, e = a * s + np.outer(u[i], k[i]), a * e + np.outer(np.abs(u[i]), np.abs(k[i]))
    return s, e


def conv_commit(x, tail, up, node):
    taps = [x[j] for j in path(up, node)][-3:]
    return np.stack([tail[:, len(taps) + i] for i in range(3 - len(taps))] + taps, axis=1)


def _probabilities(x):
    return np.clip(np.nan_to_num(x.astype(np.float64), nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)


def _best(row):
    row = np.where(np.isnan(row), -np.inf, row.astype(np.float64))
    first = np.flatnonzero(row == row.max())
    return int(first[0])


def verify(p, q, tokens, up, u, u_next):
    """One sequence: p, q [n][vocab] (q None: certain drafts; u None: greedy).  Accepted tokens, ids, next."""
    if not up:
        return [], [], -1
    greedy, here, keep, ids = u is None, 0, [0], []
    row = lambda i: p[i] if greedy else _probabilities(p[i])  # noqa: E731
    r = row(0)
    for i in range(1, len(up)):
        if up[i] != here:
            continue
        x = int(tokens[i])
        if greedy:
            ok = x == _best(r)
        elif not 0 <= x < p.shape[1]:
            ok = False
        else:
            ok = float(u[i]) * (float(_probabilities(q[here, x:x + 1])[0]) if q is not None else 1.0) < r[x]
        if ok:
            here, r = i, row(i)
            keep.append(i)
            ids.append(x)
        elif not greedy:
            if q is not None:
                r = np.maximum(r - _probabilities(q[here]), 0.0)
            else:
                r = r.copy()
                if 0 <= x < p.shape[1]:
                    r[x] = 0.0
            r = r / r.sum() if r.sum() > 0 else r
    if greedy:
        nxt = _best(r)
    else:
        r = r if r.sum() > 0 else row(here)
        total = np.cumsum(r)
        hit = np.flatnonzero(total > float(u_next) * total[-1])
        nxt = int(hit[0]) if len(hit) else -1
    return keep, ids + [nxt], nxt


class Pages:
    """Block table, pages held and the stack of free pages, as lists."""

    def __init__(self, table, held, stack, page):
        self.table, self.held, self.stack, self.page = [list(r) for r in table], list(held), list(stack), page

    def trim(self, keep):
        back = []
        for s, n in enumerate(keep):
            k = min(self.held[s], -(-n // self.page))
            back += self.table[s][k:self.held[s]]
            self.held[s] = k
        self.stack += back[::-1]

    def extend(self, lens, new, depth=None):
        """Lengths after, offsets, positions and slots of the new tokens; depth: per sequence, of its tree's tokens."""
        after, cu, positions, slots, asked, free = [], [0], [], [], 0, len(self.stack)
        for s, (n, m) in enumerate(zip(lens, new)):
            need = max(0, -(-(n + m) // self.page) - self.held[s])
            asked += need
            ok = need == 0 or asked <= free
            for _ in range(need if ok else 0):
                self.table[s][self.held[s]] = self.stack.pop()
                self.held[s] += 1
            positions += [n + (i if depth is None else depth[s][i]) for i in range(m)]
            slots += [self.table[s][(n + i) // self.page] * self.page + (n + i) % self.page if ok else -1 for i in range(m)]
            after.append(n + m if ok else n)
            cu.append(cu[-1] + m)
        return after, cu, positions, slots
