"""FP64 oracle of attention for several tokens a sequence, from its definitions (no code
shared with the library): one head at a time, all scores of a sequence at once.

Beside each result stand the sizes that error bounds use.
"""
from __future__ import annotations

import numpy as np


class Rows:
    """One head: queries q [m, D] over keys k, v [L, D]; query i sees the first seen[i] keys."""

    def __init__(self, q, k, v, seen, scale):
        self.q, self.k, self.v, self.scale = q, k, v, scale
        live = np.arange(len(k)) < np.asarray(seen)[:, None]
        self.s = np.where(live, scale * (q @ k.T), -np.inf)
        self.reach = np.where(live, abs(scale) * (np.abs(q) @ np.abs(k).T), 0.0)
        top = self.s.max(1, initial=-np.inf)[:, None]
        e = np.exp(self.s - np.where(np.isfinite(top), top, 0.0))
        total = e.sum(1, keepdims=True)
        self.p = e / np.where(total == 0, 1.0, total)
        with np.errstate(divide="ignore"):
            self.lse = (np.where(np.isfinite(top), top, 0.0) + np.log(total))[:, 0]
        self.out = self.p @ v
        self.mass = self.p @ np.abs(v)                 # the weighted mean of |v|

    def grads(self, dout):
        """(dq, dk, dv, ds)."""
        delta = (dout * self.out).sum(1, keepdims=True)
        ds = self.p * (dout @ self.v.T - delta)
        return self.scale * (ds @ self.k), self.scale * (ds.T @ self.q), self.p.T @ dout, ds


def spans(cu):
    return [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def packed(q, k, v, cu, scale):
    """{(sequence, query head): Rows} of causal attention over packed sequences."""
    G = q.shape[1] // k.shape[1]
    return {(n, h): Rows(q[a:b, h], k[a:b, h // G], v[a:b, h // G], np.arange(b - a) + 1, scale)
            for n, (a, b) in enumerate(spans(cu)) for h in range(q.shape[1])}


def pages(cache, row, length, h):
    """A request's first `length` keys or values of head h."""
    P = cache.shape[2]
    ids = row[:-(-length // P)]
    return np.concatenate([cache[p, h] for p in ids] or [cache[:0, h].reshape(0, cache.shape[3])])[:length]


def paged_prompt(q, k_cache, v_cache, table, seq_lens, cu, scale):
    """{(request, query head): Rows}: a request's queries are its last tokens."""
    G = q.shape[1] // k_cache.shape[1]
    out = {}
    for n, (a, b) in enumerate(spans(cu)):
        L = int(seq_lens[n])
        for h in range(q.shape[1]):
            k, v = (pages(c, table[n], L, h // G) for c in (k_cache, v_cache))
            out[n, h] = Rows(q[a:b, h], k, v, L - (b - a) + 1 + np.arange(b - a), scale)
    return out


def decode_shared(q, k_cache, v_cache, prefix_table, prefix_lens, cu_groups, table, seq_lens, scale):
    """{(request, query head): Rows}: the group's prefix, then the request's own tokens."""
    G = q.shape[1] // k_cache.shape[1]
    out = {}
    for g, (a, b) in enumerate(spans(cu_groups)):
        for n in range(a, b):
            for h in range(q.shape[1]):
                k, v = (np.concatenate([pages(c, prefix_table[g], int(prefix_lens[g]), h // G),
                                        pages(c, table[n], int(seq_lens[n]), h // G)])
                        for c in (k_cache, v_cache))
                out[n, h] = Rows(q[n:n + 1, h], k, v, [len(k)], scale)
    return out
