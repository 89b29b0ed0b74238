"""FP64 oracle of the paged-attention operators, from their definitions, in plain
loops (no code shared with the library)."""
from __future__ import annotations

import math

import numpy as np


def page_plan(cached, cu, T, table, free, page, start=0):
    """(table, seq_lens, positions, slots, free_end, error) of kda_page_plan; error is
    None, "arg" or "pages"."""
    table = np.array(table, dtype=np.int64).copy()
    N, M = table.shape
    cached, cu = [int(x) for x in cached], [int(x) for x in cu]
    bad = N == 0 and T > 0
    for n in range(N):
        bad = bad or cached[n] < 0 or not 0 <= cu[n] <= cu[n + 1] <= T
        bad = bad or cached[n] + cu[n + 1] - cu[n] >= 2 ** 31
    bad = bad or (N > 0 and (cu[0] != 0 or cu[N] != T))
    positions, slots = np.zeros(T, np.int64), np.full(T, -1, np.int64)
    if bad:
        return table, np.array(cached, np.int64), positions, slots, start, "arg"
    error, at, dry = None, start, False
    lens = []
    for n in range(N):
        new = cu[n + 1] - cu[n]
        have, want = -(-cached[n] // page), -(-(cached[n] + new) // page)
        ok = want <= M
        if ok and want > have:
            dry = dry or at + want - have > len(free)
            ok = not dry
        if ok:
            for j in range(have, want):
                table[n, j] = free[at]
                at += 1
        else:
            error = "pages"
        lens.append(cached[n] + (new if ok else 0))
        for t in range(cu[n], cu[n + 1]):
            positions[t] = cached[n] + t - cu[n]
            if ok:
                slots[t] = table[n, positions[t] // page] * page + positions[t] % page
    return table, np.array(lens, np.int64), positions, slots, at, error


def rotation(rot, D, position, inv_freq, interleaved, scale):
    """The D x D matrix that turns a head's channels at `position`."""
    R = np.eye(D)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        angle = float(position) * float(inv_freq[i])
        c, s = math.cos(angle) * scale, math.sin(angle) * scale
        R[a, a], R[a, b], R[b, a], R[b, b] = c, -s, s, c
    return R


def norm_rope(x, positions, inv_freq, weight, eps, norm, interleaved, scale):
    """y [T, H, D] from x [T, H, D]; every argument in FP64."""
    T, H, D = x.shape
    y = np.empty_like(x)
    for t in range(T):
        R = rotation(2 * len(inv_freq), D, positions[t], inv_freq, interleaved, scale)
        for h in range(H):
            n = x[t, h]
            if norm:
                n = n / math.sqrt(np.dot(n, n) / D + eps) * weight
            y[t, h] = R @ n
    return y


def norm_rope_grad(x, dy, positions, inv_freq, weight, eps, norm, interleaved, scale):
    """(dx, dweight) of norm_rope: the chain rule with the norm's Jacobian written out,
    J = diag(w) (I / r - x x^T / (D r^3)), r = sqrt(mean x^2 + eps)."""
    T, H, D = x.shape
    dx, dw = np.empty_like(x), np.zeros(D)
    for t in range(T):
        R = rotation(2 * len(inv_freq), D, positions[t], inv_freq, interleaved, scale)
        for h in range(H):
            d = R.T @ dy[t, h]
            if norm:
                r = math.sqrt(np.dot(x[t, h], x[t, h]) / D + eps)
                dw += d * x[t, h] / r
                J = np.eye(D) / r - np.outer(x[t, h], x[t, h]) / (D * r ** 3)
                d = J.T @ (weight * d)
            dx[t, h] = d
    return dx, dw


def paged_decode(q, k_cache, v_cache, table, seq_lens, scale):
    """(out [N, Hq, D], lse [N, Hq], mass [N, Hq, D], reach [N, Hq]): mass = the weighted
    mean of |v| and reach = the largest scale * sum |q_i k_i|, which error bounds use."""
    N, Hq, D = q.shape
    Hk, P = k_cache.shape[1:3]
    out, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    mass, reach = np.zeros((N, Hq, D)), np.zeros((N, Hq))
    for n in range(N):
        L = int(seq_lens[n])
        if L == 0:
            continue
        pages = table[n][:-(-L // P)]
        for h in range(Hq):
            hk = h // (Hq // Hk)
            k = np.concatenate([k_cache[p, hk] for p in pages])[:L]
            v = np.concatenate([v_cache[p, hk] for p in pages])[:L]
            s = scale * (k @ q[n, h])
            e = np.exp(s - s.max())
            out[n, h] = e @ v / e.sum()
            lse[n, h] = s.max() + math.log(e.sum())
            mass[n, h] = e @ np.abs(v) / e.sum()
            reach[n, h] = np.max(abs(scale) * (np.abs(k) @ np.abs(q[n, h])))
    return out, lse, mass, reach
