"""fp64 statements of the ragged-batch operators (numpy, straight loops over sequences and
heads): attention over packed prompts, K/V pages, attention of one new token over them,
linear attention with a decay per head. Shares no code with the CUDA path.

Each returns, next to the result, the sum of the absolute values of its terms, from which
the tests derive their rounding bounds.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np

from .hymba_oracle import gqa_group, visibility_mask


def _attend(q, k, v, see, scale):
    """One head: rows q [n, dh] over keys k [m, dh], values v [m, dv], see [n, m] -> the
    output, sum_j w_ij |v_j|, and the largest scale |q_i| . |k_j| a row sees."""
    x = scale * (q @ k.T)
    x = np.where(see, x, -np.inf)
    top = x.max(axis=1, initial=-np.inf, keepdims=True)
    p = np.where(see, np.exp(x - np.where(np.isfinite(top), top, 0.0)), 0.0)
    l = p.sum(axis=1, keepdims=True)
    w = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
    big = np.where(see, scale * (np.abs(q) @ np.abs(k).T), 0.0).max(axis=1, initial=0.0)
    return w @ v, w @ np.abs(v), big


def packed_attention(q, k, v, cu: Sequence[int], H: int, G: int, n_meta: int, window: int, scale: float):
    """q [rows, H*dh], k [rows, G*dh], v [rows, G*dv] -> (o, abs, big) for the rows of the
    sequences cu[s] .. cu[s+1] - 1; other rows 0. abs like o; big [rows, H]."""
    rows, dh, dv = q.shape[0], q.shape[1] // H, v.shape[1] // G
    o, a, big = np.zeros((rows, H * dv)), np.zeros((rows, H * dv)), np.zeros((rows, H))
    for lo, hi in zip(cu[:-1], cu[1:]):
        pos = np.arange(hi - lo)
        see = visibility_mask(pos, pos, n_meta, window)
        for h in range(H):
            g = gqa_group(h, H, G)
            c = slice(h * dv, (h + 1) * dv)
            o[lo:hi, c], a[lo:hi, c], big[lo:hi, h] = _attend(
                q[lo:hi, h * dh:(h + 1) * dh], k[lo:hi, g * dh:(g + 1) * dh], v[lo:hi, g * dv:(g + 1) * dv], see, scale)
    return o, a, big


def append_pages(k_pages, v_pages, table, length, k, v, cu: Optional[Sequence[int]]):
    """Copies of the pages with each sequence's rows as its newest positions."""
    k_pages, v_pages = k_pages.copy(), v_pages.copy()
    G, page = k_pages.shape[1], k_pages.shape[2]
    if cu is None:
        cu = list(range(len(length) + 1))
    for b in range(len(length)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            p = int(length[b]) - n + i
            at = table[b][p // page]
            k_pages[at, :, p % page] = k[cu[b] + i].reshape(G, -1)
            v_pages[at, :, p % page] = v[cu[b] + i].reshape(G, -1)
    return k_pages, v_pages


def paged_attention(q, k_pages, v_pages, table, length, H: int, n_meta: int, window: int, scale: float):
    """One query per sequence at position length[b] - 1 over its pages -> (o, abs, big)."""
    G, page, dh = k_pages.shape[1:]
    dv, B = v_pages.shape[3], len(length)
    o, a, big = np.zeros((B, H * dv)), np.zeros((B, H * dv)), np.zeros((B, H))
    for b in range(B):
        n = int(length[b])
        if n == 0:
            continue
        pos = np.arange(n)
        see = visibility_mask(np.array([n - 1]), pos, n_meta, window)
        pos, see = pos[see[0]], see[:, see[0]]
        at = np.asarray(table[b])[pos // page]
        for h in range(H):
            g = gqa_group(h, H, G)
            c = slice(h * dv, (h + 1) * dv)
            o[b, c], a[b, c], big[b, h] = [x[0] for x in _attend(
                q[b:b + 1, h * dh:(h + 1) * dh], k_pages[at, g, pos % page], v_pages[at, g, pos % page], see, scale)]
    return o, a, big


def linear_attention(q, k, v, g, cu: Sequence[int], Hk: int, H: int, scale: float, state=None):
    """S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t per sequence and head; state
    [n, H, dv, dk] before the first row (None: zero). Returns (o, abs of o, end, abs of end)."""
    rows, dk, dv, n = q.shape[0], q.shape[1] // Hk, v.shape[1] // H, len(cu) - 1
    o, oa = np.zeros((rows, H * dv)), np.zeros((rows, H * dv))
    end = np.zeros((n, H, dv, dk)) if state is None else np.array(state, dtype=np.float64)
    enda = np.abs(end)
    for s in range(n):
        for t in range(cu[s], cu[s + 1]):
            for h in range(H):
                hk = h // (H // Hk)
                kt, qt, vt = k[t, hk * dk:(hk + 1) * dk], q[t, hk * dk:(hk + 1) * dk], v[t, h * dv:(h + 1) * dv]
                d = math.exp(g[t, h])
                # a decay of 0 forgets what the state held, whatever it was
                end[s, h] = (d * end[s, h] if d else 0.0) + np.outer(vt, kt)
                enda[s, h] = (d * enda[s, h] if d else 0.0) + np.abs(np.outer(vt, kt))
                o[t, h * dv:(h + 1) * dv] = scale * (end[s, h] @ qt)
                oa[t, h * dv:(h + 1) * dv] = scale * (enda[s, h] @ np.abs(qt))
    return o, oa, end, enda


def linear_attention_masked(q, k, v, g, scale: float):
    """The same for one sequence and head in the closed form o = (Q K^T * L) V with the
    decay mask L_ij = exp(g_{j+1} + .. + g_i) for j <= i ("Lecture 04", section 3)."""
    n = q.shape[0]
    L = np.zeros((n, n))
    for i in range(n):
        for j in range(i + 1):
            L[i, j] = math.exp(g[j + 1:i + 1].sum())
    return scale * ((q @ k.T) * L) @ v
