"""fp64 definitions of draft-tree attention, the attention weight of cached rows, and the rows
that move when nodes are accepted or context rows leave.  Test infrastructure only, like
``mla_oracle``: the plain definitions, one node and one row at a time.

A window is (first, rows, nodes): logical row j of a sequence is ring slot (first + j) mod S, the
context is j < rows, node i is row rows + i.
"""

from __future__ import annotations

import math
from typing import List, Sequence, Tuple

import numpy as np

from . import mla_oracle as O


def clip_window(window: Sequence[int], S: int, n_nodes: int) -> Tuple[int, int, int]:
    first, rows, nodes = (int(v) for v in window)
    first = min(max(first, 0), S - 1)
    rows = min(max(rows, 0), S)
    return first, rows, min(max(nodes, 0), n_nodes, S - rows)


def slots(first: int, count: int, S: int) -> List[int]:
    return [(first + j) % S for j in range(count)]


def sees(tree, i: int, k: int) -> bool:
    """Whether node i sees node k; no tree: a chain."""
    return k <= i if tree is None else bool(tree[i][k])


def visible(tree, i: int, rows: int, nodes: int) -> List[int]:
    return list(range(rows)) + [rows + k for k in range(nodes) if sees(tree, i, k)]


def tree_write(cache, position, h, w_dkv, w_kr, window, token, wl):
    """Cache and positions after the nodes of every sequence are written."""
    cache, position = cache.copy(), position.copy()
    B, n = token.shape
    S = cache.shape[1]
    for b in range(B):
        first, rows, nodes = clip_window(window[b], S, n)
        for i in range(nodes):
            s = (first + rows + i) % S
            g = int(token[b, i])
            cache[b, s] = O.cache_rows(h[b:b + 1, i:i + 1], w_dkv, w_kr, g, wl)[0, 0]
            position[b, s] = g
    return cache, position


def tree_absorb_q(q_nope, q_rope, w_uk, token, wl):
    B, n = token.shape
    out = np.zeros(q_nope.shape[:3] + (w_uk.shape[2] + q_rope.shape[3],))
    for b in range(B):
        for i in range(n):
            out[b, i] = O.absorb_q(q_nope[b:b + 1, i:i + 1], q_rope[b:b + 1, i:i + 1], w_uk,
                                   int(token[b, i]), wl)[0, 0]
    return out


def attend_tree(q_abs, cache, window, tree, scale, d_latent):
    """(o_lat, lse, spread): spread = sum_j p_j |c_j|, the size that rounding errors of the
    softmax weights have in the output.  Rows past a sequence's nodes stay NaN."""
    B, n, H, _ = q_abs.shape
    S = cache.shape[1]
    o = np.full((B, n, H, d_latent), np.nan)
    lse = np.full((B, n, H), np.nan)
    spread = np.full((B, n, H, d_latent), np.nan)
    for b in range(B):
        first, rows, nodes = clip_window(window[b], S, n)
        at = slots(first, rows + nodes, S)
        for i in range(nodes):
            js = visible(None if tree is None else tree[b], i, rows, nodes)
            if not js:
                o[b, i], lse[b, i], spread[b, i] = 0.0, -np.inf, 0.0
                continue
            k = cache[b][[at[j] for j in js]]
            s = scale * (q_abs[b, i] @ k.T)
            m = s.max(axis=1, keepdims=True)
            e = np.exp(s - m)
            t = e.sum(axis=1, keepdims=True)
            p = e / t
            o[b, i] = p @ k[:, :d_latent]
            spread[b, i] = p @ np.abs(k[:, :d_latent])
            lse[b, i] = (m + np.log(t))[:, 0]
    return o, lse, spread


def attend_weight(q_abs, cache, window, tree, scale, lse, query_weight, weight_in, weight_out):
    """weight_out after the call (slots outside the windows as given)."""
    out = weight_out.copy()
    B, n, H, _ = q_abs.shape
    S = cache.shape[1]
    for b in range(B):
        first, rows, nodes = clip_window(window[b], S, n)
        at = slots(first, rows + nodes, S)
        total = np.zeros(rows + nodes)
        for i in range(nodes):
            g = 1.0 if query_weight is None else float(query_weight[b, i])
            js = visible(None if tree is None else tree[b], i, rows, nodes)
            if not js or g == 0.0:
                continue
            s = scale * (q_abs[b, i] @ cache[b][[at[j] for j in js]].T)       # [H, visible]
            for h in range(H):
                if lse[b, i, h] != -np.inf:
                    total[js] += g * np.exp(s[h] - lse[b, i, h])
        for j in range(rows + nodes):
            w0 = weight_in[b, at[j]] if (weight_in is not None and j < rows) else 0.0
            out[b, at[j]] = w0 + total[j]
    return out


def _move(arrays, b, kept: Sequence[bool], count: int, at: Sequence[int]):
    """Kept rows at index >= count into the holes below it, both ascending."""
    holes = [at[j] for j in range(count) if not kept[j]]
    late = [at[j] for j in range(count, len(kept)) if kept[j]]
    assert len(holes) == len(late)
    for d, s in zip(holes, late):
        for x in arrays:
            if x is not None:
                x[b, d] = x[b, s]


def tree_accept(cache, window, weight, position, accept):
    out = [None if x is None else x.copy() for x in (cache, weight, position)]
    window = window.copy()
    S, n = cache.shape[1], accept.shape[1]
    for b in range(cache.shape[0]):
        first, rows, nodes = clip_window(window[b], S, n)
        at = slots((first + rows) % S, nodes, S)
        kept = [bool(accept[b, i]) for i in range(nodes)]
        _move(out, b, kept, sum(kept), at)
        window[b] = (first, rows + sum(kept), 0)
    return out[0], window, out[1], out[2]


def cache_evict(cache, window, weight, position, n_keep, n_sink, n_recent):
    out = [x.copy() for x in (cache, weight, position)]
    window = window.copy()
    S = cache.shape[1]
    for b in range(cache.shape[0]):
        first, rows, _ = clip_window(window[b], S, S)
        window[b] = (first, min(rows, n_keep), 0)
        if rows <= n_keep:
            continue
        at = slots(first, rows, S)
        newest = max(int(position[b, s]) for s in at)

        def order(j):
            w, p = float(weight[b, at[j]]), int(position[b, at[j]])
            safe = p < n_sink or p > newest - n_recent
            # protected rows, then weights from the largest, NaN last; then the lower row
            return (0, 0.0, j) if safe else ((2, 0.0, j) if math.isnan(w) else (1, -w, j))

        stay = set(sorted(range(rows), key=order)[:n_keep])
        _move(out, b, [j in stay for j in range(rows)], n_keep, at)
    return out[0], window, out[1], out[2]
