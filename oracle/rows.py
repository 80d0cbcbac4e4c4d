"""fp64 oracle of the operators around packed attention: head norm and rotation, its
gradients, a paged key/value cache, and attention over it.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Plain loops over sequences and rows;
every function also returns (``with_size``) the size of the terms a value is summed from, from
which the tests derive their tolerances.
"""
from __future__ import annotations

import numpy as np

from .attention import _as64, sequence_spans


def rotation(d, rotary, interleaved, cos, sin):
    """The d x d matrix that turns a head by the angles of one position (rows of the tables)."""
    m = np.eye(d)
    for c in range(rotary // 2):
        i, j = (2 * c, 2 * c + 1) if interleaved else (c, c + rotary // 2)
        m[i, i], m[i, j] = cos[c], -sin[c]
        m[j, j], m[j, i] = cos[c], sin[c]
    return m


def row_places(cu_seqlens, cu_seqlens_padded, batch_size):
    """[(buffer row, sequence, place in it)] of every row of a sequence."""
    starts, lengths = sequence_spans(cu_seqlens, cu_seqlens_padded, batch_size)
    return [(int(s) + i, b, i) for b, (s, n) in enumerate(zip(starts, lengths)) for i in range(int(n))]


def _table_row(cos, sin, pos):
    if cos is None:
        return None, None
    at = min(max(pos, 0), len(cos) - 1)
    return cos[at], sin[at]


def norm_rope_row(x, weight, eps, cos, sin, interleaved):
    """Heads x [h, d] of one row, normed and turned; and the size of each value's terms."""
    n = x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    if cos is None:
        return n, np.abs(n)
    m = rotation(x.shape[-1], 2 * len(cos), interleaved, cos, sin)
    return n @ m.T, np.abs(n) @ np.abs(m).T


def norm_rope(x, weight, eps, cos, sin, interleaved, cu_seqlens, cu_seqlens_padded, batch_size, offsets=None):
    """x [T, h, d] -> (normed and turned rows, zeros elsewhere; size of the terms)."""
    x, weight = _as64(x), None if weight is None else _as64(weight)
    cos, sin = (None, None) if cos is None else (_as64(cos), _as64(sin))
    y, size = np.zeros_like(x), np.zeros_like(x)
    for t, b, i in row_places(cu_seqlens, cu_seqlens_padded, batch_size):
        c, s = _table_row(cos, sin, i + (0 if offsets is None else int(offsets[b])))
        y[t], size[t] = norm_rope_row(x[t], weight, eps, c, s, interleaved)
    return y, size


def norm_rope_bwd(g, x, weight, eps, cos, sin, interleaved, cu_seqlens, cu_seqlens_padded, batch_size, offsets=None):
    """(dx, size of its terms, dw or None, size of its terms) for gradients g of norm_rope's output."""
    g, x, weight = _as64(g), None if x is None else _as64(x), None if weight is None else _as64(weight)
    cos, sin = (None, None) if cos is None else (_as64(cos), _as64(sin))
    dx, size = np.zeros_like(g), np.zeros_like(g)
    d = g.shape[-1]
    dw, dw_size = np.zeros(d), np.zeros(d)
    for t, b, i in row_places(cu_seqlens, cu_seqlens_padded, batch_size):
        c, s = _table_row(cos, sin, i + (0 if offsets is None else int(offsets[b])))
        m = np.eye(d) if c is None else rotation(d, 2 * len(c), interleaved, c, s)
        h, hs = g[t] @ m, np.abs(g[t]) @ np.abs(m)
        if weight is None:
            dx[t], size[t] = h, hs
            continue
        r = 1.0 / np.sqrt((x[t] * x[t]).mean(-1, keepdims=True) + eps)
        unit = x[t] * r
        dw += (h * unit).sum(0)
        dw_size += (hs * np.abs(unit)).sum(0)
        u, us = h * weight, hs * np.abs(weight)
        dx[t] = r * (u - unit * (u * unit).mean(-1, keepdims=True))
        size[t] = r * (us + np.abs(unit) * (us * np.abs(unit)).mean(-1, keepdims=True))
    return (dx, size, None, None) if weight is None else (dx, size, dw, dw_size)


def append_slots(page_table, cache_lens, page_size, num_pages, cu_seqlens, cu_seqlens_padded, batch_size):
    """[(buffer row, page, token in it, slot)] of the rows that the table has a page for."""
    got = []
    for t, b, i in row_places(cu_seqlens, cu_seqlens_padded, batch_size):
        slot = int(cache_lens[b]) + i
        if slot < 0 or slot // page_size >= page_table.shape[1]:
            continue
        page = int(page_table[b, slot // page_size])
        if 0 <= page < num_pages:
            got.append((t, page, slot % page_size, slot))
    return got


def attention_paged(q, k_cache, v_cache, page_table, kv_lens, cu_seqlens_q, cu_seqlens_q_padded, batch_size, scale,
                    tree_mask=None):
    """(out, lse, size of out's terms, size of the scores' terms) of packed tokens over a paged cache."""
    q, kc, vc = _as64(q), _as64(k_cache), _as64(v_cache)
    T, hq, d = q.shape
    page_size, hkv = kc.shape[1], kc.shape[2]
    out, size = np.zeros_like(q), np.zeros_like(q)
    lse, score = np.full((hq, T), -np.inf), np.zeros((hq, T))
    starts, lengths = sequence_spans(cu_seqlens_q, cu_seqlens_q_padded, batch_size)
    for b in range(batch_size):
        L, n = min(int(kv_lens[b]), page_table.shape[1] * page_size), int(lengths[b])
        if L <= 0:
            continue
        pages = np.asarray(page_table[b, : -(-L // page_size)], dtype=np.int64)
        k = kc[pages].reshape(-1, hkv, d)[:L]
        v = vc[pages].reshape(-1, hkv, d)[:L]
        for i in range(n):
            t = int(starts[b]) + i
            j = np.arange(L) - (L - n)
            if tree_mask is None:
                seen = j <= i
            else:
                words = [int(w) & (1 << 64) - 1 for w in tree_mask[t]]
                seen = np.array([x < 0 or (x < 64 * len(words) and words[x // 64] >> (x % 64) & 1 == 1) for x in j.tolist()])
            if not seen.any():
                continue
            for h in range(hq):
                kk, vv = k[seen, h // (hq // hkv)], v[seen, h // (hq // hkv)]
                s = kk @ q[t, h] * scale
                e = np.exp(s - s.max())
                out[t, h] = e @ vv / e.sum()
                size[t, h] = e @ np.abs(vv) / e.sum()
                lse[h, t] = s.max() + np.log(e.sum())
                score[h, t] = (np.abs(kk) @ np.abs(q[t, h])).max() * scale
    return out, lse, size, score
