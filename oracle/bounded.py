"""fp64 oracle of the operators that bound what a long sequence costs: a sliding window with first
tokens that stay visible (packed attention with its gradients, attention over a paged cache),
the weight that cached keys got, and the eviction of keys by it.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Dense masks, one sequence and head at a
time; the functions also return the sizes of the terms a value is summed from, from which the
tests derive their tolerances.
"""
from __future__ import annotations

import numpy as np

from .attention import MASK_PADDING, MASK_PADDING_CAUSAL_BOTTOM_RIGHT, _as64, sequence_spans


def sees(Lq, Lkv, code, window=(-1, -1), sinks=0):
    """[Lq, Lkv]: whether query i sees key j under the mask type, the window and the first `sinks` keys."""
    i, j = np.arange(Lq)[:, None], np.arange(Lkv)[None, :]
    shift = Lkv - Lq if code == MASK_PADDING_CAUSAL_BOTTOM_RIGHT else 0
    allowed = np.ones((Lq, Lkv), bool) if code == MASK_PADDING else j <= i + shift
    left, right = window
    near = np.ones((Lq, Lkv), bool)
    if left >= 0:
        near &= j >= i + shift - left
    if right >= 0:
        near &= j <= i + shift + right
    return allowed & (near | (j < sinks))


def softmax_rows(z, seen):
    """(weights, log-sum-exp) of rows of scores; a row that sees nothing has no weight and -inf."""
    z = np.where(seen, z, -np.inf)
    top = np.where(seen.any(1), z.max(1, initial=-np.inf), 0.0)
    e = np.exp(z - top[:, None])
    total = e.sum(1)
    with np.errstate(divide="ignore"):
        return e / np.where(total > 0, total, 1.0)[:, None], top + np.log(total)


def _spans(cu_q, cu_kv, pad_q, pad_kv, batch):
    qs, ql = sequence_spans(cu_q, pad_q, batch)
    ks, kl = sequence_spans(cu_kv, pad_kv, batch)
    return [(b, int(qs[b]), int(ql[b]), int(ks[b]), int(kl[b])) for b in range(batch)]


def attention_fwd(q, k, v, cu_q, cu_kv, pad_q, pad_kv, codes, batch, scale, window=(-1, -1), sinks=0):
    """(out, lse, size of out's terms, size of the scores' terms)."""
    q, k, v = _as64(q), _as64(k), _as64(v)
    T, hq, _ = q.shape
    group = hq // k.shape[1]
    out, size = np.zeros_like(q), np.zeros_like(q)
    lse, score = np.full((hq, T), -np.inf), np.zeros((hq, T))
    for b, qs, Lq, ks, Lkv in _spans(cu_q, cu_kv, pad_q, pad_kv, batch):
        if Lq <= 0 or Lkv <= 0:
            continue
        seen = sees(Lq, Lkv, int(codes[b]), window, sinks)
        for h in range(hq):
            Q, K, V = q[qs:qs + Lq, h], k[ks:ks + Lkv, h // group], v[ks:ks + Lkv, h // group]
            p, lse[h, qs:qs + Lq] = softmax_rows(Q @ K.T * scale, seen)
            out[qs:qs + Lq, h], size[qs:qs + Lq, h] = p @ V, p @ np.abs(V)
            score[h, qs:qs + Lq] = np.where(seen, np.abs(Q) @ np.abs(K).T * scale, 0.0).max(1)
    return out, lse, size, score


def attention_bwd(q, k, v, out, lse, dout, cu_q, cu_kv, pad_q, pad_kv, codes, batch, scale, window=(-1, -1), sinks=0):
    """Gradients from the forward's results as given, and the largest size of a score's terms.  For q, k and v
    each: (gradient, size of its terms, what an error of 1 in rowsum(|dO O|) of each row would move it by, terms).
    P = exp(s - lse), D = rowsum(dO O)."""
    q, k, v, out, lse, dout = (_as64(x) for x in (q, k, v, out, lse, dout))
    hq, group = q.shape[1], q.shape[1] // k.shape[1]
    g = [tuple(np.zeros_like(x) for _ in range(3)) + (np.zeros(x.shape[:2] + (1,)),) for x in (q, k, v)]
    score = 0.0
    for b, qs, Lq, ks, Lkv in _spans(cu_q, cu_kv, pad_q, pad_kv, batch):
        if Lq <= 0 or Lkv <= 0:
            continue
        seen = sees(Lq, Lkv, int(codes[b]), window, sinks)
        for h in range(hq):
            m, rq, rk = h // group, slice(qs, qs + Lq), slice(ks, ks + Lkv)
            Q, K, V, dO, O = q[rq, h], k[rk, m], v[rk, m], dout[rq, h], out[rq, h]
            L = np.where(np.isfinite(lse[h, rq]), lse[h, rq], 0.0)
            p = np.exp(np.where(seen, Q @ K.T * scale - L[:, None], -np.inf))
            dp = dO @ V.T - (dO * O).sum(1)[:, None]
            sized, moved = p * np.abs(dp) * scale, p * np.abs(dO * O).sum(1)[:, None] * scale
            for of, where, a, s, d, c in ((g[0], (rq, h), p * dp * scale, sized, moved, K),
                                          (g[1], (rk, m), (p * dp).T * scale, sized.T, moved.T, Q),
                                          (g[2], (rk, m), p.T, p.T, 0 * p.T, dO)):
                of[0][where] += a @ c
                of[1][where] += s @ np.abs(c)
                of[2][where] += d @ np.abs(c)
                of[3][where] += (seen if of is g[0] else seen.T).sum(1)[:, None]
            score = max(score, np.where(seen, np.abs(Q) @ np.abs(K).T * scale, 0.0).max())
    return g, score


def pages_of(page_table, b, L, page):
    """(page, place in it) of keys 0..L-1 of sequence b."""
    at = np.arange(L)
    return np.asarray(page_table)[b, at // page].astype(np.int64), at % page


def paged_sees(n, L, left=-1, sinks=0, tree=None):
    """[n, L]: whether new token i sees key j; tree: the tokens' mask words."""
    i, j = np.arange(n)[:, None], np.arange(L)[None, :]
    own = L - n + i
    if tree is not None:
        bit = np.zeros((n, L), bool)
        for t in range(n):
            words = [int(w) & (1 << 64) - 1 for w in tree[t]]
            for x in range(L):
                r = x - (L - n)
                bit[t, x] = r < 0 or (r < 64 * len(words) and words[r // 64] >> (r % 64) & 1 == 1)
        return bit
    seen = (j <= own) & (j < L)
    if left >= 0:
        seen &= (j >= own - left) | (j < sinks)
    return seen


def attention_paged(q, k_cache, v_cache, page_table, kv_lens, cu_q, pad_q, batch, scale, left=-1, sinks=0, tree=None):
    """(out, lse, size of out's terms, size of the scores' terms, [weights that each key got, [Hkv, L]])."""
    q, kc, vc = _as64(q), _as64(k_cache), _as64(v_cache)
    T, hq, _ = q.shape
    page, hkv = kc.shape[1], kc.shape[2]
    group = hq // hkv
    out, size = np.zeros_like(q), np.zeros_like(q)
    lse, score = np.full((hq, T), -np.inf), np.zeros((hq, T))
    starts, lengths = sequence_spans(cu_q, pad_q, batch)
    weights = []
    for b in range(batch):
        L, n, t0 = min(int(kv_lens[b]), page_table.shape[1] * page), int(lengths[b]), int(starts[b])
        L = max(L, 0)
        weights.append(np.zeros((hkv, L)))
        if L == 0 or n <= 0:
            continue
        at = pages_of(page_table, b, L, page)
        seen = paged_sees(n, L, left, sinks, None if tree is None else tree[t0:t0 + n])
        used = seen.any(0)
        for h in range(hq):
            # what no token sees may be anything
            K, V = (np.where(used[:, None], x[at[0], at[1], h // group], 0.0) for x in (kc, vc))
            Q = q[t0:t0 + n, h]
            p, lse[h, t0:t0 + n] = softmax_rows(Q @ K.T * scale, seen)
            out[t0:t0 + n, h], size[t0:t0 + n, h] = p @ V, p @ np.abs(V)
            score[h, t0:t0 + n] = np.where(seen, np.abs(Q) @ np.abs(K).T * scale, 0.0).max(1)
            weights[-1][h // group] += p.sum(0)
    return out, lse, size, score, weights


def evict_keep(w, L, keep, sinks, recent):
    """Slots of one head that are kept, ascending: the first `sinks`, the last `recent`, and of the others those
    with the most weight (NaN above all; of equal ones the lower slot) up to `keep` in all."""
    K = max(0, min(keep, L))
    S = min(sinks, K)
    R = min(recent, K - S)
    rank = lambda x: np.inf if np.isnan(x) else float(x)  # noqa: E731
    middle = sorted(range(S, L - R), key=lambda i: (not np.isnan(w[i]), -rank(w[i]), i))[:K - S - R]
    return list(range(S)) + sorted(middle) + list(range(L - R, L))


def evict(caches, weights, page_table, kv_lens, keep_lens, new_page_table, batch, sinks, recent):
    """Copies of the caches (any list of [pages, page, Hkv, ...] arrays) and the weights after the eviction, the new
    lengths, and the kept slots [batch][Hkv]."""
    page, hkv = weights.shape[1], weights.shape[2]
    new = page_table if new_page_table is None else new_page_table
    got = [np.array(x) for x in caches] + [np.array(weights)]
    src = list(caches) + [weights]
    lens, kept = [], []
    for b in range(batch):
        L = max(0, min(int(kv_lens[b]), page_table.shape[1] * page))
        K = max(0, min(int(keep_lens[b]), L, new.shape[1] * page))
        lens.append(K)
        kept.append([])
        at, to = pages_of(page_table, b, L, page), pages_of(new, b, K, page)
        real = lambda x: (x >= 0) & (x < weights.shape[0])  # noqa: E731
        for h in range(hkv):
            # a slot of no page has no weight, and neither goes nor comes
            w = np.where(real(at[0]), np.asarray(weights)[np.where(real(at[0]), at[0], 0), at[1], h], 0.0)
            slots = evict_keep(w, L, K, sinks, recent)
            kept[-1].append(slots)
            f, go = np.array(slots, int), real(to[0]) & real(at[0][slots])
            for x, y in zip(got, src):
                x[to[0][go], to[1][go], h] = np.asarray(y)[at[0][f[go]], at[1][f[go]], h]
    return got[:-1], got[-1], lens, kept
