"""The oracle of window, sinks, key weights and eviction against independent statements (no GPU)."""
import numpy as np
import pytest

import oracle
from oracle import bounded, rows


@pytest.mark.parametrize("code", [0, 1, 2])
@pytest.mark.parametrize("window", [(-1, -1), (0, 0), (2, 0), (-1, 3), (3, 2)])
@pytest.mark.parametrize("Lq,Lkv", [(7, 7), (4, 9), (9, 4), (1, 5)])
def test_sees_without_sinks_is_the_window_of_the_packed_oracle(code, window, Lq, Lkv):
    seen = bounded.sees(Lq, Lkv, code, window)
    for i in range(Lq):
        lo, hi = oracle.visible_range(i, Lq, Lkv, code, window)
        assert np.array_equal(np.nonzero(seen[i])[0], np.arange(max(lo, 0), max(hi, lo)))


def test_sees_pairs_by_hand():
    # causal, window of one key back, two sinks
    seen = bounded.sees(5, 5, 1, (1, 0), 2)
    assert [list(np.nonzero(r)[0]) for r in seen] == [[0], [0, 1], [0, 1, 2], [0, 1, 2, 3], [0, 1, 3, 4]]
    # full context, window of width zero: the sinks are seen by the rows before them too
    seen = bounded.sees(4, 4, 0, (0, 0), 2)
    assert [list(np.nonzero(r)[0]) for r in seen] == [[0, 1], [0, 1], [0, 1, 2], [0, 1, 3]]
    # bottom-right with fewer keys than queries: the mask type hides the sinks too
    assert bounded.sees(4, 2, 2, (0, 0), 1).sum(1).tolist() == [0, 0, 1, 2]


def _batch(rng, hq=4, hkv=2, d=8):
    lens = np.array([6, 1, 9, 0, 5])
    cu = np.concatenate([[0], np.cumsum(lens)])
    pad = np.array([1, 8, 9, 20, 20])
    T = 27
    return lens, cu, pad, [rng.standard_normal((T, h, d)) for h in (hq, hkv, hkv)]


def test_gradients_against_differences():
    rng = np.random.default_rng(0)
    _, cu, pad, x = _batch(rng)
    codes, kw = [1, 0, 2, 1, 0], dict(window=(2, 1), sinks=2)
    dout = rng.standard_normal(x[0].shape)
    loss = lambda: (bounded.attention_fwd(*x, cu, cu, pad, pad, codes, 5, 0.4, **kw)[0] * dout).sum()  # noqa: E731
    out, lse, _, _ = bounded.attention_fwd(*x, cu, cu, pad, pad, codes, 5, 0.4, **kw)
    grads, _ = bounded.attention_bwd(*x, out, lse, dout, cu, cu, pad, pad, codes, 5, 0.4, **kw)
    for t, (g, size, _, _) in zip(x, grads):
        assert np.all(np.abs(g) <= size + 1e-12)
        for _ in range(25):
            at = tuple(int(rng.integers(n)) for n in t.shape)
            had, step = t[at], 1e-5
            t[at] = had + step
            up = loss()
            t[at] = had - step
            down = loss()
            t[at] = had
            assert abs((up - down) / (2 * step) - g[at]) < 1e-7


def test_without_window_they_are_the_oracles_of_the_plain_operators():
    rng = np.random.default_rng(1)
    _, cu, pad, x = _batch(rng)
    codes = np.array([1, 0, 2, 1, 0], np.uint8)
    out, lse, _, _ = bounded.attention_fwd(*x, cu, cu, pad, pad, codes, 5, 0.4)
    ref, ref_lse = oracle.thd_attention_fwd_general(*x, cu, cu, pad, pad, codes, 5, 0.4)
    assert np.allclose(out, ref, atol=1e-13) and np.allclose(lse, ref_lse, atol=1e-13)
    dout = rng.standard_normal(x[0].shape)
    grads, _ = bounded.attention_bwd(*x, out, lse, dout, cu, cu, pad, pad, codes, 5, 0.4)
    for (g, _, _, _), r in zip(grads, oracle.thd_attention_bwd(*x, dout, cu, cu, pad, pad, codes, 5, 0.4)):
        assert np.allclose(g, r, atol=1e-12)


def test_paged_is_the_packed_form_over_pages_and_weights_sum_to_the_rows():
    rng = np.random.default_rng(2)
    kc, vc = rng.standard_normal((2, 9, 4, 2, 8))
    table = rng.permutation(9).reshape(3, 3)
    keys, cu = [11, 5, 0], np.array([0, 3, 5, 6])
    q = rng.standard_normal((6, 4, 8))
    out, lse, _, _, w = bounded.attention_paged(q, kc, vc, table, keys, cu, None, 3, 0.4)
    ref, ref_lse, _, _ = rows.attention_paged(q, kc, vc, table, keys, cu, None, 3, 0.4)
    assert np.allclose(out, ref, atol=1e-13) and np.allclose(lse, ref_lse, atol=1e-13)
    assert np.allclose([x.sum(1) for x in w[:2]], [[6, 6], [4, 4]]) and w[2].shape == (2, 0)
    out, lse, _, _, w = bounded.attention_paged(q, kc, vc, table, keys, cu, None, 3, 0.4, left=1, sinks=2)
    at = bounded.pages_of(table, 0, 11, 4)
    p_out, p_lse, _, _ = bounded.attention_fwd(q[:3], kc[at], vc[at], [0, 3], [0, 11], None, None, [2], 1, 0.4, (1, 0), 2)
    assert np.allclose(out[:3], p_out) and np.allclose(lse[:, :3], p_lse) and np.all(w[0][:, 2:7] == 0)


def test_evict_by_hand():
    w = np.array([0.0, 5.0, 1.0, 3.0, 3.0, np.nan, 0.0, -1.0, 2.0, 0.1])
    assert bounded.evict_keep(w, 10, 5, 1, 2) == [0, 1, 5, 8, 9]
    assert bounded.evict_keep(w, 10, 6, 1, 2) == [0, 1, 3, 5, 8, 9]      # of 3.0 and 3.0 the lower slot
    assert bounded.evict_keep(w, 10, 2, 4, 4) == [0, 1]                  # sinks first
    assert bounded.evict_keep(w, 10, 6, 4, 4) == [0, 1, 2, 3, 8, 9]
    assert bounded.evict_keep(w, 10, 99, 0, 0) == list(range(10))
    assert bounded.evict_keep(w, 10, 0, 3, 3) == [] == bounded.evict_keep(w, 10, -4, 3, 3)


def test_evict_in_place_and_into_other_pages_agree():
    rng = np.random.default_rng(3)
    kc, vc = rng.standard_normal((2, 12, 4, 2, 8))
    w = rng.integers(0, 4, (12, 4, 2)).astype(float)
    order = rng.permutation(12)
    table, other = order[:6].reshape(2, 3), order[6:].reshape(2, 3)
    a = bounded.evict([kc, vc], w, table, [11, 7], [6, 9], None, 2, 1, 2)
    b = bounded.evict([kc, vc], w, table, [11, 7], [6, 9], other, 2, 1, 2)
    assert a[2] == b[2] == [6, 7] and a[3] == b[3]
    for x, y in zip(a[0] + [a[1]], b[0] + [b[1]]):
        for i, n in enumerate(a[2]):
            assert np.array_equal(x[bounded.pages_of(table, i, n, 4)], y[bounded.pages_of(other, i, n, 4)])
    assert np.array_equal(a[0][0][bounded.pages_of(table, 1, 7, 4)], kc[bounded.pages_of(table, 1, 7, 4)])
