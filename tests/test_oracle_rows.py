"""CPU pins of the fp64 oracle of the row operators: closed forms, autograd, differences, and the
packed attention oracle."""
import numpy as np
import pytest
import torch

import oracle
from oracle import rows


def tables(n, rotary, base=100.0):
    angle = np.arange(n)[:, None] * base ** (-np.arange(0, rotary, 2) / rotary)
    return np.cos(angle), np.sin(angle)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(interleaved):
    rng = np.random.default_rng(0)
    cos, sin = tables(20, 16)
    a, b = rng.standard_normal(32), rng.standard_normal(32)
    at = lambda x, p: rows.norm_rope_row(x[None], None, 0.0, cos[p], sin[p], interleaved)[0][0]
    assert np.allclose(at(a, 0), a)
    assert np.isclose(np.linalg.norm(at(a, 7)), np.linalg.norm(a))
    assert np.isclose(at(a, 9) @ at(b, 4), at(a, 16) @ at(b, 11))
    assert np.array_equal(at(a, 5)[16:], a[16:])


def test_interleaved_is_a_permutation_of_half_split():
    rng = np.random.default_rng(1)
    cos, sin = tables(9, 16)
    x = rng.standard_normal((3, 16))
    order = np.arange(16).reshape(2, 8).T.reshape(-1)   # place 2c holds value c, 2c + 1 value c + 8
    y = rows.norm_rope_row(x, None, 0.0, cos[5], sin[5], False)[0]
    z = rows.norm_rope_row(x[:, order], None, 0.0, cos[5], sin[5], True)[0]
    assert np.allclose(z, y[:, order])


def test_norm_of_a_constant_head():
    w = np.linspace(0.5, 1.5, 16)
    y = rows.norm_rope_row(np.full((1, 16), -3.0), w, 0.0, None, None, False)[0]
    assert np.allclose(y, -w)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_gradients_against_autograd_and_differences(interleaved, normed):
    rng = np.random.default_rng(2)
    cos, sin = tables(12, 16)
    cu, padded, T = [0, 3, 3, 7], [1, 4, 6], 12
    x, g, w = rng.standard_normal((T, 2, 32)), rng.standard_normal((T, 2, 32)), rng.standard_normal(32)
    weight = w if normed else None
    f = lambda x, w: rows.norm_rope(x, w if normed else None, 1e-3, cos, sin, interleaved, cu, padded, 3, [0, 0, 4])[0]
    dx, size, dw, _ = rows.norm_rope_bwd(g, x, weight, 1e-3, cos, sin, interleaved, cu, padded, 3, [0, 0, 4])
    assert np.all(np.abs(dx) <= size + 1e-12)
    assert np.all(dx[[0, 4, 5, 10, 11]] == 0) and np.all(f(x, w)[[0, 4, 5, 10, 11]] == 0)
    for _ in range(4):
        e, ew = rng.standard_normal(x.shape), rng.standard_normal(32)
        step = 1e-6
        want = ((f(x + step * e, w) - f(x - step * e, w)) * g).sum() / (2 * step)
        assert np.isclose((dx * e).sum(), want, rtol=1e-6, atol=1e-6)
        if normed:
            want = ((f(x, w + step * ew) - f(x, w - step * ew)) * g).sum() / (2 * step)
            assert np.isclose((dw * ew).sum(), want, rtol=1e-6, atol=1e-6)
    # torch autograd of the same formula, sequence by sequence
    xt = torch.tensor(x, requires_grad=True)
    wt = torch.tensor(w, requires_grad=True)
    total = 0.0
    for t, b, i in rows.row_places(cu, padded, 3):
        h = xt[t]
        if normed:
            h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-3) * wt
        p = i + [0, 0, 4][b]
        total = total + ((h @ torch.tensor(rows.rotation(32, 16, interleaved, cos[p], sin[p])).T) * torch.tensor(g[t])).sum()
    total.backward()
    assert np.allclose(xt.grad.numpy(), dx, atol=1e-12)
    if normed:
        assert np.allclose(wt.grad.numpy(), dw, atol=1e-12)


def paged_batch(rng, keys, page, hkv, d):
    """A cache with the pages in no order, and the keys and values of each sequence."""
    need = [-(-n // page) for n in keys]
    order = rng.permutation(sum(need) + 2)
    kc, vc = (rng.standard_normal((len(order), page, hkv, d)) for _ in range(2))
    table, at = np.full((len(keys), max(need) + 1), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return kc, vc, table


def test_paged_attention_is_bottom_right_packed_attention():
    rng = np.random.default_rng(3)
    new, keys, page, hq, hkv, d = [1, 4, 6, 0, 3], [9, 4, 20, 5, 2], 4, 4, 2, 8
    kc, vc, table = paged_batch(rng, keys, page, hkv, d)
    cu_q, cu_k = np.cumsum([0] + new), np.cumsum([0] + keys)
    T = int(max(cu_q[-1], cu_k[-1]))
    q = rng.standard_normal((T, hq, d))
    k, v = (np.zeros((T, hkv, d)) for _ in range(2))
    for b, n in enumerate(keys):
        k[cu_k[b]:cu_k[b + 1]] = kc[table[b, :-(-n // page)]].reshape(-1, hkv, d)[:n]
        v[cu_k[b]:cu_k[b + 1]] = vc[table[b, :-(-n // page)]].reshape(-1, hkv, d)[:n]
    want, want_lse = oracle.thd_attention_fwd_general(q, k, v, cu_q, cu_k, None, None, np.full(5, 2, np.uint8), 5, 0.3)
    out, lse, size, _ = rows.attention_paged(q, kc, vc, table, keys, cu_q, None, 5, 0.3)
    assert np.allclose(out, want) and np.allclose(lse[np.isfinite(lse)], want_lse[np.isfinite(want_lse)])
    assert np.array_equal(np.isfinite(lse), np.isfinite(want_lse))
    assert np.all(np.abs(out) <= size + 1e-12)
    # a chain is the tree of causal attention, whatever the number of words
    for words in (1, 2):
        mask = np.zeros((T, words), np.int64)
        for t, b, i in rows.row_places(cu_q, None, 5):
            mask[t, 0] = (1 << (i + 1)) - 1
        got, got_lse, _, _ = rows.attention_paged(q, kc, vc, table, keys, cu_q, None, 5, 0.3, mask)
        chain = np.isfinite(lse).all(0) & (np.array([keys[b] >= new[b] for t, b, i in rows.row_places(cu_q, None, 5)] + [False] * (T - cu_q[-1])))
        assert np.allclose(got[chain], out[chain]) and np.allclose(got_lse[:, chain], lse[:, chain])


def test_append_then_attend_is_attention_over_all_keys():
    rng = np.random.default_rng(4)
    page, hkv, d = 4, 1, 8
    before, new = [5, 0, 3], [2, 3, 1]
    kc, vc, table = paged_batch(rng, [a + b for a, b in zip(before, new)], page, hkv, d)
    table[2, 0] = -1   # no page: nothing is written
    cu = np.cumsum([0] + new)
    slots = rows.append_slots(table, before, page, len(kc), cu, None, 3)
    assert [s[0] for s in slots] == [0, 1, 2, 3, 4]
    assert [s[3] for s in slots] == [5, 6, 0, 1, 2]
    assert all(table[b, s // page] == p for (t, p, o, s), b in zip(slots, [0, 0, 1, 1, 1]))
