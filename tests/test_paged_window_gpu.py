"""GPU tests of attention over a paged cache with a window, first tokens that stay visible and the weights
that cached keys got, against the fp64 oracle.

Outputs and log-sum-exps as in test_paged_gpu.  A key's weight from one row is exp(s - lse): with e the share by
which an fp32 score moves its weight (test_paged_gpu), the log-sum-exp moves it by e and 4 * 2^-24 |lse| more, the
exponential and its argument by 2^-21 (1 + |lse|): 2 e + 2^-20 (1 + |lse|) of it.  The sum over n rows of weights that
are not negative is off by n 2^-24 of itself, adding it to what the key had by 2^-24 of the result.
"""
import numpy as np
import pytest
import torch

from oracle import bounded
from test_paged_gpu import BF16, FP16, f64, ints, make

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")


def weights_of(x, first=True, seed=0):
    """Weights that the keys had, laid out by heads or by tokens within a page."""
    pages, page, hkv, _ = x["kc"].shape
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(pages, hkv, page, generator=g).cuda() * 3
    return w.transpose(1, 2) if first else w.transpose(1, 2).contiguous()


def hide(x, left, sinks):
    """Keys that no token sees are not finite, and pages of such keys alone leave the table."""
    page, kept = x["kc"].shape[1], x["table"].copy()
    for b, (L, n) in enumerate(zip(x["keys"], np.diff(x["cu"]))):
        used = bounded.paged_sees(int(n), int(L), left, sinks).any(0)
        for p0 in range(0, int(L), page):
            here = used[p0:p0 + page]
            at = x["table"][b, p0 // page]
            hidden = torch.from_numpy(np.nonzero(~here)[0]).cuda()
            x["kc"][at, hidden], x["vc"][at, hidden] = float("nan"), float("inf")
            if not here.any():
                kept[b, p0 // page] = -1
    return kept


def run(x, table, left, sinks, weights=None, **over):
    work = torch.zeros(vlp.thd_attn_paged_workspace_size(x["q"].shape[2]) + (1 << 22), dtype=torch.uint8, device="cuda")
    kw = dict(cu_seqlens_q_padded=None if x["padded"] is None else ints(x["padded"]), batch_size=x["B"], workspace=work,
              tree_mask=None if x["tree"] is None else torch.tensor(x["tree"]).cuda(), window=(left, -1),
              sink_tokens=sinks, key_weights=weights)
    kw.update(over)
    got = vlp.thd_attn_paged(x["q"], x["kc"], x["vc"], ints(table), ints(x["keys"]), ints(x["cu"]), **kw)
    torch.cuda.synchronize()
    assert int(work[8:12].view(torch.int32).item()) == 0   # of a workspace that the call was given
    return got


def check(x, got, left, sinks, had=None, weights=None):
    """Outputs, and (had: the weights before) the keys' weights; every other place of theirs as it was."""
    q, scale = x["q"], x["q"].shape[2] ** -0.5
    dtype = q.dtype
    ref, ref_lse, size, score, added = bounded.attention_paged(f64(q), f64(x["kc"]), f64(x["vc"]), x["table"], x["keys"],
                                                               x["cu"], x["padded"], x["B"], scale, left, sinks, x["tree"])
    u = torch.finfo(dtype).eps / 2
    seen = np.isfinite(ref_lse)
    lse = got[1].cpu().double().numpy()
    assert np.array_equal(np.isneginf(lse), ~seen)
    lse, ref_lse = np.where(seen, lse, 0), np.where(seen, ref_lse, 0)
    e = 136 * 2.0 ** -23 * score + 2.0 ** -21 * (1 + score)
    assert np.all(np.abs(lse - ref_lse) <= e + 4 * 2.0 ** -24 * np.abs(ref_lse))
    o = f64(got[0])
    assert np.all(o[~seen.T] == 0)
    vmax = np.abs(np.nan_to_num(f64(x["vc"]), nan=0, posinf=0)).max()
    tiny = 2.0 ** -25 * x["keys"].max() * vmax if dtype == FP16 else 0.0
    bound = 2 * u * size + u * np.abs(ref) + 2 * e.T[:, :, None] * size + tiny + 2.0 ** -25
    worst = (np.abs(o - ref) / bound).max() if o.size else 0.0
    print(f"largest share of the bound {worst:.3f}")
    assert worst <= 1.0, worst
    if weights is None:
        return
    expect, err = had.cpu().double().numpy(), np.zeros(had.shape)
    starts = x["cu"] if x["padded"] is None else x["padded"]
    group = q.shape[1] // x["kc"].shape[2]
    for b in range(x["B"]):
        n, t0 = int(x["cu"][b + 1] - x["cu"][b]), int(starts[b])
        L = added[b].shape[1]
        if n <= 0 or L == 0:
            continue
        page, at = bounded.pages_of(x["table"], b, L, x["kc"].shape[1])
        fresh = np.arange(L) >= L - n
        base = np.where(fresh[:, None], 0.0, expect[page, at])
        expect[page, at] = base + added[b].T
        share = 2 * e[:, t0:t0 + n].max() + 2.0 ** -20 * (1 + np.abs(ref_lse[:, t0:t0 + n]).max()) + n * group * 2.0 ** -24
        err[page, at] = share * added[b].T + 2.0 ** -24 * np.abs(expect[page, at]) + 2.0 ** -126
    w = weights.cpu().double().numpy()
    worst = (np.abs(w - expect) / np.where(err > 0, err, 1)).max()
    print(f"weights: largest share of the bound {worst:.3f}")
    assert np.array_equal(w[err == 0], expect[err == 0]) and worst <= 1.0, worst


CASES = [
    # keys, new, page, hq, hkv, d, dtype, gap, heads first, left, sinks
    ([1], [1], 16, 4, 1, 128, BF16, 0, False, 0, 0),
    ([777], [1], 16, 8, 2, 128, BF16, 0, False, 127, 4),
    ([777, 64, 65, 3, 0, 1000], [1] * 6, 16, 8, 2, 128, BF16, 3, False, 63, 1),
    ([5000, 200, 129], [1, 1, 1], 24, 16, 2, 64, FP16, 0, True, 128, 70),
    ([5000, 200, 129], [1, 0, 2], 1, 5, 5, 40, BF16, 0, False, 1, 130),
    ([900, 2000], [4, 3], 8, 8, 2, 96, BF16, 0, False, 200, 64),         # several tokens of a narrow tile
    ([900, 2000, 30], [70, 130, 30], 16, 16, 4, 128, BF16, 5, False, 99, 4),
    ([900, 2000, 3000], [300, 1, 33], 32, 8, 1, 64, FP16, 0, True, 0, 0),
    ([4000], [600], 64, 4, 1, 80, BF16, 0, False, 333, 65),
    ([3], [9], 16, 4, 2, 128, BF16, 0, False, 2, 1),                     # fewer keys than tokens
    ([3000], [40], 16, 32, 8, 128, FP16, 0, False, 2999, 5),             # a window over all keys
    ([100], [3], 16, 32, 8, 128, BF16, 0, False, 5000, 5),               # and over more
]


@pytest.mark.parametrize("keys,new,page,hq,hkv,d,dtype,gap,first,left,sinks", CASES)
def test_window_matches_oracle(keys, new, page, hq, hkv, d, dtype, gap, first, left, sinks):
    x = make(keys, new, page, hq, hkv, d, dtype, gap=gap, first=first)
    table = hide(x, left, sinks)
    for hint in (0, max(new)):
        check(x, run(x, table, left, sinks, max_seqlen_q=hint), left, sinks)


@pytest.mark.parametrize("keys,new,page,hq,hkv,d,dtype,gap,first,left,sinks", CASES)
def test_weights_under_a_window(keys, new, page, hq, hkv, d, dtype, gap, first, left, sinks):
    x = make(keys, new, page, hq, hkv, d, dtype, gap=gap, first=first, seed=1)
    table = hide(x, left, sinks)
    for hint in (0, max(new)):
        w = weights_of(x, first)
        had = w.clone()
        check(x, run(x, table, left, sinks, w, max_seqlen_q=hint), left, sinks, had, w)


@pytest.mark.parametrize("keys,new,page,hq,hkv,d,dtype,gap,words,first", [
    ([1], [1], 1, 1, 1, 8, BF16, 0, 0, False),
    ([777], [1], 16, 8, 2, 128, BF16, 0, 0, False),
    ([777, 0, 64, 65, 1], [1, 0, 1, 1, 1], 16, 32, 8, 128, FP16, 4, 0, True),
    ([5000, 70], [1, 1], 24, 6, 2, 72, BF16, 0, 0, False),
    ([300, 17], [27, 9], 16, 16, 4, 128, BF16, 0, 1, False),             # trees
    ([300, 170], [5, 100], 16, 8, 2, 64, FP16, 0, 2, True),
    ([900, 2000, 30], [70, 130, 30], 16, 16, 4, 128, BF16, 5, 0, False),
    ([3], [9], 16, 4, 2, 128, BF16, 0, 0, False),
    ([40000], [3], 64, 4, 1, 128, BF16, 0, 0, True),
    ([1500], [1500], 128, 4, 2, 64, FP16, 0, 0, False),
])
def test_weights_match_oracle(keys, new, page, hq, hkv, d, dtype, gap, words, first):
    x = make(keys, new, page, hq, hkv, d, dtype, gap=gap, words=words, first=first, seed=2)
    for hint in (0, max(new)):
        w = weights_of(x, not first)
        had = w.clone()
        got = run(x, x["table"], -1, 0, w, max_seqlen_q=hint)
        check(x, got, -1, 0, had, w)
        # the attention itself is the call without them
        plain = run(x, x["table"], -1, 0, max_seqlen_q=hint)
        assert torch.equal(plain[0], got[0]) and torch.equal(plain[1], got[1])
        # twice the same: the same bits
        again = had.clone()
        run(x, x["table"], -1, 0, again, max_seqlen_q=hint)
        assert torch.equal(again, w)


@pytest.mark.parametrize("keys,new,page,hq,hkv,d,dtype,words,left,sinks", [
    ([2000, 300], [40, 90], 16, 10, 2, 128, BF16, 0, -1, 0),             # tiles of 125 rows
    ([700, 1300], [200, 1], 16, 48, 3, 64, FP16, 0, -1, 0),              # of 8 tokens
    ([500], [30], 16, 100, 1, 40, BF16, 0, -1, 0),                       # of one token
    ([400], [3], 16, 200, 1, 32, BF16, 0, -1, 0),                        # more heads in a group than rows in a tile
    ([900, 257, 256], [60, 60, 256], 8, 4, 2, 8, BF16, 0, -1, 0),        # the narrowest heads
    ([900, 129, 128], [60, 60, 128], 8, 4, 2, 16, FP16, 0, 77, 3),
    ([3000, 1] * 40, [33, 1] * 40, 16, 8, 4, 128, BF16, 0, -1, 0),       # several items for each CTA
    ([5000] * 6, [300] * 6, 16, 8, 2, 64, BF16, 0, 1000, 300),
    ([400, 900], [100, 130], 16, 8, 2, 96, FP16, 3, -1, 0),              # trees over several words and tiles
])
def test_weights_from_many_rows(keys, new, page, hq, hkv, d, dtype, words, left, sinks):
    x = make(keys, new, page, hq, hkv, d, dtype, words=words, seed=3, gap=2)
    table = hide(x, left, sinks) if left >= 0 else x["table"]
    w = weights_of(x)
    had = w.clone()
    check(x, run(x, table, left, sinks, w), left, sinks, had, w)


def test_weights_with_and_without_room_for_the_scores():
    for left, sinks in ((-1, 0), (100, 5)):
        x = make([777, 64, 65, 3, 0, 1000], [1, 2, 1, 3, 1, 4], 16, 16, 4, 128, BF16, gap=3)
        sizes = (128, 16, 6, 4, len(x["kc"]), 16, x["table"].shape[1], (left, -1), sinks)
        base, full = vlp.thd_attn_paged_workspace_size(128), vlp.thd_attn_paged_weights_workspace_size(*sizes)
        assert full > base and vlp.thd_attn_paged_weights_workspace_size(129, *sizes[1:]) == 0
        for size in (base, base + 4096, full):
            w = weights_of(x)
            had = w.clone()
            work = torch.empty(size, dtype=torch.uint8, device="cuda")
            check(x, vlp.thd_attn_paged(x["q"], x["kc"], x["vc"], ints(x["table"]), ints(x["keys"]), ints(x["cu"]),
                                        ints(x["padded"]), max_seqlen_q=4, workspace=work, window=(left, -1),
                                        sink_tokens=sinks, key_weights=w), left, sinks, had, w)
        # a hint that is too small: a sequence of several narrow tiles
        y = make([300, 500], [9, 2], 16, 16, 4, 128, BF16)
        w = weights_of(y)
        had = w.clone()
        check(y, run(y, y["table"], left, sinks, w, max_seqlen_q=2, workspace=None), left, sinks, had, w)


def test_sinks_without_a_window_and_weights_without_the_lse():
    x = make([300, 40], [2, 5], 16, 8, 2, 64, BF16)
    a, b = run(x, x["table"], -1, 0), run(x, x["table"], -1, 9)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    w, v = weights_of(x), weights_of(x)
    run(x, x["table"], -1, 0, w)
    out, lse = run(x, x["table"], -1, 0, v, return_lse=False)
    assert lse is None and torch.equal(out, a[0]) and torch.equal(w, v)


def test_weights_of_bad_pages_and_metadata_stay_in_the_buffers():
    x = make([50, 60, 70], [3, 4, 5], 8, 4, 2, 64, BF16)
    x["kc"].nan_to_num_(0, 0, 0), x["vc"].nan_to_num_(0, 0, 0)
    rng = np.random.default_rng(6)
    for left in (-1, 20):
        for _ in range(6):
            y = dict(x, table=rng.integers(-5, 60, x["table"].shape), keys=rng.integers(-10, 10**6, 3),
                     cu=rng.integers(-30, 30, 4))
            run(y, y["table"], left, 3, weights_of(x))
    bad = dict(x, table=np.full_like(x["table"], -1))
    w = weights_of(x)
    had = w.clone()
    run(bad, bad["table"], -1, 0, w)
    assert torch.equal(w, had)   # keys of no page have no weight
    had = w.clone()
    check(x, run(x, x["table"], 20, 3, w), 20, 3, had, w)


def test_refusals():
    x = make([30], [2], 16, 4, 2, 64, BF16, words=1)
    w = weights_of(x)
    with pytest.raises(vlp.ThdError) as err:
        run(x, x["table"], 5, 0)   # a window and a tree
    assert err.value.status == vlp.THD_ERR_UNSUPPORTED
    for over, kind in ((dict(window=(-2, 0)), ValueError), (dict(window=(3, 0), sink_tokens=-1), ValueError),
                       (dict(sink_tokens=-1), ValueError), (dict(key_weights=w.double()), TypeError),
                       (dict(key_weights=w[:-1]), ValueError), (dict(key_weights=w.cpu()), TypeError),
                       (dict(key_weights=w[:1].expand(w.shape)), ValueError), (dict(window=(2 ** 31, 0)), ValueError)):
        with pytest.raises(kind):
            run(x, x["table"], -1, 0, **over)


def test_graph_with_weights_replayed_with_other_lengths():
    x = make([70, 900, 5], [1, 1, 1], 16, 8, 2, 128, BF16)
    table, keys = ints(x["table"]), ints(x["keys"])
    held = weights_of(x)
    work = torch.empty(vlp.thd_attn_paged_workspace_size(128), dtype=torch.uint8, device="cuda")
    call = lambda: vlp.thd_attn_paged(x["q"], x["kc"], x["vc"], table, keys, ints_cu, max_seqlen_q=1, workspace=work,  # noqa: E731
                                      window=(300, 0), sink_tokens=4, key_weights=held)
    ints_cu = ints(x["cu"])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for lens in ([70, 900, 5], [60, 500, 1], [1, 899, 0]):
        y = dict(x, keys=np.array(lens))
        keys.copy_(ints(lens))
        had = weights_of(x, seed=lens[0])
        held.copy_(had)
        graph.replay()
        torch.cuda.synchronize()
        check(y, got, 300, 4, had, held)
