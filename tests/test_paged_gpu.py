"""GPU tests of attention over a paged cache against the fp64 oracle.

Tolerances, u = finfo(dtype).eps / 2 the relative rounding of the 16-bit type.  The weights are
rounded to it, in the numerator and in the sum that normalises them: 2 u of A = sum_j w_j |v_j|; the
output once more: u |out| (and half the least subnormal).  A score is an fp32 sum of up to 128
products, each step off by at most 2^-23 (the matrix units truncate) of S = scale * sum |q k|: with
the product by the scale and the exponential's 2 ulp, e = 136 * 2^-23 * S + 2^-21 * (1 + |s|), which moves
the weights by that share, twice (numerator and sum).  fp16 weights below 2^-14 of the largest round
absolutely, by 2^-25 each: 2^-25 * keys * max |v|.  The log-sum-exp: e, and 4 * 2^-24 of its size.
"""
import numpy as np
import pytest
import torch

from oracle import rows as oracle_rows

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")

BF16, FP16 = torch.bfloat16, torch.float16


def f64(t):
    return t.detach().float().cpu().double().numpy()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def tree_masks(rng, n, words):
    """Masks [n, words] of a random tree (each token sees itself and those above it)."""
    sees = [1]
    for i in range(1, n):
        sees.append(sees[int(rng.integers(max(0, i - 7), i))] | 1 << i)
    out = np.zeros((n, words), np.uint64)
    for i, x in enumerate(sees):
        for w in range(words):
            out[i, w] = x >> (64 * w) & (1 << 64) - 1
    return out.astype(np.int64)


def make(keys, new, page, hq, hkv, d, dtype, gap=0, words=0, first=False, seed=0, extra=3):
    rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    B = len(keys)
    cu = np.concatenate([[0], np.cumsum(new)])
    padded, T = None, int(cu[-1])
    if gap:
        starts, at = [], 0
        for n in new:
            at += int(rng.integers(0, gap + 1))
            starts.append(at)
            at += n
        padded, T = np.array(starts), at + gap
    need = [-(-n // page) for n in keys]
    order = rng.permutation(sum(need) + 2)
    table = np.full((B, max(need + [0]) + extra), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    kv = [torch.randn(len(order), hkv, page, d, generator=g).to(dtype).cuda().transpose(1, 2) if first else
          torch.randn(len(order), page, hkv, d, generator=g).to(dtype).cuda() for _ in range(2)]
    # what lies behind the keys of a sequence is not finite
    for b, n in enumerate(keys):
        if n % page:
            for x, bad in zip(kv, (float("nan"), float("inf"))):
                x[table[b, n // page], n % page:] = bad
    for p in order[at:]:
        kv[0][p], kv[1][p] = float("inf"), float("nan")
    q = torch.randn(T, hq, d, generator=g).to(dtype).cuda()
    tree = None
    if words:
        tree = np.full((T, words), -1, np.int64)
        starts = cu if padded is None else padded
        for b, n in enumerate(new):
            if n:
                tree[starts[b]:starts[b] + n] = tree_masks(rng, n, words)
    return dict(q=q, kc=kv[0], vc=kv[1], table=table, keys=np.array(keys), cu=cu, padded=padded, B=B, tree=tree)


def run(x, **over):
    kw = dict(cu_seqlens_q_padded=None if x["padded"] is None else ints(x["padded"]), batch_size=x["B"],
              tree_mask=None if x["tree"] is None else torch.tensor(x["tree"]).cuda())
    kw.update(over)
    out = vlp.thd_attn_paged(x["q"], x["kc"], x["vc"], ints(x["table"]), ints(x["keys"]), ints(x["cu"]), **kw)
    torch.cuda.synchronize()
    return out


def check(x, got, scale=None):
    out, lse = got
    q = x["q"]
    d, dtype = q.shape[2], q.dtype
    scale = d ** -0.5 if scale is None else scale
    kc, vc = np.nan_to_num(f64(x["kc"]), nan=0, posinf=0), np.nan_to_num(f64(x["vc"]), nan=0, posinf=0)
    ref, ref_lse, size, score = oracle_rows.attention_paged(f64(q), kc, vc, x["table"], x["keys"], x["cu"], x["padded"],
                                                            x["B"], scale, x["tree"])
    u = torch.finfo(dtype).eps / 2
    seen = np.isfinite(ref_lse)
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), ~seen)
    e = 136 * 2.0 ** -23 * score + 2.0 ** -21 * (1 + score)
    l64 = lse.cpu().double().numpy()
    lse_err = np.abs(np.where(seen, l64, 0) - np.where(seen, ref_lse, 0))
    assert np.all(lse_err <= e + 4 * 2.0 ** -24 * np.abs(np.where(seen, ref_lse, 0))), lse_err.max()
    o = f64(out)
    assert np.all(o[~seen.T] == 0)
    least = 2.0 ** -25 if dtype == FP16 else 2.0 ** -134
    tiny = 2.0 ** -25 * x["keys"].max() * np.abs(vc).max() if dtype == FP16 else 0.0
    bound = 2 * u * size + u * np.abs(ref) + 2 * e.T[:, :, None] * size + least + tiny
    worst = (np.abs(o - ref) / np.where(seen.T[:, :, None], bound, 1)).max() if o.size else 0.0
    print(f"largest share of the bound {worst:.3f}")
    assert worst <= 1.0, worst


CASES = [
    # keys, new, page, hq, hkv, d, dtype, gap, tree words, heads first
    ([1], [1], 1, 1, 1, 8, BF16, 0, 0, False),
    ([1], [1], 16, 4, 1, 128, BF16, 0, 0, False),
    ([777], [1], 16, 8, 2, 128, BF16, 0, 0, False),
    ([0, 1, 63, 64, 65, 128, 500], [1] * 7, 16, 4, 4, 128, FP16, 0, 0, False),
    ([300, 0, 17, 1000, 5], [1, 1, 0, 1, 1], 24, 10, 2, 80, BF16, 3, 0, True),
    ([130, 64, 3], [5, 64, 3], 8, 6, 2, 64, BF16, 2, 0, False),
    ([40, 9, 200], [3, 20, 33], 32, 8, 1, 128, FP16, 0, 0, False),      # fewer keys than new tokens
    ([90, 200, 64, 70], [27, 64, 64, 1], 16, 8, 2, 128, BF16, 0, 1, False),
    ([150, 333], [70, 130], 64, 4, 2, 64, FP16, 3, 3, True),
    ([100, 50], [70, 7], 16, 2, 2, 48, BF16, 0, 1, False),              # tokens past the mask's words
    ([4100], [2], 256, 32, 2, 96, BF16, 0, 0, False),
    ([20, 21], [1, 2], 7, 34, 1, 40, FP16, 0, 0, False),                # 34 heads share one key head
    ([700, 900], [160, 150], 16, 4, 2, 128, BF16, 0, 0, False),         # a chunk of new tokens
]


@pytest.mark.parametrize("hint", [True, False])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_paged(case, hint):
    keys, new, page, hq, hkv, d, dtype, gap, words, first = case
    x = make(keys, new, page, hq, hkv, d, dtype, gap, words, first)
    check(x, run(x, max_seqlen_q=max(new) if hint else 0))


def test_masks_that_leave_a_row_empty():
    """No cached keys before the tree, and rows whose mask is empty."""
    x = make([9, 40], [9, 9], 4, 4, 2, 64, BF16, words=1)
    x["tree"][3] = x["tree"][12] = 0
    x["tree"][4] = 1 << 60            # bits past the new tokens show nothing
    check(x, run(x))
    assert torch.all(run(x)[0][3] == 0) and torch.all(run(x)[0][4] == 0)
    x = make([5, 70], [9, 71], 4, 4, 2, 64, BF16, words=2)   # fewer keys than drafted tokens
    for hint in (1, 71):
        check(x, run(x, max_seqlen_q=hint))


def test_many_sequences_and_a_wrong_hint():
    rng = np.random.default_rng(5)
    keys = rng.integers(0, 40, 700)
    new = np.minimum(rng.integers(0, 4, 700), keys)
    x = make(keys.tolist(), new.tolist(), 8, 4, 2, 32, BF16)
    check(x, run(x, max_seqlen_q=1))


@pytest.mark.parametrize("scale", [1e-3, 3.0])
def test_scales_and_large_scores(scale):
    x = make([200, 31], [1, 3], 16, 8, 4, 64, FP16, seed=2)
    x["q"] *= 4
    check(x, run(x, softmax_scale=scale), scale)


def test_one_long_sequence_sampled():
    """131,071 keys over every CTA, and a cache whose offsets pass 2^31 elements."""
    keys, page, hkv, d = 131071, 16, 1, 128
    g = torch.Generator("cuda").manual_seed(1)
    pages = 1 << 20                    # 2^31 elements a cache
    kc = torch.empty(pages + 4, page, hkv, d, dtype=BF16, device="cuda").normal_(generator=g)
    vc = torch.empty_like(kc).normal_(generator=g)
    need = -(-keys // page)
    table = torch.arange(pages + 3, pages + 3 - need, -1, dtype=torch.int32, device="cuda")[None]
    q = torch.empty(1, 8, d, dtype=BF16, device="cuda").normal_(generator=g)
    out, lse = vlp.thd_attn_paged(q, kc, vc, table, ints([keys]), ints([0, 1]), max_seqlen_q=1)
    k = kc[table[0].long()].reshape(-1, d)[:keys].double()
    v = vc[table[0].long()].reshape(-1, d)[:keys].double()
    s = q[0].double() @ k.T * d ** -0.5
    p = s.softmax(-1)
    ref, A = p @ v, p @ v.abs()
    S = (q[0].double().abs() @ k.abs().T * d ** -0.5).max()
    e = 136 * 2.0 ** -23 * S + 2.0 ** -21 * (1 + S)
    assert torch.all((out[0].double() - ref).abs() <= 2 * 2.0 ** -8 * A + 2.0 ** -8 * ref.abs() + 2 * e * A)
    # beside e, the sum of 131,071 weights: 900 of them one after another in a lane at the most
    assert torch.all((lse[:, 0].double() - s.logsumexp(-1)).abs() <= e + 1024 * 2.0 ** -24)


@pytest.mark.parametrize("keys,new,hq,hkv,d,words", [
    ([40000], [16], 32, 8, 64, 1),                        # over 30 units of one tile for each CTA
    ([900 + 37 * i for i in range(40)], [10] * 40, 16, 4, 128, 0),   # several tiles for each CTA, two rows of blocks
    ([70] * 300, [9] * 300, 16, 4, 64, 1),                # tiles of one or two units, many for each CTA
    ([5000, 4000], [300, 5], 4, 1, 128, 0),               # ten tiles over the same keys
])
def test_many_units_for_each_cta(keys, new, hq, hkv, d, words):
    x = make(keys, new, 16, hq, hkv, d, BF16, words=words)
    work = torch.zeros(vlp.thd_attn_paged_workspace_size(d), dtype=torch.uint8, device="cuda")
    got = run(x, max_seqlen_q=max(new), workspace=work)
    assert int(work[8:12].view(torch.int32).item()) == 0
    check(x, got)


def test_rows_of_no_sequence_and_no_pages():
    x = make([5], [2], 4, 4, 2, 64, BF16, gap=6)
    out = torch.full_like(x["q"], 9.0)
    lse = torch.full((4, len(out)), 9.0, device="cuda")
    check(x, run(x, out=out, lse=lse))
    for B in (0, 1):
        o, l = vlp.thd_attn_paged(x["q"], x["kc"][:0], x["vc"][:0], ints(np.zeros((1, 0))), ints([5]), ints([0, 2]),
                                  batch_size=B)
        assert torch.all(o == 0) and torch.all(torch.isneginf(l))
    o, l = vlp.thd_attn_paged(x["q"][:0], x["kc"], x["vc"], ints(x["table"]), ints([5]), ints([0, 0]))
    assert o.shape == (0, 4, 64) and l.shape == (4, 0)
    o, l = run(x, return_lse=False)
    assert l is None and torch.equal(o, out)


def test_bad_metadata_stays_in_the_buffers():
    x = make([50, 60, 70], [3, 4, 5], 8, 4, 2, 64, BF16)
    rng = np.random.default_rng(6)
    for _ in range(6):
        y = dict(x, table=rng.integers(-5, 60, x["table"].shape), keys=rng.integers(-10, 10**6, 3),
                 cu=rng.integers(-30, 30, 4))
        run(y)
    check(x, run(x))


def test_graph_replayed_with_other_lengths_and_another_stream():
    x = make([70, 900, 5], [2, 1, 3], 16, 8, 2, 128, BF16)
    y = make([300, 20, 64], [1, 4, 1], 16, 8, 2, 128, BF16, seed=1, extra=60)
    w = max(x["table"].shape[1], y["table"].shape[1])
    pages = max(len(x["kc"]), len(y["kc"]))
    held = dict(q=torch.zeros_like(x["q"]), kc=torch.zeros(pages, 16, 2, 128, dtype=BF16, device="cuda"),
                vc=torch.zeros(pages, 16, 2, 128, dtype=BF16, device="cuda"),
                table=torch.zeros(3, w, dtype=torch.int32, device="cuda"), keys=ints([0] * 3), cu=ints([0] * 4))
    work = torch.empty(vlp.thd_attn_paged_workspace_size(128), dtype=torch.uint8, device="cuda")
    call = lambda: vlp.thd_attn_paged(held["q"], held["kc"], held["vc"], held["table"], held["keys"], held["cu"],
                                      max_seqlen_q=4, workspace=work)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):   # two graphs that share the workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        graphs.append((graph, got))
    for z in (x, y, x):
        for name in ("q", "kc", "vc"):
            held[name][:len(z[name])].copy_(z[name])
        held["table"].fill_(-1)
        held["table"][:, :z["table"].shape[1]] = ints(z["table"])
        held["keys"].copy_(ints(z["keys"]))
        held["cu"].copy_(ints(z["cu"]))
        for graph, got in graphs:
            graph.replay()
            torch.cuda.synchronize()
            check(dict(z, q=held["q"]), got)


def test_two_streams_at_once():
    xs = [make([400 + i, 30], [1, 2], 16, 8, 2, 128, BF16, seed=i) for i in range(2)]
    want = [run(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    args = [(x["q"], x["kc"], x["vc"], ints(x["table"]), ints(x["keys"]), ints(x["cu"])) for x in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, s in zip(args, streams):
            with torch.cuda.stream(s):
                got.append(vlp.thd_attn_paged(*a))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_decoding_a_packed_batch_step_by_step():
    """Norm, rotation, append and attention over the cache give, token by token and as trees, what the
    packed operators give for the whole sequences."""
    d, hq, hkv, page = 64, 4, 2, 8
    lens = [13, 1, 30]
    g = torch.Generator().manual_seed(3)
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    x = torch.randn(T, (hq + 2 * hkv) * d, generator=g).to(BF16).cuda()
    split = lambda x: [p.unflatten(1, (-1, d)) for p in x.split([hq * d, hkv * d, hkv * d], 1)]
    q, k, v = split(x)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(BF16).cuda()
    angle = torch.arange(64, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    cos, sin = angle.cos().float().cuda(), angle.sin().float().cuda()
    qr, kr = vlp.thd_qk_norm_rope(q, k, ints(cu), cos, sin, q_weight=w, k_weight=w)
    want, want_lse = vlp.thd_attn_fwd(qr, kr, v.contiguous(), ints(cu), ints(cu),
                                      seq_is_causal=torch.ones(3, dtype=torch.bool, device="cuda"), max_seqlen=30)
    kc = torch.zeros(12, page, hkv, d, dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    table = ints([[0, 7, 2, 3], [5, 1, 1, 1], [4, 6, 8, 9]])
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    done = np.zeros(3, np.int64)
    for step, sizes in enumerate([(1, 1, 1), (4, 0, 5), (7, 0, 1), (1, 0, 20), (0, 0, 3)]):
        rows = np.concatenate([np.arange(cu[b] + done[b], cu[b] + done[b] + n) for b, n in enumerate(sizes)])
        rows = torch.tensor(rows).cuda()
        c = ints(np.concatenate([[0], np.cumsum(sizes)]))
        qs, ks, vs = split(x[rows])
        got = vlp.thd_kv_append(ks, vs, kc, vc, table, ints(done), c, q=qs, rope_cos=cos, rope_sin=sin, q_weight=w,
                                k_weight=w)
        assert torch.equal(got, qr[rows])
        tree = None
        if step % 2:   # a chain, as a tree
            tree = torch.cat([torch.tensor([(2 << i) - 1 for i in range(n)], dtype=torch.int64) for n in sizes])[:, None].cuda()
        done += sizes
        o, l = vlp.thd_attn_paged(got, kc, vc, table, ints(done), c, max_seqlen_q=max(sizes), tree_mask=tree)
        out[rows], lse[:, rows] = o, l
    assert list(done) == lens
    # both sides round weights and outputs to bf16 once: 2 * (2 u A + u |out|), A <= max |v|
    assert (out - want).abs().max() <= 2 * 3 * 2.0 ** -8 * v.abs().max()
    assert (lse - want_lse).abs().max() <= 1e-3


def test_binding_refusals():
    x = make([5], [2], 4, 4, 2, 64, BF16)
    q, kc, vc, t, n, cu = x["q"], x["kc"], x["vc"], ints(x["table"]), ints([5]), ints([0, 2])
    f = vlp.thd_attn_paged
    mask = torch.zeros(2, 1, dtype=torch.int64, device="cuda")
    bad = [
        (TypeError, lambda: f(q.float(), kc, vc, t, n, cu)), (TypeError, lambda: f(q, kc.half(), vc, t, n, cu)),
        (TypeError, lambda: f(q, kc, vc, t.long(), n, cu)), (TypeError, lambda: f(q, kc, vc, t, n.long(), cu)),
        (TypeError, lambda: f(q, kc, vc, t, None, cu)), (ValueError, lambda: f(q, kc, vc[:1], t, n, cu)),
        (ValueError, lambda: f(q[:, :, :32].contiguous(), kc, vc, t, n, cu)),
        (ValueError, lambda: f(q, kc, vc, t, n, cu, batch_size=2)), (ValueError, lambda: f(q, kc, vc, t, n[:0], cu)),
        (ValueError, lambda: f(q[:, ::2], kc, vc, t, n, cu)), (ValueError, lambda: f(q[0], kc, vc, t, n, cu)),
        (ValueError, lambda: f(q, kc.transpose(2, 3), vc.transpose(2, 3), t, n, cu)),
        (ValueError, lambda: f(q, kc, vc, t, n, cu, tree_mask=mask[:1])),
        (TypeError, lambda: f(q, kc, vc, t, n, cu, tree_mask=mask.int())),
        (ValueError, lambda: f(q, kc, vc, t, n, cu, out=q[:1])),
        (ValueError, lambda: f(q, kc, vc, t, n, cu, lse=torch.zeros(2, 4, device="cuda"))),
        (vlp.ThdError, lambda: f(q, kc, vc, t, n, cu, softmax_scale=-1.0)),
        (vlp.ThdError, lambda: f(q[:, :3].contiguous(), kc, vc, t, n, cu)),
        (vlp.ThdError, lambda: f(q, kc, vc, t, n, cu, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))),
        (vlp.ThdError, lambda: f(q, kc, vc, t, n, cu, max_seqlen_q=-1)),
    ]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was not refused")


def test_counts_past_32_bits_are_refused():
    """A cache expanded to more pages than the library counts: refused, not cut to what fits 32 bits."""
    x = make([5], [2], 4, 4, 2, 64, BF16)
    kc, vc = (x[c][:1].expand(2 ** 32 + 1, -1, -1, -1) for c in ("kc", "vc"))
    q, t, n, cu = x["q"], ints(x["table"]), ints([5]), ints([0, 2])
    with pytest.raises(ValueError, match="32 bits"):
        vlp.thd_attn_paged(q, kc, vc, t, n, cu)
    table = torch.empty((1, 2 ** 31), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        vlp.thd_attn_paged(q, x["kc"], x["vc"], table, n, cu)
    with pytest.raises(ValueError, match="32 bits"):
        vlp.thd_kv_append(q[:, :2].contiguous(), q[:, :2].contiguous(), x["kc"], x["vc"], table, n, cu)


def test_a_wait_that_runs_out_is_reported():
    """Wide tiles wait on barriers: with an injected wait and a short limit the call comes back with the
    status bit set, and the next call is as if nothing had been."""
    x = make([300, 500], [40, 33], 16, 8, 2, 128, BF16, words=1)
    work = torch.zeros(vlp.thd_attn_paged_workspace_size(128), dtype=torch.uint8, device="cuda")
    want = run(x, workspace=work, max_seqlen_q=40)
    status = lambda: int(work[8:12].view(torch.int32).item())
    assert status() == 0
    vlp.thd_set_wait_limit_ns(1)
    vlp.thd_set_wait_injection(True)
    try:
        run(x, workspace=work, max_seqlen_q=40)
        assert status() == vlp.STATUS_WAIT_TIMEOUT
    finally:
        vlp.thd_set_wait_injection(False)
        vlp.thd_set_wait_limit_ns(0)
    got = run(x, workspace=work, max_seqlen_q=40)
    assert status() == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(x, got)
