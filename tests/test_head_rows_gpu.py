"""GPU tests of the head norm and rotation, its gradients, and the append to a paged cache, against
the fp64 oracle.

Tolerances.  The kernels compute in fp32 and round once to 16 bits, half a step: u = finfo.eps / 2
relative to the value, or half the least subnormal.  Before that a value is a sum of terms of which
each passed fewer than 32 fp32 roundings (the mean of up to 128 squares in a tree, rsqrt, products,
the rotation), each at most 2^-24 of the size of the terms: 2^-19 of it.  A weight gradient sums
over the rows one after another in a lane, then in trees: (rows per lane + 64) * 2^-24 of the sizes.
"""
import numpy as np
import pytest
import torch

from oracle import rows as oracle_rows

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")

BF16, FP16 = torch.bfloat16, torch.float16
LEAST = {BF16: 2.0 ** -133, FP16: 2.0 ** -24}


def f64(t):
    return t.detach().float().cpu().double().numpy()


def assert_near(got, ref, size, dtype, what):
    got = f64(got)
    bound = torch.finfo(dtype).eps / 2 * np.abs(ref) * 1.0001 + 2.0 ** -19 * size + LEAST[dtype] / 2
    worst = np.max(np.abs(got - ref) / bound) if ref.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


def tables(n, rotary, base=10000.0):
    angle = np.arange(n)[:, None] * base ** (-np.arange(0, rotary, 2) / rotary)
    return torch.tensor(np.cos(angle), dtype=torch.float32).cuda(), torch.tensor(np.sin(angle), dtype=torch.float32).cuda()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def batch(lens, gap, rng):
    """cu, padded starts (or None), rows of the buffer."""
    cu = np.concatenate([[0], np.cumsum(lens)])
    if not gap:
        return cu, None, int(cu[-1])
    starts, at = [], 0
    for n in lens:
        at += int(rng.integers(0, gap + 1))
        starts.append(at)
        at += n
    return cu, np.array(starts), at + gap


def draw(shape, dtype, g, fused=False):
    """Row tensors [T, h, d] for each h of `heads`, apart or parts of one buffer."""
    T, heads, d = shape
    if not fused:
        return [torch.randn(T, h, d, generator=g).to(dtype).cuda() for h in heads]
    x = torch.randn(T, sum(heads) * d, generator=g).to(dtype).cuda()
    return [p.unflatten(1, (h, d)) for p, h in zip(x.split([h * d for h in heads], 1), heads)]


CASES = [
    # lens, gap, hq, hkv, d, rotary, dtype, norm, interleaved, fused, w32, offsets
    ([1], 0, 1, 1, 16, 16, BF16, True, False, False, False, False),
    ([5, 0, 1, 17], 0, 8, 2, 128, 128, BF16, True, False, False, False, False),
    ([5, 0, 1, 17], 4, 8, 2, 128, 128, FP16, True, True, True, False, True),
    ([3, 40, 2], 3, 5, 5, 64, 32, BF16, True, False, True, True, True),
    ([33], 0, 6, 3, 48, 16, FP16, False, False, False, False, False),
    ([2, 0, 0, 9], 6, 3, 1, 80, 48, BF16, True, True, True, False, False),
    ([7, 7], 1, 17, 4, 96, 96, BF16, False, True, False, False, True),
    ([4, 12], 0, 2, 0, 112, 64, FP16, True, False, False, True, False),
    ([1] * 40 + [0] * 37 + [3] * 5, 2, 4, 2, 32, 0, BF16, True, False, False, False, False),
    # many heads: items of one row each
    ([5, 0, 9], 4, 32, 8, 128, 128, BF16, True, False, True, False, False),
    ([11, 6], 0, 33, 16, 112, 64, FP16, True, True, False, True, True),
    ([7, 3, 0, 0, 2], 2, 32, 32, 64, 48, BF16, True, False, False, False, True),
    ([40], 0, 48, 24, 32, 32, FP16, False, True, False, False, False),
    ([9], 3, 96, 64, 16, 16, BF16, True, False, True, False, False),
    # few heads: rows of several sequences, and of none, in one item
    ([1, 2, 1, 0, 3, 1, 1, 30], 3, 1, 1, 128, 128, BF16, True, False, False, False, True),
    ([2] * 70, 1, 2, 1, 64, 32, FP16, True, True, True, False, False),
]


def make(case, seed=0):
    lens, gap, hq, hkv, d, rot, dtype, norm, inter, fused, w32, offs = case
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    cu, padded, T = batch(lens, gap, rng)
    q, k = draw((T, [hq, max(hkv, 1)], d), dtype, g, fused)
    k = k if hkv else None
    wd = torch.float32 if w32 else dtype
    wq = (1 + 0.3 * torch.randn(d, generator=g)).to(wd).cuda() if norm else None
    wk = (1 + 0.3 * torch.randn(d, generator=g)).to(wd).cuda() if norm and hkv else None
    cos, sin = tables(max(lens) + 50, rot) if rot else (None, None)
    offsets = rng.integers(0, 40, len(lens)) if offs else None
    kw = dict(cu_seqlens_padded=None if padded is None else ints(padded), batch_size=len(lens),
              position_offsets=None if offsets is None else ints(offsets), q_weight=wq, k_weight=wk, eps=1e-5,
              interleaved=inter)
    return q, k, cu, padded, offsets, wq, wk, cos, sin, kw


def cpu(t):
    return None if t is None else t.detach().float().cpu().numpy()


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_norm_rope(case):
    q, k, cu, padded, offsets, wq, wk, cos, sin, kw = make(case)
    got = vlp.thd_qk_norm_rope(q, k, ints(cu), cos, sin, **kw)
    torch.cuda.synchronize()
    for name, x, w, y in (("q", q, wq, got[0]), ("k", k, wk, got[1])):
        if x is None:
            assert y is None
            continue
        ref, size = oracle_rows.norm_rope(f64(x), cpu(w), 1e-5, cpu(cos), cpu(sin), kw["interleaved"], cu, padded,
                                          len(case[0]), offsets)
        assert_near(y, ref, size, x.dtype, name)


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_norm_rope_gradients(case):
    q, k, cu, padded, offsets, wq, wk, cos, sin, kw = make(case)
    g = torch.Generator().manual_seed(7)
    gq = torch.randn(q.shape, generator=g).to(q.dtype).cuda()
    gk = None if k is None else torch.randn(k.shape, generator=g).to(q.dtype).cuda()
    got = vlp.thd_qk_norm_rope_bwd(gq, gk, q, k, ints(cu), cos, sin, **kw)
    again = vlp.thd_qk_norm_rope_bwd(gq, gk, q, k, ints(cu), cos, sin, **kw)
    torch.cuda.synchronize()
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)
    for name, x, w, gr, dx, dw in (("q", q, wq, gq, got[0], got[2]), ("k", k, wk, gk, got[1], got[3])):
        if x is None:
            assert dx is None and dw is None
            continue
        ref, size, wref, wsize = oracle_rows.norm_rope_bwd(f64(gr), f64(x), cpu(w), 1e-5, cpu(cos), cpu(sin),
                                                           kw["interleaved"], cu, padded, len(case[0]), offsets)
        assert_near(dx, ref, size, x.dtype, "d" + name)
        if w is None:
            assert dw is None
        else:
            bound = (len(x) + 64) * 2.0 ** -24 * wsize + 1e-30
            assert np.all(np.abs(f64(dw) - wref) <= bound), name


def test_gradients_into_a_fused_buffer_and_in_place():
    q, k, cu, padded, offsets, wq, wk, cos, sin, kw = make(CASES[2], seed=3)
    T, hq, d = q.shape
    g = torch.Generator().manual_seed(8)
    gq, gk = draw((T, [hq, k.shape[1]], d), q.dtype, g)
    want = vlp.thd_qk_norm_rope_bwd(gq, gk, q, k, ints(cu), cos, sin, **kw)
    whole = torch.full((T, (hq + 2 * k.shape[1]) * d), 7.0, dtype=q.dtype, device="cuda")
    parts = [p.unflatten(1, (-1, d)) for p in whole.split([hq * d, k.shape[1] * d, k.shape[1] * d], 1)]
    got = vlp.thd_qk_norm_rope_bwd(gq, gk, q, k, ints(cu), cos, sin, dq=parts[0], dk=parts[1], **kw)
    assert got[0] is parts[0] and torch.equal(parts[0], want[0]) and torch.equal(parts[1], want[1])
    assert torch.all(parts[2] == 7.0)
    vlp.thd_qk_norm_rope_bwd(gq, gk, q, k, ints(cu), cos, sin, dq=gq, dk=gk, **kw)
    assert torch.equal(gq, want[0]) and torch.equal(gk, want[1])
    qc, kc = q.contiguous(), k.contiguous()
    want = vlp.thd_qk_norm_rope(q, k, ints(cu), cos, sin, **kw)
    vlp.thd_qk_norm_rope(qc, kc, ints(cu), cos, sin, q_out=qc, k_out=kc, **kw)
    assert torch.equal(qc, want[0]) and torch.equal(kc, want[1])


def test_no_rows_gives_zero_weight_gradients():
    w = torch.ones(64, dtype=BF16, device="cuda")
    x = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    dq, dk, dwq, dwk = vlp.thd_qk_norm_rope_bwd(x, x, x, x, ints([0]), batch_size=0, q_weight=w, k_weight=w)
    assert dq.shape == x.shape and torch.all(dwq == 0) and torch.all(dwk == 0)
    x = torch.randn(6, 4, 64, device="cuda").to(BF16)   # rows, but no sequence
    dq, dk, dwq, dwk = vlp.thd_qk_norm_rope_bwd(x, x, x, x, ints([0]), batch_size=0, q_weight=w, k_weight=w)
    assert torch.all(dq == 0) and torch.all(dk == 0) and torch.all(dwq == 0)
    y, _ = vlp.thd_qk_norm_rope(x, None, ints([0]), batch_size=0, q_weight=w)
    assert torch.all(y == 0)


def test_zero_heads_zero_eps_and_far_positions():
    """eps = 0 with a part-filled pass (5 heads of 128), and positions past and before the tables."""
    x = torch.randn(3, 5, 128, device="cuda").to(BF16)
    w = torch.ones(128, dtype=BF16, device="cuda")
    cos, sin = tables(4, 128)
    out = vlp.thd_qk_norm_rope_bwd(x, x, x, x, ints([0, 3]), cos, sin, q_weight=w, k_weight=w, eps=0.0)
    assert all(torch.isfinite(t).all() for t in out)
    for off in (-7, 2**31 - 2):
        y, _ = vlp.thd_qk_norm_rope(x, None, ints([0, 3]), cos, sin, position_offsets=ints([off]))
        ref, size = oracle_rows.norm_rope(f64(x), None, 0.0, cpu(cos), cpu(sin), False, [0, 3], None, 1, [off])
        assert_near(y, ref, size, BF16, "clamped")


def test_empty_sequences_that_share_a_start():
    """A sequence without rows may have the start of the one before it."""
    x = torch.randn(12, 2, 64, device="cuda").to(BF16)
    cos, sin = tables(12, 64)
    for cu, padded in (([0, 5, 5, 8], [0, 0, 8]), ([0, 5] + [5] * 70 + [8], [0] + [0] * 70 + [8]),
                       ([0, 4, 4, 4], [1, 12, 12])):
        B = len(padded)
        y, _ = vlp.thd_qk_norm_rope(x, None, ints(cu), cos, sin, cu_seqlens_padded=ints(padded), batch_size=B)
        ref, size = oracle_rows.norm_rope(f64(x), None, 0.0, cpu(cos), cpu(sin), False, cu, padded, B)
        assert_near(y, ref, size, BF16, str(padded))


def test_metadata_out_of_order_does_not_fault():
    x = torch.randn(50, 3, 64, device="cuda").to(BF16)
    cos, sin = tables(16, 64)
    rng = np.random.default_rng(0)
    for _ in range(5):
        cu, pad = rng.integers(-100, 200, 41), rng.integers(-100, 200, 40)
        vlp.thd_qk_norm_rope(x, x, ints(cu), cos, sin, cu_seqlens_padded=ints(pad), batch_size=40)
    torch.cuda.synchronize()


def test_training_step_through_packed_attention():
    """Norm and rotation, attention and both backward passes in a row, out of and into fused buffers, against
    torch autograd of the whole in 64 bits.  Six tensors are rounded to bf16 on the way (heads, weights, output,
    dS, gradients of the heads, gradients), each by at most 2^-8 of itself; with the steps' relative condition
    taken as 2: 12 * 2^-8 of the norm."""
    lens, hq, hkv, d = [40, 1, 23, 0, 70], 4, 2, 64
    rng, g = np.random.default_rng(5), torch.Generator().manual_seed(5)
    cu, padded, T = batch(lens, 3, rng)
    x = torch.randn(T, (hq + 2 * hkv) * d, generator=g).to(BF16).cuda()
    split = lambda x: [p.unflatten(1, (-1, d)) for p in x.split([hq * d, hkv * d, hkv * d], 1)]
    q, k, v = split(x)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(BF16).cuda() for _ in range(2))
    cos, sin = tables(max(lens), d, 100.0)
    dout = torch.randn(T, hq, d, generator=g).to(BF16).cuda()
    c, p, B = ints(cu), ints(padded), len(lens)
    causal = torch.ones(B, dtype=torch.bool, device="cuda")
    kw = dict(cu_seqlens_padded=p, batch_size=B, q_weight=wq, k_weight=wk)
    qr, kr = vlp.thd_qk_norm_rope(q, k, c, cos, sin, **kw)
    vc = v.contiguous()
    out, lse = vlp.thd_attn_fwd(qr, kr, vc, c, c, p, p, causal, B, max(lens))
    gq, gk, gv = vlp.thd_attn_bwd(qr, kr, vc, out, lse, dout, c, c, p, p, causal, B, max(lens))
    dx = torch.zeros_like(x)
    parts = split(dx)
    _, _, dwq, dwk = vlp.thd_qk_norm_rope_bwd(gq, gk, q, k, c, cos, sin, dq=parts[0], dk=parts[1], **kw)
    parts[2].copy_(gv)

    leaf = x.double().requires_grad_()
    w = [t.double().requires_grad_() for t in (wq, wk)]
    heads, total = split(leaf), 0.0
    for start, n in zip(padded, lens):
        rows = slice(int(start), int(start) + n)
        turned = []
        for t, weight in zip(heads[:2], w):
            h = t[rows]
            h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * weight
            a, b = h[..., :d // 2], h[..., d // 2:]
            cc, ss = cos[:n, None].double(), sin[:n, None].double()
            turned.append(torch.cat([a * cc - b * ss, b * cc + a * ss], -1))
        qh = turned[0].transpose(0, 1)
        kh, vh = (t.repeat_interleave(hq // hkv, 1).transpose(0, 1) for t in (turned[1], heads[2][rows]))
        s = (qh @ kh.transpose(1, 2) * d ** -0.5).masked_fill(
            torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
        total = total + ((s.softmax(-1) @ vh).transpose(0, 1) * dout[rows].double()).sum()
    total.backward()
    for name, got, want in (("dx", dx, leaf.grad), ("dwq", dwq, w[0].grad), ("dwk", dwk, w[1].grad)):
        rel = float((got.double() - want).norm() / want.norm())
        print(f"{name}: {rel:.2e}")
        assert rel <= 12 * 2.0 ** -8, (name, rel)
    gone = torch.ones(T, dtype=torch.bool)
    for start, n in zip(padded, lens):
        gone[int(start):int(start) + n] = False
    assert torch.all(dx[gone.cuda()] == 0)


def test_rows_captured_and_replayed_with_other_lengths():
    """A captured forward, backward and append, replayed after the lengths and inputs changed, on another stream."""
    T, hq, hkv, d = 24, 8, 2, 128
    g = torch.Generator().manual_seed(6)
    x, k = draw((T, [hq, hkv], d), BF16, g)
    gq, gk = draw((T, [hq, hkv], d), BF16, g)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(BF16).cuda()
    cos, sin = tables(64, d)
    cu, lens, table = ints([0, 10, 24]), ints([3, 0]), ints([[2, 0, 1], [5, 4, 3]])
    kc = torch.zeros(6, 16, hkv, d, dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    call = lambda: (vlp.thd_qk_norm_rope(x, k, cu, cos, sin, q_weight=w, k_weight=w),
                    vlp.thd_qk_norm_rope_bwd(gq, gk, x, k, cu, cos, sin, q_weight=w, k_weight=w),
                    vlp.thd_kv_append(k, k, kc, vc, table, lens, cu, q=x, rope_cos=cos, rope_sin=sin, k_weight=w))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for sizes, before in (([0, 24, 24], [20, 1]), ([0, 1, 9], [0, 7])):
        cu.copy_(ints(sizes))
        lens.copy_(ints(before))
        x.copy_(draw((T, [hq], d), BF16, g)[0])
        kc.zero_(), vc.zero_()
        want = call()
        caches = kc.clone(), vc.clone()
        kc.zero_(), vc.zero_()
        with torch.cuda.stream(torch.cuda.Stream()):
            torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
            graph.replay()
            torch.cuda.current_stream().synchronize()
        flat = lambda r: [*r[0], *r[1], r[2]]
        assert all(torch.equal(a, b) for a, b in zip(flat(got), flat(want)))
        assert torch.equal(kc, caches[0]) and torch.equal(vc, caches[1])


# ------------------------------------------------------------------------------ append
APPENDS = [
    # before, new, gap, page, hq, hkv, d, rotary, dtype, norm, interleaved, fused, positions, heads first
    ([0], [1], 0, 1, 1, 1, 16, 16, BF16, False, False, False, False, False),
    ([13, 0, 7, 30], [1, 1, 1, 1], 0, 16, 8, 2, 128, 128, BF16, False, False, False, False, False),
    ([13, 0, 7], [9, 0, 21], 3, 8, 4, 4, 64, 64, FP16, True, True, True, True, True),
    ([3, 500], [20, 5], 2, 24, 6, 3, 80, 32, BF16, True, False, True, False, False),
    ([1, 2, 3], [4, 5, 6], 0, 7, 0, 2, 96, 0, FP16, False, False, False, False, True),
    ([6, 40, 0], [3, 1, 12], 2, 16, 32, 8, 128, 128, BF16, True, False, True, False, False),
    ([6, 40], [9, 8], 0, 8, 16, 16, 64, 32, FP16, True, True, False, True, True),
    ([5, 1, 90], [1, 30, 2], 3, 4, 1, 1, 128, 128, BF16, True, False, False, True, False),
]


@pytest.mark.parametrize("case", APPENDS, ids=[str(i) for i in range(len(APPENDS))])
def test_append(case):
    before, new, gap, page, hq, hkv, d, rot, dtype, norm, inter, fused, given, first = case
    rng, g = np.random.default_rng(1), torch.Generator().manual_seed(1)
    cu, padded, T = batch(new, gap, rng)
    q, k, v = draw((T, [max(hq, 1), hkv, hkv], d), dtype, g, fused)
    q = q if hq else None
    B = len(new)
    need = [-(-(a + b) // page) for a, b in zip(before, new)]
    pages = sum(need) + 2
    order = rng.permutation(pages)
    table = np.full((B, max(need) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    if B > 2:
        table[1, 0] = pages          # a page that the cache does not have
    kv = [torch.randn(pages, hkv, page, d, generator=g).to(dtype).cuda().transpose(1, 2) if first else
          torch.randn(pages, page, hkv, d, generator=g).to(dtype).cuda() for _ in range(2)]
    old = [f64(x) for x in kv]
    wq = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda() if norm and hq else None
    wk = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda() if norm else None
    cos, sin = tables(max(before) + max(new) + 9, rot) if rot else (None, None)
    positions = rng.integers(0, 9, T) if given else None
    wide = torch.full((B, table.shape[1] + 5), 10**9, dtype=torch.int32)
    wide[:, :table.shape[1]] = torch.tensor(table)
    got = vlp.thd_kv_append(k, v, kv[0], kv[1], wide.cuda()[:, :table.shape[1]], ints(before), ints(cu),
                            cu_seqlens_padded=None if padded is None else ints(padded), batch_size=B, q=q, rope_cos=cos,
                            rope_sin=sin, positions=None if positions is None else ints(positions), q_weight=wq,
                            k_weight=wk, eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    c, s = (None, None) if cos is None else (cpu(cos).astype(np.float64), cpu(sin).astype(np.float64))
    angle = lambda t, slot: (None, None) if c is None else oracle_rows._table_row(c, s, int(positions[t]) if given else slot)
    want, size, vals = old[0].copy(), np.zeros_like(old[0]), old[1].copy()
    exact = np.ones(old[0].shape[:2], bool)
    for t, pg, off, slot in oracle_rows.append_slots(table, before, page, pages, cu, padded, B):
        want[pg, off], size[pg, off] = oracle_rows.norm_rope_row(f64(k[t]), None if wk is None else f64(wk), 1e-5,
                                                                 *angle(t, slot), inter)
        vals[pg, off] = f64(v[t])
        exact[pg, off] = False
    assert np.array_equal(f64(kv[1]), vals)
    assert np.array_equal(f64(kv[0])[exact], old[0][exact])
    assert_near(kv[0], want, size, dtype, "k")
    if q is None:
        assert got is None
        return
    ref, rsize = np.zeros(q.shape), np.zeros(q.shape)
    for t, b, i in oracle_rows.row_places(cu, padded, B):
        ref[t], rsize[t] = oracle_rows.norm_rope_row(f64(q[t]), None if wq is None else f64(wq), 1e-5,
                                                     *angle(t, before[b] + i), inter)
    assert_near(got, ref, rsize, dtype, "q")


def test_append_past_the_table_writes_nothing():
    x = torch.randn(4, 2, 64, device="cuda").to(BF16)
    kc = torch.zeros(3, 4, 2, 64, dtype=BF16, device="cuda")
    vc = kc.clone()
    for lens in ([8], [-5], [2**31 - 2]):
        vlp.thd_kv_append(x, x, kc, vc, ints([[0, 1]]), ints(lens), ints([0, 4]))
        torch.cuda.synchronize()
        assert torch.all(kc == 0) and torch.all(vc == 0)
    vlp.thd_kv_append(x, x, kc, vc, ints([[-1, 2]]), ints([2]), ints([0, 4]))   # two without a page, two in page 2
    assert torch.equal(kc[2, :2], x[2:]) and torch.all(kc[:2] == 0) and torch.all(kc[2, 2:] == 0)
    one = torch.zeros(3, 2, 4, 2, 64, dtype=BF16, device="cuda")   # keys and values in one buffer
    vlp.thd_kv_append(x, 2 * x, one[:, 0], one[:, 1], ints([[1]]), ints([0]), ints([0, 4]))
    assert torch.equal(one[1, 0], x) and torch.equal(one[1, 1], 2 * x) and torch.all(one[[0, 2]] == 0)


def test_append_past_two_to_the_31_elements():
    x = torch.randn(3, 1, 128, device="cuda").to(BF16)
    kc = torch.zeros((1 << 20) + 2, 16, 1, 128, dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    last = (1 << 20) + 1
    vlp.thd_kv_append(x, 2 * x, kc, vc, ints([[last, 7]]), ints([14]), ints([0, 3]))
    assert torch.equal(kc[last, 14:], x[:2]) and torch.equal(vc[last, 14:], 2 * x[:2])
    assert torch.equal(kc[7, :1], x[2:]) and torch.equal(vc[7, :1], 2 * x[2:])
    assert int(kc.count_nonzero()) == int(x.count_nonzero())


def test_binding_refusals():
    x = torch.zeros(4, 2, 64, dtype=BF16, device="cuda")
    cu, w = ints([0, 4]), torch.ones(64, dtype=BF16, device="cuda")
    cos, sin = tables(8, 64)
    bad = [
        (TypeError, lambda: vlp.thd_qk_norm_rope(x.float(), x, cu)),
        (TypeError, lambda: vlp.thd_qk_norm_rope(x, x.half(), cu)),
        (ValueError, lambda: vlp.thd_qk_norm_rope(x, x[:3], cu)),
        (ValueError, lambda: vlp.thd_qk_norm_rope(x.transpose(0, 1), x, cu)),
        (ValueError, lambda: vlp.thd_qk_norm_rope(x[:1].expand(4, 2, 64), x, cu)),
        (ValueError, lambda: vlp.thd_qk_norm_rope(x, x, cu, batch_size=2)),
        (ValueError, lambda: vlp.thd_qk_norm_rope(x, x, cu, cos)),
        (ValueError, lambda: vlp.thd_qk_norm_rope(x, x, cu, cos, sin[:4])),
        (ValueError, lambda: vlp.thd_qk_norm_rope(x, x, cu, *tables(8, 96))),
        (TypeError, lambda: vlp.thd_qk_norm_rope(x, x, cu.long())),
        (TypeError, lambda: vlp.thd_qk_norm_rope(x, x, cu, q_weight=w.half())),
        (TypeError, lambda: vlp.thd_qk_norm_rope(x, x, cu, q_weight=w, k_weight=w.float())),
        (ValueError, lambda: vlp.thd_qk_norm_rope(x, x, cu, q_weight=w[:32])),
        (ValueError, lambda: vlp.thd_qk_norm_rope(x, x, cu, q_out=x[:2])),
        (ValueError, lambda: vlp.thd_qk_norm_rope(x, None, cu, k_weight=w)),
        (ValueError, lambda: vlp.thd_qk_norm_rope(x, x, cu, position_offsets=cu[:0])),
        (vlp.ThdError, lambda: vlp.thd_qk_norm_rope(x, x, cu, *tables(8, 24))),
        (vlp.ThdError, lambda: vlp.thd_qk_norm_rope(x, x, cu, q_weight=w, eps=-1.0)),
        (ValueError, lambda: vlp.thd_qk_norm_rope_bwd(x, x, x, x, cu, dq_weight=w)),
        (ValueError, lambda: vlp.thd_qk_norm_rope_bwd(x, x[:3], x, x, cu)),
        (ValueError, lambda: vlp.thd_qk_norm_rope_bwd(x, x, x[:3], x, cu, q_weight=w)),
        (vlp.ThdError, lambda: vlp.thd_qk_norm_rope_bwd(x, x, x, x, cu, q_weight=w,
                                                        workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
    ]
    c = torch.zeros(3, 4, 2, 64, dtype=BF16, device="cuda")
    t = ints([[0, 1]])
    bad += [
        (ValueError, lambda: vlp.thd_kv_append(x, x, c, c[:2], t, cu, cu)),
        (ValueError, lambda: vlp.thd_kv_append(x, x, c[:, :, :1], c[:, :, :1], t, cu, cu)),
        (ValueError, lambda: vlp.thd_kv_append(x, x, c[:1].expand(3, 4, 2, 64), c, t, cu, cu)),
        (ValueError, lambda: vlp.thd_kv_append(x, x, c, c, t[0], cu, cu)),
        (TypeError, lambda: vlp.thd_kv_append(x, x, c, c, t.long(), cu, cu)),
        (TypeError, lambda: vlp.thd_kv_append(x, x, c, c, t, None, cu)),
        (ValueError, lambda: vlp.thd_kv_append(x, x, c, c, t, cu, cu, positions=cu)),
        (ValueError, lambda: vlp.thd_kv_append(x, x, c, c, t, cu, cu, q_out=x)),
        (ValueError, lambda: vlp.thd_kv_append(x, x, c, c, ints([[0, 9, 1, 9]])[:, ::2], cu, cu)),
    ]
    for i, (error, f) in enumerate(bad):
        with pytest.raises(error):
            f()
            pytest.fail(f"call {i} was not refused")
