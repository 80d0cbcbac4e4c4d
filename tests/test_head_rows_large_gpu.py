"""GPU tests of the head norm and rotation, its gradients, and the append at sizes where a warp takes several
items one after another: stages of the shared-memory ring filled again, angles kept over a row's blocks of
heads, rows of many sequences and of none in one run, weight gradients over several items.

The reference is the operators' definition in 64 bits, in torch operations on the GPU.  Tolerances as
in test_head_rows_gpu.py: u |ref|, half a step of the 16-bit type, and 2^-19 of the size of a value's
terms.  A weight gradient is at most 36 terms one after another in a lane (the longest run here is 18 items of
two heads each lane), 9 over lanes and warps, 32 and 7 over the blocks, each term with fewer than 32
roundings of its own: 128 * 2^-24 of the sizes.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")

BF16, FP16 = torch.bfloat16, torch.float16
LEAST = {BF16: 2.0 ** -133, FP16: 2.0 ** -24}
EPS = 1e-5

CASES = [
    # sequences, rows, gap, hq, hkv, d, rotary, dtype, norm, interleaved, fused, offsets
    (40, 30000, 9, 32, 8, 128, 128, BF16, True, False, True, False),      # two blocks of query heads; gradients: runs of 10
    (9000, 30000, 3, 32, 8, 128, 128, BF16, True, False, False, True),    # a new sequence every few rows
    (500, 40000, 5, 40, 36, 64, 32, FP16, True, True, True, True),        # two blocks of each kind, part of a head turned
    (300, 60000, 40, 17, 16, 96, 96, BF16, False, False, False, False),   # rotation alone, a block of one head
    (64, 70000, 0, 33, 8, 48, 16, FP16, True, False, False, False),
    (20000, 70000, 2, 8, 1, 128, 128, BF16, True, False, True, False),    # few heads: whole rows to an item
    (700, 70000, 4, 2, 2, 64, 64, FP16, True, True, False, True),
]


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


class Batch:
    """Uneven lengths (empty sequences among them), gaps, and the sequence and place of each buffer row."""

    def __init__(self, seqs, rows, gap, rng):
        cuts = np.sort(rng.integers(0, rows + 1, seqs - 1))
        self.lens = np.diff(np.concatenate([[0], cuts, [rows]]))
        self.cu = np.concatenate([[0], np.cumsum(self.lens)])
        starts = self.cu[:-1] + np.cumsum(rng.integers(0, gap + 1, seqs)) if gap else self.cu[:-1]
        self.T = int(starts[-1] + self.lens[-1] + (gap if gap else 0))
        self.padded = ints(starts) if gap else None
        seq = np.repeat(np.arange(seqs), self.lens)
        place = np.arange(rows) - self.cu[seq]
        self.seqs, self.seq, self.place = seqs, torch.tensor(seq).cuda(), torch.tensor(place).cuda()
        self.rows = torch.tensor(starts[seq] + place).cuda()
        self.outside = torch.ones(self.T, dtype=torch.bool, device="cuda")
        self.outside[self.rows] = False


def row_tensors(T, heads, d, dtype, g, fused):
    if not fused:
        return [torch.randn(T, h, d, generator=g, device="cuda").to(dtype) for h in heads]
    x = torch.randn(T, sum(heads) * d, generator=g, device="cuda").to(dtype)
    return [p.unflatten(1, (h, d)) for p, h in zip(x.split([h * d for h in heads], 1), heads)]


def tables(n, rotary, base=10000.0):
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * base ** (
        -torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    return angle.cos().float(), angle.sin().float()


def turned(x, cos, sin, pos, interleaved, back=False):
    """Rows x [n, h, d] in 64 bits turned by their positions' angles, and the size of each value's terms."""
    if cos is None:
        return x, x.abs()
    at = pos.clamp(0, len(cos) - 1)
    c, s = cos.double()[at][:, None], sin.double()[at][:, None] * (-1 if back else 1)
    half = cos.shape[1]
    i = torch.arange(half, device="cuda") * (2 if interleaved else 1)
    j = i + 1 if interleaved else i + half
    y, size = x.clone(), x.abs()
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    size[..., i] = (x[..., i] * c).abs() + (x[..., j] * s).abs()
    size[..., j] = (x[..., j] * c).abs() + (x[..., i] * s).abs()
    return y, size


def normed(x, w):
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()


def assert_near(got, ref, size, what):
    dtype = got.dtype
    bound = torch.finfo(dtype).eps / 2 * ref.abs() * 1.0001 + 2.0 ** -19 * size + LEAST[dtype] / 2
    worst = float(((got.double() - ref).abs() / bound).nan_to_num(nan=1e30).max())
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


def setup(case, seed=0):
    seqs, rows, gap, hq, hkv, d, rot, dtype, norm, inter, fused, offs = case
    rng = np.random.default_rng(seed)
    g = torch.Generator("cuda").manual_seed(seed)
    b = Batch(seqs, rows, gap, rng)
    q, k, v = row_tensors(b.T, [hq, hkv, hkv], d, dtype, g, fused)
    for x in (q, k, v):   # rows of no sequence are not looked at
        x[b.outside] = float("nan")
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype) if norm else None for _ in range(2))
    offsets = ints(rng.integers(0, 40, seqs)) if offs else None
    cos, sin = tables(int(b.lens.max()) + 30, rot)
    pos = b.place + (offsets.long()[b.seq] if offs else 0)
    kw = dict(cu_seqlens_padded=b.padded, batch_size=seqs, position_offsets=offsets, q_weight=wq, k_weight=wk, eps=EPS,
              interleaved=inter)
    return b, q, k, v, wq, wk, cos, sin, pos, kw, g


def whole(b, x, fill=0.0):
    """Values of the batch's rows in a buffer of all rows."""
    y = torch.full((b.T, *x.shape[1:]), fill, dtype=x.dtype, device="cuda")
    y[b.rows] = x
    return y


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_norm_rope_over_many_items(case):
    b, q, k, _, wq, wk, cos, sin, pos, kw, _ = setup(case)
    got = vlp.thd_qk_norm_rope(q, k, ints(b.cu), cos, sin, **kw)
    for name, x, w, y in (("q", q, wq, got[0]), ("k", k, wk, got[1])):
        ref, size = turned(normed(x[b.rows].double(), w), cos, sin, pos, kw["interleaved"])
        assert_near(y, whole(b, ref), whole(b, size), name)


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_gradients_over_many_items(case):
    b, q, k, _, wq, wk, cos, sin, pos, kw, g = setup(case)
    gq, gk = row_tensors(b.T, [q.shape[1], k.shape[1]], q.shape[2], q.dtype, g, False)
    gq[b.outside], gk[b.outside] = float("nan"), float("inf")
    args = (gq, gk, q, k, ints(b.cu), cos, sin)
    got = vlp.thd_qk_norm_rope_bwd(*args, **kw)
    again = vlp.thd_qk_norm_rope_bwd(*args, **kw)
    assert all(x is None and y is None or torch.equal(x, y) for x, y in zip(got, again))
    for name, gr, x, w, dx, dw in (("q", gq, q, wq, got[0], got[2]), ("k", gk, k, wk, got[1], got[3])):
        h, hs = turned(gr[b.rows].double(), cos, sin, pos, kw["interleaved"], back=True)
        if w is None:
            assert_near(dx, whole(b, h), whole(b, hs), "d" + name)
            continue
        v = x[b.rows].double()
        r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        unit = v * r
        ref, size = (h * unit).sum((0, 1)), (hs * unit.abs()).sum((0, 1))
        assert torch.all((dw.double() - ref).abs() <= 128 * 2.0 ** -24 * size), name
        u, us = h * w.double(), hs * w.double().abs()
        ref = r * (u - unit * (u * unit).mean(-1, keepdim=True))
        size = r * (us + unit.abs() * (us * unit.abs()).mean(-1, keepdim=True))
        assert_near(dx, whole(b, ref), whole(b, size), "d" + name)


@pytest.mark.parametrize("case", [CASES[i] for i in (0, 2, 6)], ids=["0", "2", "6"])
def test_a_weight_on_one_side_and_no_heads_on_the_other(case):
    b, q, k, _, wq, wk, cos, sin, _, kw, g = setup(case)
    cu, d, dtype = ints(b.cu), q.shape[2], q.dtype
    gq, gk = row_tensors(b.T, [q.shape[1], k.shape[1]], d, dtype, g, False)
    both = vlp.thd_qk_norm_rope(q, k, cu, cos, sin, **kw)
    grads = vlp.thd_qk_norm_rope_bwd(gq, gk, q, k, cu, cos, sin, **kw)
    bare = dict(kw, q_weight=None, k_weight=None)
    turn = vlp.thd_qk_norm_rope(q, k, cu, cos, sin, **bare)
    back = vlp.thd_qk_norm_rope_bwd(gq, gk, None, None, cu, cos, sin, **bare)
    got = vlp.thd_qk_norm_rope(q, k, cu, cos, sin, **dict(kw, k_weight=None))
    assert torch.equal(got[0], both[0]) and torch.equal(got[1], turn[1])
    got = vlp.thd_qk_norm_rope_bwd(gq, gk, q, None, cu, cos, sin, **dict(kw, k_weight=None))
    assert torch.equal(got[0], grads[0]) and torch.equal(got[1], back[1]) and got[3] is None
    assert torch.equal(got[2], grads[2])
    got = vlp.thd_qk_norm_rope_bwd(gq, gk, None, k, cu, cos, sin, **dict(kw, q_weight=None))
    assert torch.equal(got[0], back[0]) and torch.equal(got[1], grads[1]) and got[2] is None
    assert torch.equal(got[3], grads[3])
    none = q[:, :0]   # keys alone, and queries alone
    got = vlp.thd_qk_norm_rope(none, k, cu, cos, sin, **dict(kw, q_weight=None))
    assert got[0].shape == none.shape
    near = lambda x, y: torch.all((x.double() - y.double()).abs() <=   # each rounded once, in whichever kernel
                                  torch.finfo(dtype).eps * y.double().abs() + 2.0 ** -18 * y.abs().max().double())
    assert near(got[1], both[1])
    got = vlp.thd_qk_norm_rope(q, None, cu, cos, sin, **dict(kw, k_weight=None))
    assert got[1] is None
    assert near(got[0], both[0])


@pytest.mark.parametrize("positions", [False, True])
@pytest.mark.parametrize("case", [CASES[i] for i in (0, 1, 2, 5, 6)], ids=["0", "1", "2", "5", "6"])
def test_append_over_many_items(case, positions):
    """Slots behind uneven cached lengths, pages in no order, and sequences whose table names no page or ends."""
    b, q, k, v, wq, wk, cos, sin, _, kw, g = setup(case)
    seqs, d, hkv, page = b.seqs, q.shape[2], k.shape[1], 16
    rng = np.random.default_rng(1)
    before = rng.integers(0, 30, seqs)
    need = -(-(before + b.lens) // page)
    pages = int(need.sum()) + 2
    first = np.concatenate([[0], np.cumsum(need)])
    order = rng.permutation(pages)
    table = np.full((seqs, int(need.max()) + 1), -1, np.int64)
    at = np.arange(int(need.sum())) - np.repeat(first[:-1], need)
    table[np.repeat(np.arange(seqs), need), at] = order[:int(need.sum())]
    table[3, 0], table[5] = pages, -1     # a page that the cache does not have, and none at all
    given = torch.tensor(rng.integers(-2, len(cos) + 2, b.T), dtype=torch.int32).cuda() if positions else None
    fill = 9.0
    kc, vc = (torch.full((pages, page, hkv, d), fill, dtype=k.dtype, device="cuda") for _ in range(2))
    out = vlp.thd_kv_append(k, v, kc, vc, ints(table), ints(before), ints(b.cu), b.padded, seqs, q, cos, sin, given, wq, wk,
                            EPS, kw["interleaved"])
    slot = torch.tensor(before).cuda()[b.seq] + b.place
    pos = given.long()[b.rows] if positions else slot
    ref, size = turned(normed(q[b.rows].double(), wq), cos, sin, pos, kw["interleaved"])
    assert_near(out, whole(b, ref), whole(b, size), "q")
    entry = torch.tensor(table).cuda()[b.seq, slot // page]
    kept = (entry >= 0) & (entry < pages)
    place = entry[kept] * page + slot[kept] % page
    ref, size = turned(normed(k[b.rows].double(), wk), cos, sin, pos, kw["interleaved"])
    want, wsize = (torch.full((pages * page, hkv, d), x, dtype=torch.float64, device="cuda") for x in (fill, 0.0))
    want[place], wsize[place] = ref[kept], size[kept]
    assert_near(kc.flatten(0, 1), want, wsize, "k")
    vals = torch.full((pages * page, hkv, d), fill, dtype=v.dtype, device="cuda")
    vals[place] = v[b.rows][kept]
    assert torch.equal(vc.flatten(0, 1), vals)
