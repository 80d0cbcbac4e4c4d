"""GPU tests of attention over a paged cache where a CTA works on many units of a tile, where a sequence's new
tokens take many tiles, and of both kernels (tiles of 16 and of 128 rows) on the same inputs.

Tolerances as in test_paged_gpu.py; the reference here is the definition in 64 bits in torch operations on
the GPU, so that sizes may be larger.  An fp16 weight below 2^-14 rounds absolutely, by 2^-25; weights are
held times 2^7 at the least relative to the largest so far, so that is 2^-32 of the largest, for each key.
"""
import numpy as np
import pytest
import torch

from test_paged_gpu import BF16, FP16, ints, make, run

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")


def visible(x, b, n, L):
    """[n, L] whether new token i of sequence b sees key j."""
    j, i = torch.arange(L, device="cuda") - (L - n), torch.arange(n, device="cuda")
    if x["tree"] is None:
        return j[None] <= i[:, None]
    start = int((x["cu"] if x["padded"] is None else x["padded"])[b])
    words = torch.tensor(x["tree"][start:start + n]).cuda()
    w, s = (j // 64).clamp(0, words.shape[1] - 1), j.clamp(min=0) % 64
    bit = (words[:, w] >> s[None] & 1).bool() & (j // 64 < words.shape[1])[None]
    return (j < 0)[None] | bit


def check(x, got, scale=None):
    out, lse = got
    q, page = x["q"], x["kc"].shape[1]
    T, hq, d = q.shape
    hkv, dtype = x["kc"].shape[2], q.dtype
    scale = d ** -0.5 if scale is None else scale
    u = torch.finfo(dtype).eps / 2
    none = torch.ones(T, dtype=torch.bool, device="cuda")
    worst, worst_lse = 0.0, 0.0
    for b in range(x["B"]):
        n, L = int(x["cu"][b + 1] - x["cu"][b]), int(x["keys"][b])
        start = int((x["cu"] if x["padded"] is None else x["padded"])[b])
        rows = slice(start, start + n)
        if n == 0 or L == 0:
            continue
        none[rows] = False
        pages = torch.tensor(x["table"][b, :-(-L // page)]).long().cuda()
        k, v = (c[pages].flatten(0, 1)[:L].double().repeat_interleave(hq // hkv, 1) for c in (x["kc"], x["vc"]))
        see = visible(x, b, n, L)
        qq = q[rows].double()
        s = (torch.einsum("ihd,jhd->hij", qq, k) * scale).masked_fill(~see, float("-inf"))
        S = (torch.einsum("ihd,jhd->hij", qq.abs(), k.abs()) * scale).masked_fill(~see, 0).amax(2)   # [h, i]
        some = see.any(1)
        want_lse = s.logsumexp(2)
        p = torch.exp(s - want_lse.masked_fill(~some, 0)[..., None])
        ref, A = torch.einsum("hij,jhd->ihd", p, v), torch.einsum("hij,jhd->ihd", p, v.abs())
        e = 136 * 2.0 ** -23 * S + 2.0 ** -21 * (1 + S)
        got_lse = lse[:, rows].double()
        assert torch.equal(torch.isneginf(got_lse), torch.isneginf(want_lse))
        off = (got_lse - want_lse)[:, some].abs()
        # beside e, the sum's own roundings: a product and a sum for each unit of 64 keys
        room = e + 4 * 2.0 ** -24 * want_lse.abs().nan_to_num(posinf=0) + 2 * L / 64 * 2.0 ** -24
        worst_lse = max(worst_lse, float((off / room[:, some]).max()) if off.numel() else 0.0)
        least = 2.0 ** -25 if dtype == FP16 else 2.0 ** -134
        tiny = 2.0 ** -32 * L * float(v.abs().max()) if dtype == FP16 else 0.0
        bound = 2 * u * A + u * ref.abs() + 2 * e.T[..., None] * A + least + tiny
        o = out[rows].double()
        assert torch.all(o[~some] == 0)
        worst = max(worst, float(((o - ref).abs() / bound)[some].nan_to_num(nan=1e30).max()) if some.any() else 0.0)
    assert torch.all(out[none] == 0) and torch.all(torch.isneginf(lse[:, none]))
    print(f"largest share of the bound {worst:.3f}, of the log-sum-exp's {worst_lse:.3f}")
    assert worst <= 1.0 and worst_lse <= 1.0, (worst, worst_lse)


def on_keys(x, f):
    """The cached keys of every sequence times f(their places)."""
    page = x["kc"].shape[1]
    for b, L in enumerate(x["keys"]):
        j = np.arange(int(L))
        pages, inside = torch.tensor(x["table"][b, j // page]).long().cuda(), torch.tensor(j % page).cuda()
        x["kc"][pages, inside] = (x["kc"][pages, inside].float() * torch.tensor(f(j)).cuda()[:, None, None]).to(x["kc"].dtype)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("dtype,d,hq,hkv,new", [(BF16, 128, 16, 4, 9), (FP16, 128, 16, 4, 30), (BF16, 64, 16, 4, 30),
                                                (FP16, 64, 32, 4, 8), (BF16, 128, 16, 4, 4)])
def test_a_maximum_that_keeps_growing(dtype, d, hq, hkv, new, tree):
    """Eight and more units for each CTA, the keys of every 64 three steps larger than those before, back to
    small after five: the output is rescaled by what the maximum grew by, in some rows of a warp and (small
    queries) never in others."""
    keys = [5000 + 130 * i for i in range(8)]
    x = make(keys, [new] * 8, 16, hq, hkv, d, dtype, words=1 if tree else 0)
    on_keys(x, lambda j: 0.5 + 3.0 * (j // 64 % 5))
    x["q"][::3] *= 0.05
    work = torch.zeros(vlp.thd_attn_paged_workspace_size(d), dtype=torch.uint8, device="cuda")
    got = run(x, max_seqlen_q=new, workspace=work)
    assert int(work[8:12].view(torch.int32).item()) == 0
    check(x, got)


@pytest.mark.parametrize("hint", [True, False])
@pytest.mark.parametrize("keys,new,hq,hkv,d,dtype,gap,words", [
    ([2500], [2500], 4, 1, 128, BF16, 0, 0),                             # a fresh prompt: half of the units hidden
    ([1024, 1100, 3000, 40], [1024, 900, 1300, 40], 8, 2, 64, FP16, 5, 0),
    ([4000, 700], [1025, 1100], 4, 4, 80, BF16, 3, 0),                   # the second with fewer keys than tokens
    ([1500, 90], [1200, 70], 2, 2, 128, FP16, 0, 19),                    # a mask of 19 words
])
def test_prompt_chunks(keys, new, hq, hkv, d, dtype, gap, words, hint):
    x = make(keys, new, 16, hq, hkv, d, dtype, gap, words)
    check(x, run(x, max_seqlen_q=max(new) if hint else 1))


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_small_fp16_weights_of_many_keys(rows, d):
    """One key at the maximum and many at 2^-23.5 of it, whose sum counts: near the least subnormal of fp16."""
    L, B = 20000, 304   # as many tiles as CTAs, so that one keeps the maximum over all of its keys
    x = make([L + rows], [rows], 16, 1, 1, d, FP16)
    pages = torch.tensor(x["table"][0, :-(-(L + rows) // 16)]).long().cuda()
    x["q"].zero_()[:, :, 0] = 4.0
    x["kc"][pages], x["vc"][pages] = 0.0, 1.0
    x["kc"][pages, :, :, 0] = -23.5 * np.log(2) / 4
    first = pages[len(pages) // 2]
    x["kc"][first, 3], x["vc"][first, 3] = 0.0, 0.0
    x.update(q=x["q"].repeat(B, 1, 1), table=x["table"].repeat(B, 0), keys=x["keys"].repeat(B), B=B,
             cu=rows * np.arange(B + 1))   # all of them over the same pages
    check(x, run(x, max_seqlen_q=rows, softmax_scale=1.0), 1.0)


@pytest.mark.parametrize("hint", [1, 0])
def test_what_is_not_finite_among_the_visible(hint):
    """As the definition has it, and in no other row or column: a NaN query or key gives NaN in the rows that see it, an
    infinite score NaN or weight 0 by its sign, an infinite value a column that is not finite."""
    n, L, hq, d = 24, 900, 2, 64
    plain = make([L], [n], 16, hq, 2, d, BF16)
    want, want_lse = run(plain, max_seqlen_q=hint)
    table = torch.tensor(plain["table"]).long().cuda()
    at = lambda j: (table[0, j // 16], j % 16)

    x = dict(plain, q=plain["q"].clone())
    x["q"][3, 1, 5] = float("nan")
    out, lse = run(x, max_seqlen_q=hint)
    bad = torch.zeros(n, hq, dtype=torch.bool, device="cuda")
    bad[3, 1] = True
    assert torch.all(out[bad].isnan()) and torch.all(lse.T[bad].isnan())
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse.T[~bad], want_lse.T[~bad])

    x = dict(plain, kc=plain["kc"].clone())
    x["kc"][(*at(L - n + 7), 0, 7)] = float("nan")   # the key of new token 7, for head 0: tokens from 7 on see it
    out, lse = run(x, max_seqlen_q=hint)
    bad = torch.zeros(n, hq, dtype=torch.bool, device="cuda")
    bad[7:, 0] = True
    assert torch.all(out[bad].isnan()) and torch.all(lse.T[bad].isnan())
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse.T[~bad], want_lse.T[~bad])

    x = dict(plain, kc=plain["kc"].clone())
    x["kc"][(*at(100), 1, 9)] = float("inf")     # a cached key of head 1: its score is infinite, by the query's sign
    out, lse = run(x, max_seqlen_q=hint)
    up = plain["q"][:, 1, 9] > 0
    assert torch.all(out[up, 1].isnan()) and not torch.any(lse[1, up].isfinite())
    assert torch.equal(out[:, 0], want[:, 0]) and torch.all(out[~up, 1].isfinite()) and torch.all(lse[1, ~up].isfinite())

    x = dict(plain, vc=plain["vc"].clone())
    x["vc"][(*at(200), 0, 11)] = float("inf")
    out, lse = run(x, max_seqlen_q=hint)
    bad = torch.zeros(n, hq, d, dtype=torch.bool, device="cuda")
    bad[:, 0, 11] = True
    assert not torch.any(out[bad].isfinite()) and torch.equal(out[~bad], want[~bad]) and torch.equal(lse, want_lse)


# ------------------------------------------------------------------------------ both kernels
# The hint picks the kernel: heads of a group times new tokens up to 16 the 16-row tiles, more the 128-row ones.
@pytest.mark.parametrize("hint", [1, 5])
def test_bad_metadata_stays_in_the_buffers(hint):
    x = make([50, 60, 70], [3, 4, 5], 8, 16, 2, 64, BF16)
    rng = np.random.default_rng(6)
    for _ in range(6):
        y = dict(x, table=rng.integers(-5, 60, x["table"].shape), keys=rng.integers(-10, 10**6, 3),
                 cu=rng.integers(-30, 30, 4))
        run(y, max_seqlen_q=hint)
    check(x, run(x, max_seqlen_q=hint))


@pytest.mark.parametrize("hint", [2, 9])
def test_two_streams_at_once(hint):
    xs = [make([4000 + i, 300], [8, 2], 16, 8, 2, 128, BF16, seed=i) for i in range(2)]
    want = [run(x, max_seqlen_q=hint) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    args = [(x["q"], x["kc"], x["vc"], ints(x["table"]), ints(x["keys"]), ints(x["cu"])) for x in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, s in zip(args, streams):
            with torch.cuda.stream(s):
                got.append(vlp.thd_attn_paged(*a, max_seqlen_q=hint))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    for x, w in zip(xs, want):
        check(x, w)


@pytest.mark.parametrize("hint", [4, 40])
def test_graph_replayed_with_other_lengths(hint):
    x = make([70, 900, 5], [20, 1, 3], 16, 8, 2, 128, BF16)
    y = make([3000, 200, 64], [1, 22, 1], 16, 8, 2, 128, BF16, seed=1, extra=60)
    w = max(x["table"].shape[1], y["table"].shape[1])
    pages = max(len(x["kc"]), len(y["kc"]))
    held = dict(q=torch.zeros_like(x["q"]), kc=torch.zeros(pages, 16, 2, 128, dtype=BF16, device="cuda"),
                vc=torch.zeros(pages, 16, 2, 128, dtype=BF16, device="cuda"),
                table=torch.zeros(3, w, dtype=torch.int32, device="cuda"), keys=ints([0] * 3), cu=ints([0] * 4))
    work = torch.empty(vlp.thd_attn_paged_workspace_size(128), dtype=torch.uint8, device="cuda")
    call = lambda: vlp.thd_attn_paged(held["q"], held["kc"], held["vc"], held["table"], held["keys"], held["cu"],
                                      max_seqlen_q=hint, workspace=work)
    with torch.cuda.stream(torch.cuda.Stream()):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for z in (x, y, x):
        for name in ("q", "kc", "vc"):
            held[name][:len(z[name])].copy_(z[name])
        held["table"].fill_(-1)
        held["table"][:, :z["table"].shape[1]] = ints(z["table"])
        held["keys"].copy_(ints(z["keys"]))
        held["cu"].copy_(ints(z["cu"]))
        graph.replay()
        torch.cuda.synchronize()
        check(dict(z, q=held["q"]), got)


def test_wide_tiles_past_two_to_the_31_elements():
    keys, page, d, rows = 20000, 16, 128, 20
    pages = (1 << 20) + 4
    kc = torch.zeros(pages, page, 1, d, dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    x = make([keys], [rows], page, 8, 1, d, BF16)
    need = -(-keys // page)
    last = torch.arange(pages - 1, pages - 1 - need, -1)
    old = torch.tensor(x["table"][0, :need]).long().cuda()
    kc[last.cuda()], vc[last.cuda()] = x["kc"][old], x["vc"][old]
    x.update(kc=kc, vc=vc, table=last.int().numpy()[None])
    check(x, run(x, max_seqlen_q=rows))


def test_several_tiles_for_each_cta():
    """Tiles of 5 units, 1600 and more: a CTA's share begins and ends inside a tile and holds whole ones."""
    x = make([300 + i % 20 for i in range(400)], [6] * 400, 16, 16, 4, 64, BF16)
    for hint in (4, 6):   # 16 rows to a tile and two tiles a sequence, or one of 128
        check(x, run(x, max_seqlen_q=hint))


@pytest.mark.parametrize("hint", [8, 16])
def test_one_tile_over_many_units_of_a_cta(hint):
    """140,000 keys of 8 key heads: 57 units of one tile and more for each CTA."""
    x = make([140000], [16], 64, 16, 8, 64, BF16, words=1)
    check(x, run(x, max_seqlen_q=hint))
