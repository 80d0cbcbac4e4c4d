"""GPU tests of attention over a paged cache where a CTA works on many units of a tile.

Tolerances as in test_paged_gpu.py; the reference here is the definition in 64 bits in torch operations on
the GPU, so that sizes may be larger.  An fp16 weight below 2^-14 rounds absolutely, by 2^-25; weights are
held times 2^7 at the least relative to the largest so far, so that is 2^-32 of the largest, for each key.
"""
import numpy as np
import pytest
import torch

from test_paged_gpu import FP16, make, run

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
