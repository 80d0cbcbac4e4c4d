"""Packed attention with a sliding window and first tokens that stay visible (thd_attn_fwd /
thd_attn_bwd with sink_tokens) on the GPU against the fp64 oracle.

Tolerances, u = finfo(dtype).eps / 2 the relative rounding of the 16-bit type and e the share by which an
fp32 score moves its weight: a score is a sum of up to 128 products, each step off by at most 2^-23 (the matrix
units truncate) of S = scale * sum |q k|; with the product by the scale and the exponential's 2 ulp
e = 136 * 2^-23 * S + 2^-21 * (1 + S).
Forward: the weights are rounded to the type, in the numerator and in the sum that normalises them, 2 u of
A = sum_j w_j |v_j|, and move by e, twice: 2 e A; the output is rounded once more, u |out|.  fp16 weights below
2^-14 round absolutely, by 2^-25 each: 2^-25 * keys * max |v|.  The log-sum-exp: e, and 4 * 2^-24 of its size.
Backward: P and dS are rounded once, P moves by e and by the log-sum-exp's 2^-24 |lse| <= e, and the fp32 sums
of a key's up to 2^13 rows here are off by 2^-24 of their terms a step, less than u: a gradient is within
(2 u + 4 e) M of the exact one, M the sum of its terms' sizes, and its own rounding u |g|.  D = rowsum(dO O) is
an fp32 sum of 128 products in fewer than 32 steps one after another: off by 2^-19 of sum |dO O| at most, which
moves dQ and dK by P times that.  fp16 as above, 2^-25 for each term times the other factor.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import bounded
from thd_testutil import to_device

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")

BF16, FP16 = torch.bfloat16, torch.float16
LENS = [700, 1, 129, 90, 300, 0, 257, 41, 128, 900]
CODES = np.array([1, 0, 2, 1, 0, 1, 2, 0, 1, 0], np.uint8)


def f64(t):
    return t.detach().float().cpu().double().numpy()


def batch(d, dtype, seed, hq=4, hkv=2):
    return workloads.from_lengths("sinks", LENS, CODES != 0, gaps_before=[3, 0, 5, 1, 0, 2, 7, 0, 1, 4], trailing=6,
                                  heads_q=hq, heads_kv=hkv, head_dim=d, dtype=dtype, seed=seed, with_padded=True)


def forward(w, dev, window, sinks, **over):
    kw = dict(window=window, sink_tokens=sinks)
    kw.update(over)
    ws = torch.zeros(vlp.thd_attn_workspace_size(), dtype=torch.uint8, device="cuda")
    out, lse = vlp.thd_attn_fwd(dev["q"], dev["k"], dev["v"], dev["cu"], dev["cu"], dev["padded"], dev["padded"],
                                torch.from_numpy(CODES).cuda(), w.batch_size, w.max_seqlen, w.softmax_scale, workspace=ws,
                                **kw)
    torch.cuda.synchronize()
    assert int(ws[8:12].cpu().numpy().view(np.uint32)[0]) == 0
    return out, lse


def check_fwd(got, ref, v, dtype, what):
    out, lse = f64(got[0]), got[1].cpu().double().numpy()
    r, r_lse, size, score = ref
    u = torch.finfo(dtype).eps / 2
    seen = np.isfinite(r_lse)
    assert np.array_equal(np.isneginf(lse), ~seen), what
    assert np.all(out[~seen.T] == 0), what
    e = 136 * 2.0 ** -23 * score + 2.0 ** -21 * (1 + score)
    err = np.abs(np.where(seen, lse, 0) - np.where(seen, r_lse, 0))
    assert np.all(err <= e + 4 * 2.0 ** -24 * np.abs(np.where(seen, r_lse, 0))), (what, err.max())
    tiny = 2.0 ** -25 * max(LENS) * np.abs(v).max() if dtype == FP16 else 0.0
    bound = 2 * u * size + u * np.abs(r) + 2 * e.T[:, :, None] * size + tiny + 2.0 ** -25
    worst = (np.abs(out - r) / bound).max()
    print(f"{what}: largest share of the bound {worst:.3f}")
    assert worst <= 1.0, (what, worst)


BOUNDS = [((64, -1), 1), ((64, 0), 4), ((100, 50), 130), ((0, 0), 3), ((130, 0), 300), ((-1, 37), 90), ((129, 129), 64),
          ((300, 7), 2000), ((1000, 1000), 5), ((0, 200), 128), ((64, 64), 129)]


@pytest.mark.parametrize("d,dtype,hq,hkv", [(128, BF16, 4, 2), (64, FP16, 3, 3), (128, FP16, 5, 1), (40, BF16, 4, 2),
                                            (96, FP16, 2, 1)])
def test_forward_matches_oracle(d, dtype, hq, hkv):
    w = batch(d, dtype, seed=d, hq=hq, hkv=hkv)
    dev = to_device(w)
    for window, sinks in BOUNDS:
        got = forward(w, dev, window, sinks)
        ref = bounded.attention_fwd(w.q, w.k, w.v, w.cu_seqlens, w.cu_seqlens, w.cu_seqlens_padded, w.cu_seqlens_padded,
                                    CODES, w.batch_size, w.softmax_scale, window, sinks)
        check_fwd(got, ref, f64(w.v), dtype, f"d {d} window {window} sinks {sinks}")


@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, FP16), (40, BF16)])
def test_no_sinks_and_no_window_are_the_calls_without_them_bit_for_bit(d, dtype):
    w = batch(d, dtype, seed=3)
    dev = to_device(w)
    codes = torch.from_numpy(CODES).cuda()
    args = (dev["q"], dev["k"], dev["v"], dev["cu"], dev["cu"], dev["padded"], dev["padded"], codes, w.batch_size,
            w.max_seqlen, w.softmax_scale)
    for window, sinks in (((64, 3), 0), ((-1, -1), 7)):
        a, b = vlp.thd_attn_fwd(*args, window=window), forward(w, dev, window, sinks)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("window,sinks", [((5, 0), 2), ((0, 3), 70), ((40, 20), 130)])
def test_forward_with_separate_q_kv_sequences(window, sinks):
    lq, lkv = [250, 300, 7, 200, 130], [100, 64, 40, 400, 0]
    codes = np.array([2, 1, 2, 2, 1], np.uint8)
    qs = np.array([0, 250, 550, 557, 757], np.int32)
    ks = np.array([887, 987, 1051, 1091, 1491], np.int32)
    w = workloads.from_lengths("rect", [1500], [0], heads_q=4, heads_kv=2, head_dim=128, dtype=BF16, seed=9)
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (lq, lkv))
    dv = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    q, k, v = w.q.cuda(), w.k.cuda(), w.v.cuda()
    got = vlp.thd_attn_fwd(q, k, v, dv(cu_q), dv(cu_k), dv(qs), dv(ks), dv(codes), 5, 300, w.softmax_scale,
                           window=window, sink_tokens=sinks)
    ref = bounded.attention_fwd(w.q, w.k, w.v, cu_q, cu_k, qs, ks, codes, 5, w.softmax_scale, window, sinks)
    check_fwd(got, ref, f64(w.v), BF16, f"separate {window} {sinks}")
    dout = workloads.grad_output(w, 5)
    grads = vlp.thd_attn_bwd(q, k, v, *got, dout.cuda(), dv(cu_q), dv(cu_k), dv(qs), dv(ks), dv(codes), 5, 300,
                             w.softmax_scale, window=window, sink_tokens=sinks)
    ref = bounded.attention_bwd(w.q, w.k, w.v, f64(got[0]), f64(got[1]), dout, cu_q, cu_k, qs, ks, codes, 5,
                                w.softmax_scale, window, sinks)
    check_bwd(grads, ref, (w.q, w.k, w.v), dout, w.softmax_scale, BF16, f"separate {window} {sinks}")


def check_bwd(grads, ref, qkv, dout, scale, dtype, what):
    u = torch.finfo(dtype).eps / 2
    g, score = ref
    e = 136 * 2.0 ** -23 * score + 2.0 ** -21 * (1 + score)
    q, k, _ = (np.abs(f64(x)).max() for x in qkv)
    tiny = 2.0 ** -25 if dtype == FP16 else 0.0
    for got, (r, size, moved, terms), name, other in zip(grads, g, ("dq", "dk", "dv"), (scale * k, scale * q,
                                                                                        np.abs(f64(dout)).max())):
        bound = (2 * u + 4 * e) * size + u * np.abs(r) + 2.0 ** -19 * moved + tiny * terms * other + 2.0 ** -25
        worst = (np.abs(f64(got) - r) / bound).max()
        print(f"{what} {name}: largest share of the bound {worst:.3f}")
        assert worst <= 1.0, (what, name, worst)


@pytest.mark.parametrize("d,dtype,hq,hkv", [(128, BF16, 4, 2), (64, FP16, 3, 3), (64, BF16, 5, 1), (128, FP16, 2, 1)])
def test_backward_matches_oracle(d, dtype, hq, hkv):
    w = batch(d, dtype, seed=20 + d, hq=hq, hkv=hkv)
    dev = to_device(w)
    codes = torch.from_numpy(CODES).cuda()
    dout = workloads.grad_output(w, 7)
    for window, sinks in BOUNDS:
        out, lse = forward(w, dev, window, sinks)
        grads = vlp.thd_attn_bwd(dev["q"], dev["k"], dev["v"], out, lse, dout.cuda(), dev["cu"], dev["cu"], dev["padded"],
                                 dev["padded"], codes, w.batch_size, w.max_seqlen, w.softmax_scale, window=window,
                                 sink_tokens=sinks)
        torch.cuda.synchronize()
        ref = bounded.attention_bwd(w.q, w.k, w.v, f64(out), f64(lse), dout, w.cu_seqlens, w.cu_seqlens,
                                    w.cu_seqlens_padded, w.cu_seqlens_padded, CODES, w.batch_size, w.softmax_scale,
                                    window, sinks)
        check_bwd(grads, ref, (w.q, w.k, w.v), dout, w.softmax_scale, dtype, f"d {d} window {window} sinks {sinks}")


@pytest.mark.parametrize("d,dtype,hq,hkv,window,sinks", [(64, BF16, 2, 1, (100, 0), 4), (128, FP16, 3, 3, (500, 0), 130),
                                                       (128, BF16, 2, 2, (0, 0), 1), (64, FP16, 4, 1, (1023, 0), 16),
                                                       (64, BF16, 1, 1, (10, 10), 600)])
def test_keys_seen_by_the_queries_of_several_chunks(d, dtype, hq, hkv, window, sinks):
    """Sequences of several times 2048 rows: the sums of their first keys come from several items."""
    lens = [5000, 60, 2300, 4096]
    codes = np.array([1, 1, 2, 0], np.uint8)
    w = workloads.from_lengths("far", lens, codes != 0, gaps_before=[3, 1, 900, 0], trailing=5, heads_q=hq, heads_kv=hkv,
                               head_dim=d, dtype=dtype, seed=1, with_padded=True)
    dev = to_device(w)
    c = torch.from_numpy(codes).cuda()
    args = (dev["cu"], dev["cu"], dev["padded"], dev["padded"], c, w.batch_size, w.max_seqlen, w.softmax_scale)
    out, lse = vlp.thd_attn_fwd(dev["q"], dev["k"], dev["v"], *args, window=window, sink_tokens=sinks)
    dout = workloads.grad_output(w, 7)
    grads = [vlp.thd_attn_bwd(dev["q"], dev["k"], dev["v"], out, lse, dout.cuda(), *args, window=window, sink_tokens=sinks)
             for _ in range(2)]
    torch.cuda.synchronize()
    ref = bounded.attention_bwd(w.q, w.k, w.v, f64(out), f64(lse), dout, w.cu_seqlens, w.cu_seqlens, w.cu_seqlens_padded,
                                w.cu_seqlens_padded, codes, w.batch_size, w.softmax_scale, window, sinks)
    check_bwd(grads[0], ref, (w.q, w.k, w.v), dout, w.softmax_scale, dtype, f"d {d} window {window} sinks {sinks}")
    assert torch.equal(grads[0][1], grads[1][1]) and torch.equal(grads[0][2], grads[1][2])   # one order of the sums


def test_workspace_sizes():
    plain = vlp.load_library().thd_attn_bwd_workspace_size(5000, 4, 64)
    size = lambda *a: vlp.load_library().thd_attn_bwd_sinks_workspace_size(*a)  # noqa: E731
    assert size(5000, 4, 2, 64, 3, 100, 0) == plain == size(5000, 4, 2, 64, 3, -1, 4) == size(5000, 4, 2, 64, 3, 100, 513)
    assert size(5000, 4, 2, 64, 3, 100, 4) == plain + 3 * 2 * 2 * 4 * 64 * 4 + (3 + 2 + 1) * 2 * 2 * 4 * 64 * 4
    assert size(-1, 4, 2, 64, 3, 100, 4) == 0
    w = batch(64, BF16, 1)
    dev = to_device(w)
    out, lse = forward(w, dev, (64, 0), 4)
    short = vlp.load_library().thd_attn_bwd_workspace_size(w.total_tokens, 4, 64)
    with pytest.raises(vlp.ThdError) as err:
        vlp.thd_attn_bwd(dev["q"], dev["k"], dev["v"], out, lse, out, dev["cu"], dev["cu"], dev["padded"], dev["padded"],
                         torch.from_numpy(CODES).cuda(), w.batch_size, w.max_seqlen, w.softmax_scale, window=(64, 0),
                         sink_tokens=4, workspace=torch.empty(short, dtype=torch.uint8, device="cuda"))
    assert err.value.status == vlp.THD_ERR_WORKSPACE
