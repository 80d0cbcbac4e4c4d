"""Calls around the edges of the operators that bound what a long sequence costs: sizes at their limits, streams at once,
captured and replayed calls, empty batches and caches, waits that run out."""
import numpy as np
import pytest
import torch

import workloads
from oracle import bounded
from test_evict_gpu import bits
from test_evict_gpu import check as check_evict
from test_evict_gpu import make as make_evict
from test_paged_gpu import BF16, FP16, ints, make
from test_paged_window_gpu import check, run, weights_of
from test_sinks_gpu import check_bwd, check_fwd, f64
from thd_testutil import to_device

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")


def packed(lens, codes, d, dtype, hq=4, hkv=2, seed=0, gaps=None):
    w = workloads.from_lengths("more", lens, np.asarray(codes) != 0, gaps_before=gaps, trailing=3, heads_q=hq, heads_kv=hkv,
                               head_dim=d, dtype=dtype, seed=seed, with_padded=True)
    dev = to_device(w)
    c = torch.tensor(codes, dtype=torch.uint8).cuda()
    return w, dev, (dev["cu"], dev["cu"], dev["padded"], dev["padded"], c, w.batch_size, w.max_seqlen, w.softmax_scale)


@pytest.mark.parametrize("window,sinks", [((0, 0), 2 ** 31 - 1), ((2 ** 31 - 1, 0), 3), ((50, 2 ** 31 - 1), 7), ((0, 0), 0)])
def test_sizes_at_their_limits(window, sinks):
    codes = [1, 0, 2]
    w, dev, args = packed([300, 129, 1], codes, 64, FP16)
    q, k, v = dev["q"], dev["k"], dev["v"]
    got = vlp.thd_attn_fwd(q, k, v, *args, window=window, sink_tokens=sinks)
    ref = bounded.attention_fwd(w.q, w.k, w.v, w.cu_seqlens, w.cu_seqlens, w.cu_seqlens_padded, w.cu_seqlens_padded, codes, 3,
                                w.softmax_scale, window, sinks)
    check_fwd(got, ref, f64(w.v), FP16, f"{window} {sinks}")
    dout = workloads.grad_output(w, 5)
    grads = vlp.thd_attn_bwd(q, k, v, *got, dout.cuda(), *args, window=window, sink_tokens=sinks)
    ref = bounded.attention_bwd(w.q, w.k, w.v, f64(got[0]), f64(got[1]), dout, w.cu_seqlens, w.cu_seqlens,
                                w.cu_seqlens_padded, w.cu_seqlens_padded, codes, 3, w.softmax_scale, window, sinks)
    if window != (0, 0) or sinks:   # a row that sees itself alone has no gradients of q and k but roundings
        check_bwd(grads, ref, (w.q, w.k, w.v), dout, w.softmax_scale, FP16, f"{window} {sinks}")


def test_rows_of_no_sequence_keep_their_zeros_and_batches_may_be_empty():
    w, dev, args = packed([40, 0, 200], [1, 1, 0], 128, BF16, gaps=[5, 3, 60])
    out, lse = torch.full_like(dev["q"], 7.0), torch.full((4, w.total_tokens), 7.0, device="cuda")
    vlp.thd_attn_fwd(dev["q"], dev["k"], dev["v"], *args, window=(20, 0), sink_tokens=2, out=out, lse=lse)
    grads = [torch.full_like(dev[n], 7.0) for n in "qkv"]
    vlp.thd_attn_bwd(dev["q"], dev["k"], dev["v"], out, lse, dev["q"], *args, window=(20, 0), sink_tokens=2, dq=grads[0],
                     dk=grads[1], dv=grads[2])
    rows = torch.ones(w.total_tokens, dtype=torch.bool)
    for s, n in zip(w.starts, w.lengths):
        rows[int(s):int(s) + int(n)] = False
    rows = rows.cuda()
    assert torch.all(out[rows] == 0) and torch.all(torch.isneginf(lse[:, rows])) and all(torch.all(g[rows] == 0) for g in grads)
    assert not torch.any(out[~rows] == 7) and not any(torch.any(g[~rows] == 7) for g in grads)
    none = (args[0], args[1], None, None, None, 0, 0, 0.1)
    o, l = vlp.thd_attn_fwd(dev["q"], dev["k"], dev["v"], *none, window=(5, 0), sink_tokens=2)
    g = vlp.thd_attn_bwd(dev["q"], dev["k"], dev["v"], o, l, dev["q"], *none, window=(5, 0), sink_tokens=2)
    assert torch.all(o == 0) and torch.all(torch.isneginf(l)) and all(torch.all(x == 0) for x in g)
    e = dev["q"][:0], dev["k"][:0], dev["v"][:0]
    assert vlp.thd_attn_fwd(*e, *none, window=(5, 0), sink_tokens=2)[0].shape == (0, 4, 128)


def test_training_step_captured_and_replayed_with_other_lengths():
    w, dev, args = packed([700, 90, 2500], [1, 0, 1], 128, BF16)
    cu, padded, codes = args[0], args[2], args[4]
    dout = workloads.grad_output(w, 5).cuda()

    def step():
        out, lse = vlp.thd_attn_fwd(dev["q"], dev["k"], dev["v"], cu, cu, padded, padded, codes, 3, 2500, w.softmax_scale,
                                    window=(100, 0), sink_tokens=4)
        return (out, lse) + tuple(vlp.thd_attn_bwd(dev["q"], dev["k"], dev["v"], out, lse, dout, cu, cu, padded, padded, codes,
                                                   3, 2500, w.softmax_scale, window=(100, 0), sink_tokens=4))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for lens in ([700, 90, 2500], [1, 90, 2000], [650, 0, 130]):
        cu.copy_(ints(np.concatenate([[0], np.cumsum(lens)])))
        graph.replay()
        torch.cuda.synchronize()
        held = [g.clone() for g in got]
        for a, b, what in zip(held, step(), ("out", "lse", "dq", "dk", "dv")):
            # dq is added up by atomics, in any order: a few fp32 roundings before the one to bf16
            assert torch.equal(a, b) if what != "dq" else (a.float() - b.float()).abs().max() <= 2.0 ** -7 * a.abs().max()


def test_calls_on_two_streams_at_once():
    x = [make([4000, 300], [n, 1], 16, 16, 4, 128, BF16, seed=n) for n in (1, 200)]
    y = [make_evict([3000, 700], [900, 650], 16, 4, 64, seed=s, apart=s > 0) for s in range(2)]
    had = [weights_of(z) for z in x]
    alone = []
    for z, e in zip(x, y):
        weights = weights_of(z)
        alone.append(run(z, z["table"], 500, 4, weights) + (weights,))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    together, lens = [], []
    for s, z, e in zip(streams, x, y):
        with torch.cuda.stream(s):
            weights = weights_of(z)
            table, keys, cu = ints(z["table"]), ints(z["keys"]), ints(z["cu"])
            for _ in range(3):
                weights.copy_(had[len(together)])
                got = vlp.thd_attn_paged(z["q"], z["kc"], z["vc"], table, keys, cu, window=(500, 0), sink_tokens=4,
                                         key_weights=weights)
            together.append(got + (weights,))
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        for p, q in zip(a, b):
            assert torch.equal(p, q)
    refs = []
    for e in y:
        caches = [bits(e["kc"]).copy(), bits(e["vc"]).copy()]
        refs.append(bounded.evict(caches, e["w"].cpu().numpy(), e["table"], e["keys"], e["keep"], e["new"], 2, 4, 20))
    for s, e in zip(streams, y):
        with torch.cuda.stream(s):
            lens.append(vlp.thd_kv_evict(e["kc"], e["vc"], e["w"], ints(e["table"]), ints(e["keys"]), ints(e["keep"]),
                                         new_page_table=None if e["new"] is None else ints(e["new"]), sink_tokens=4,
                                         recent_tokens=20))
    torch.cuda.synchronize()
    for e, n, r in zip(y, lens, refs):
        assert n.tolist() == r[2] and np.array_equal(bits(e["kc"]), r[0][0]) and np.array_equal(bits(e["vc"]), r[0][1])


def test_weights_and_eviction_of_views():
    """Caches and weights that are parts of larger tensors, tables with rows apart."""
    x = make([200, 70], [1, 40], 16, 4, 2, 64, BF16)
    pages = len(x["kc"])
    big = [torch.zeros(pages, 16, 5, 64, dtype=BF16, device="cuda") for _ in range(2)]
    for b, n in zip(big, ("kc", "vc")):
        b[:, :, 1:3] = x[n]
        x[n] = b[:, :, 1:3]
    wide = torch.rand(pages, 5, 40, device="cuda")
    w = wide.transpose(1, 2)[:, 2:18, 1:3]
    had, around = w.clone(), wide.clone()
    check(x, run(x, x["table"], -1, 0, w), -1, 0, had, w)
    around.transpose(1, 2)[:, 2:18, 1:3] = w
    assert torch.equal(wide, around)
    table = torch.full((2, x["table"].shape[1] + 7), -1, dtype=torch.int32, device="cuda")
    table[:, :x["table"].shape[1]] = ints(x["table"])
    caches = [bits(x["kc"].contiguous()).copy(), bits(x["vc"].contiguous()).copy()]
    ref = bounded.evict(caches, w.cpu().numpy(), x["table"], [200, 70], [90, 30], None, 2, 3, 9)
    lens = vlp.thd_kv_evict(x["kc"], x["vc"], w, table[:, :x["table"].shape[1]], ints([200, 70]), ints([90, 30]),
                            sink_tokens=3, recent_tokens=9)
    assert lens.tolist() == [90, 30] and torch.equal(w.cpu(), torch.from_numpy(ref[1]))
    assert np.array_equal(bits(x["kc"].contiguous()), ref[0][0]) and np.array_equal(bits(x["vc"].contiguous()), ref[0][1])
    assert all(torch.all(b[:, :, [0, 3, 4]] == 0) for b in big)


def test_caches_without_pages():
    none = torch.empty(0, 16, 2, 64, dtype=BF16, device="cuda")
    w = torch.empty(0, 16, 2, device="cuda")
    table = ints(np.zeros((2, 3)))
    lens = vlp.thd_kv_evict(none, none.clone(), w, table, ints([5, 0]), ints([3, 3]))
    assert lens.tolist() == [0, 0]
    q = torch.randn(2, 4, 64, device="cuda").to(BF16)
    out, lse = vlp.thd_attn_paged(q, none, none, table, ints([5, 5]), ints([0, 1, 2]), window=(3, 0), sink_tokens=1,
                                  key_weights=w)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


def test_long_lists_by_several_ctas():
    check_evict(make_evict([150000, 30], [70000, 30], 64, 1, 16, few=True), 5, 100, width=70000)
    check_evict(make_evict([40000, 30001, 1], [1, 30000, 1], 16, 2, 8, apart=True), 0, 0, width=30000)


def test_waits_that_run_out_are_reported():
    w, dev, args = packed([300, 2600], [1, 1], 64, BF16)
    kw = dict(window=(64, 0), sink_tokens=4)
    x = make([900, 300], [40, 40], 16, 16, 4, 128, BF16)
    fwd = torch.zeros(vlp.thd_attn_workspace_size(), dtype=torch.uint8, device="cuda")
    bwd = torch.zeros(vlp.load_library().thd_attn_bwd_sinks_workspace_size(w.total_tokens, 4, 2, 64, 2, 64, 4),
                      dtype=torch.uint8, device="cuda")
    paged = torch.zeros(vlp.thd_attn_paged_workspace_size(128), dtype=torch.uint8, device="cuda")
    weights = weights_of(x)
    good = vlp.thd_attn_fwd(dev["q"], dev["k"], dev["v"], *args, **kw)

    def words():
        out = []
        vlp.thd_attn_fwd(dev["q"], dev["k"], dev["v"], *args, workspace=fwd, **kw)
        vlp.thd_attn_bwd(dev["q"], dev["k"], dev["v"], *good, dev["q"], *args, workspace=bwd, **kw)
        vlp.thd_attn_paged(x["q"], x["kc"], x["vc"], ints(x["table"]), ints(x["keys"]), ints(x["cu"]), workspace=paged,
                           key_weights=weights)
        torch.cuda.synchronize()
        for t in (fwd, bwd, paged):
            out.append(int(t[8:12].cpu().numpy().view(np.uint32)[0]))
        return out
    before = vlp.thd_set_wait_limit_ns(1)   # a wait still pending after its first poll runs out
    vlp.thd_set_wait_injection(True)
    try:
        assert words() == [vlp.STATUS_WAIT_TIMEOUT] * 3
    finally:
        vlp.thd_set_wait_limit_ns(before)
        vlp.thd_set_wait_injection(False)
    assert words() == [0, 0, 0]
    again = vlp.thd_attn_fwd(dev["q"], dev["k"], dev["v"], *args, **kw)
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
