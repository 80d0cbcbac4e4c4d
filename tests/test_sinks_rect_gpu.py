"""Window with first tokens that stay visible, two consecutive row blocks of one head over fewer keys than queries: blocks
whose window lies partly or wholly behind the last key.  Tolerances as test_sinks_gpu.py derives them; no row sees
more than 900 keys."""
import numpy as np
import pytest
import torch

import workloads
from oracle import bounded
from test_sinks_gpu import BF16, FP16, check_bwd, check_fwd, f64

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")

LQ, LKV = [1400, 700, 300, 1400, 1300, 900, 600, 1400], [1024, 256, 128, 900, 896, 512, 128, 640]
CODES = np.array([1, 1, 0, 0, 0, 1, 1, 2], np.uint8)


@pytest.mark.parametrize("d,dtype,hq,hkv", [(128, BF16, 3, 3), (64, FP16, 3, 1), (64, BF16, 1, 1), (128, FP16, 5, 1)])
@pytest.mark.parametrize("window,sinks", [((127, -1), 4), ((0, -1), 1), ((127, 0), 130), ((300, 7), 4), ((5, 0), 600)])
def test_windows_behind_the_last_key(d, dtype, hq, hkv, window, sinks):
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (LQ, LKV))
    T, B = int(cu_q[-1]), len(LQ)
    w = workloads.from_lengths("behind", [T], [0], heads_q=hq, heads_kv=hkv, head_dim=d, dtype=dtype, seed=hq + d)
    dv = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    q, k, v = w.q.cuda(), w.k.cuda(), w.v.cuda()
    args = (dv(cu_q), dv(cu_k), None, None, dv(CODES), B, max(LQ), w.softmax_scale)
    ws = torch.zeros(vlp.thd_attn_workspace_size(), dtype=torch.uint8, device="cuda")
    runs = [vlp.thd_attn_fwd(q, k, v, *args, window=window, sink_tokens=sinks, workspace=ws) for _ in range(2)]
    torch.cuda.synchronize()
    assert int(ws[8:12].cpu().numpy().view(np.uint32)[0]) == 0   # no wait ran out
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    what = f"d {d} heads {hq}+{hkv} window {window} sinks {sinks}"
    ref = bounded.attention_fwd(w.q, w.k, w.v, cu_q, cu_k, None, None, CODES, B, w.softmax_scale, window, sinks)
    check_fwd(runs[0], ref, f64(w.v), dtype, what)
    out, lse = runs[0]
    dout = workloads.grad_output(w, 5)
    grads = vlp.thd_attn_bwd(q, k, v, out, lse, dout.cuda(), *args, window=window, sink_tokens=sinks)
    ref = bounded.attention_bwd(w.q, w.k, w.v, f64(out), f64(lse), dout, cu_q, cu_k, None, None, CODES, B,
                                w.softmax_scale, window, sinks)
    check_bwd(grads, ref, (w.q, w.k, w.v), dout, w.softmax_scale, dtype, what)
