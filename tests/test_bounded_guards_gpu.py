"""Bad metadata of the operators that bound long sequences: every buffer that a call writes lies between guard values,
which stay as they were, and what the metadata still determines is compared with the oracle."""
import numpy as np
import pytest
import torch

import workloads
from oracle import bounded
from test_evict_gpu import check as check_evict
from test_evict_gpu import ints, make as make_evict
from test_paged_gpu import BF16, FP16, make as make_paged

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")

GUARD = 1 << 14   # bytes on each side


class Guarded:
    """Tensors inside larger buffers."""

    def __init__(self):
        self.held = []

    def put(self, t):
        """A copy of t, whole or a transposed whole one, between guard bytes."""
        flip = not t.is_contiguous()
        src = t.transpose(1, 2) if flip else t
        size = src.numel() * src.element_size()
        buf = torch.full((size + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        inner = buf[GUARD:GUARD + size].view(src.dtype).view(src.shape)
        inner.copy_(src)
        self.held.append((buf, size))
        return inner.transpose(1, 2) if flip else inner

    def check(self):
        torch.cuda.synchronize()
        for buf, size in self.held:
            assert torch.all(buf[:GUARD] == 0xA5) and torch.all(buf[GUARD + size:] == 0xA5)


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("apart", [False, True])
def test_evict_with_bad_tables_and_lengths(apart, first):
    base = make_evict([50, 60, 70], [30, 40, 50], 8, 2, 64, apart=apart, first=first)
    rng = np.random.default_rng(6)
    pages, page, hkv, _ = base["kc"].shape
    room = base["table"].shape[1] * page
    to_room = base["new"].shape[1] * page if apart else room
    for _ in range(8):
        g = Guarded()
        kc, vc, w = (g.put(base[n]) for n in ("kc", "vc", "w"))
        table = rng.integers(-5, 2 * pages, base["table"].shape)
        new = rng.integers(-5, 2 * pages, base["new"].shape) if apart else None
        keys, keep = (rng.integers(-10, 2 * room, 3).tolist() for _ in range(2))
        width = int(rng.integers(1, room))
        kept, lens = g.put(torch.full((3, hkv, width), 77, dtype=torch.int32, device="cuda")), g.put(ints([9, 9, 9]))
        before = base["w"].cpu().numpy()
        vlp.thd_kv_evict(kc, vc, w, ints(table), ints(keys), ints(keep), new_page_table=ints(new) if apart else None,
                         sink_tokens=3, recent_tokens=4, kept=kept, new_lens=lens)
        g.check()
        real = (table >= 0) & (table < pages)
        for b in range(3):
            L = min(max(keys[b], 0), room)
            K = min(max(keep[b], 0), L, to_room, width)
            assert int(lens[b]) == K
            at = np.arange(L)
            for h in range(hkv):
                named = real[b, at // page]
                had = np.where(named, before[np.where(named, table[b, at // page], 0), at % page, h], 0.0)
                assert kept[b, h].tolist() == bounded.evict_keep(had, L, K, 3, 4) + [-1] * (width - K), (b, h)


@pytest.mark.parametrize("apart", [False, True])
def test_evict_where_the_table_names_no_page(apart):
    """Keys of no page count with weight 0 and do not move, nor does a key whose new slot has none."""
    x = make_evict([50, 60, 70], [30, 40, 50], 8, 2, 64, apart=apart)
    x["table"][1, 2:4] = (-1, 10 ** 6)
    x["table"][0, 0] = 2 ** 31 - 1
    if apart:
        x["new"][2, 1] = -(2 ** 31)
    check_evict(x, 3, 4, width=50)


@pytest.mark.parametrize("left,sinks", [(-1, 0), (20, 3)])
@pytest.mark.parametrize("hq,hint,room", [(4, 0, 0), (4, 2, 1 << 20), (32, 0, 0)])
def test_paged_attention_and_key_weights(left, sinks, hq, hint, room):
    """Tiles of 16 rows with and without kept scores, and of 128 rows."""
    x = make_paged([50, 60, 70], [3, 4, 5], 8, hq, 2, 64, BF16)
    rng = np.random.default_rng(7)
    pages, page, hkv, d = x["kc"].shape
    T = x["q"].shape[0]
    for _ in range(8):
        g = Guarded()
        kc, vc = (g.put(x[n].nan_to_num(0, 0, 0)) for n in ("kc", "vc"))
        had = [kc.clone(), vc.clone()]
        w = g.put(torch.rand(pages, page, hkv, device="cuda"))
        out, lse = g.put(torch.zeros_like(x["q"])), g.put(torch.zeros(hq, T, device="cuda"))
        work = g.put(torch.zeros(vlp.thd_attn_paged_workspace_size(d) + room, dtype=torch.uint8, device="cuda"))
        vlp.thd_attn_paged(x["q"], kc, vc, ints(rng.integers(-5, 2 * pages, x["table"].shape)),
                           ints(rng.integers(-10, 10 ** 6, 3)), ints(rng.integers(-30, 30, 4)), max_seqlen_q=hint,
                           window=(left, -1), sink_tokens=sinks, key_weights=w, out=out, lse=lse, workspace=work)
        g.check()
        assert int(work[8:12].view(torch.int32).item()) == 0   # no wait ran out
        assert torch.equal(kc, had[0]) and torch.equal(vc, had[1])


@pytest.mark.parametrize("d,dtype,hq,hkv", [(128, BF16, 4, 2), (64, FP16, 3, 1), (40, BF16, 2, 2)])
def test_packed_attention_and_gradients(d, dtype, hq, hkv):
    """Starts and lengths in any order, past the rows and negative."""
    T = 5000
    w = workloads.from_lengths("bad", [T], [0], heads_q=hq, heads_kv=hkv, head_dim=d, dtype=dtype, seed=1)
    rng = np.random.default_rng(8)
    q, k, v = w.q.cuda(), w.k.cuda(), w.v.cuda()
    dout = workloads.grad_output(w, 7).cuda()
    codes = torch.tensor([0, 1, 2, 1, 0, 2], dtype=torch.uint8, device="cuda")
    size = vlp.load_library().thd_attn_bwd_sinks_workspace_size
    for window, sinks in (((100, 0), 4), ((0, -1), 130), ((-1, 50), 7), ((300, 20), 1000)):
        for _ in range(2):
            cu_q, cu_k, pad_q, pad_k = (ints(rng.integers(-1000, 7000, n)) for n in (7, 7, 6, 6))
            g = Guarded()
            out, lse = g.put(torch.zeros_like(q)), g.put(torch.zeros(hq, T, device="cuda"))
            work = g.put(torch.zeros(vlp.thd_attn_workspace_size(), dtype=torch.uint8, device="cuda"))
            vlp.thd_attn_fwd(q, k, v, cu_q, cu_k, pad_q, pad_k, codes, 6, window=window, sink_tokens=sinks, out=out, lse=lse,
                             workspace=work)
            torch.cuda.synchronize()
            assert int(work[8:12].view(torch.int32).item()) == 0
            if d != 40:
                grads = [g.put(torch.zeros_like(t)) for t in (q, k, v)]
                need = size(T, hq, hkv, d, 6, window[0], sinks)
                work = g.put(torch.zeros(need, dtype=torch.uint8, device="cuda"))
                vlp.thd_attn_bwd(q, k, v, out, lse, dout, cu_q, cu_k, pad_q, pad_k, codes, 6, window=window,
                                 sink_tokens=sinks, dq=grads[0], dk=grads[1], dv=grads[2], workspace=work)
                torch.cuda.synchronize()
                assert int(work[8:12].view(torch.int32).item()) == 0
            g.check()
