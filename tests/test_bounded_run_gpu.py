"""The operators that bound a cache, one after another as a serving program calls them: a prompt in chunks, decoding
steps that append and add up the keys' weights, evictions in place and into other pages; every step against the
oracle on what the caches hold at that moment."""
import numpy as np
import pytest
import torch

from oracle import bounded
from test_evict_gpu import bits
from test_paged_gpu import BF16, ints
from test_paged_window_gpu import check

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")


@pytest.mark.parametrize("left,sinks", [(-1, 0), (150, 3)])
def test_prompt_decoding_and_evictions(left, sinks):
    rng, g = np.random.default_rng(0), torch.Generator("cuda").manual_seed(0)
    B, hq, hkv, d, page, wide, pages = 3, 8, 2, 64, 16, 40, 260
    order = rng.permutation(pages).astype(np.int32)
    table, spare = order[:B * wide].reshape(B, wide), order[B * wide:2 * B * wide].reshape(B, wide)
    kc, vc = (torch.zeros(pages, page, hkv, d, dtype=BF16, device="cuda") for _ in range(2))
    w = torch.full((pages, hkv, page), float("nan"), device="cuda").transpose(1, 2)   # new keys begin with none
    lens = ints([0] * B)
    angles = torch.arange(2000, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2) / d)
    cos, sin = angles.cos().float().cuda(), angles.sin().float().cuda()
    positions = np.zeros(B, np.int64)
    steps = [[120, 37, 200], [90, 300, 1]] + [[1, 1, 1]] * 3 + ["keep"] + [[1, 1, 1]] * 3 + ["move"] + [[1, 0, 4], [40, 1, 1]]
    for step in steps:
        if isinstance(step, str):
            keep = ints([100, 250, 60])
            had = [bits(kc).copy(), bits(vc).copy()]
            ref, w_ref, n_ref, kept_ref = bounded.evict(had, w.cpu().numpy(), table, lens.tolist(), keep.tolist(),
                                                        spare if step == "move" else None, B, 4, 20)
            kept = torch.zeros(B, hkv, 250, dtype=torch.int32, device="cuda")
            lens = vlp.thd_kv_evict(kc, vc, w, ints(table), lens, keep, sink_tokens=4, recent_tokens=20, kept=kept,
                                    new_page_table=ints(spare) if step == "move" else None)
            assert lens.tolist() == n_ref
            assert all(kept[b, h, :len(s)].tolist() == s for b, heads in enumerate(kept_ref) for h, s in enumerate(heads))
            assert np.array_equal(bits(kc), ref[0]) and np.array_equal(bits(vc), ref[1])
            assert np.array_equal(w.cpu().numpy(), w_ref, equal_nan=True)
            if step == "move":
                table, spare = spare, table
            continue
        cu = np.concatenate([[0], np.cumsum(step)])
        rows = [torch.randn(int(cu[-1]), h, d, generator=g, device="cuda").to(BF16) for h in (hq, hkv, hkv)]
        at = np.concatenate([p + np.arange(n) for p, n in zip(positions, step)])
        positions += step
        q = vlp.thd_kv_append(rows[1], rows[2], kc, vc, ints(table), lens, ints(cu), q=rows[0], rope_cos=cos, rope_sin=sin,
                              positions=ints(at))
        lens = lens + ints(step)
        had = w.clone()
        got = vlp.thd_attn_paged(q, kc, vc, ints(table), lens, ints(cu), max_seqlen_q=max(step), window=(left, 0 if left >= 0 else -1),
                                 sink_tokens=sinks, key_weights=w)
        torch.cuda.synchronize()
        x = dict(q=q, kc=kc, vc=vc, table=table, keys=np.array(lens.tolist()), cu=cu, padded=None, B=B, tree=None)
        # a key that no token sees keeps what it had, and so does every place of no key
        fresh = torch.isnan(had) & ~torch.isnan(w)
        assert torch.all(torch.isnan(had) | ~torch.isnan(w)) and int(fresh.sum()) <= hkv * sum(step)
        check(x, got, left, sinks, had.nan_to_num(0.0), w.nan_to_num(0.0))


def test_training_step_with_window_and_sinks():
    """Norm and rotation, attention under a window with sinks, and all gradients back, against autograd in 64 bits."""
    g = torch.Generator().manual_seed(3)
    lens, hq, hkv, d, window, sinks = [150, 1, 300, 77], 4, 2, 64, (60, 0), 5
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    x = [torch.randn(T, h, d, generator=g).to(BF16) for h in (hq, hkv, hkv)]
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2))
    dout = torch.randn(T, hq, d, generator=g).to(BF16)
    angles = torch.arange(300, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2) / d)
    cos, sin = angles.cos().float(), angles.sin().float()
    # 64 bits
    leaf = [t.double().requires_grad_() for t in x + [wq, wk]]
    pos = torch.cat([torch.arange(n) for n in lens])

    def turned(t, w):
        n = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = n[..., :d // 2], n[..., d // 2:]
        c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
        return torch.cat([a * c - b * s, b * c + a * s], -1)
    q64, k64 = turned(leaf[0], leaf[3]), turned(leaf[1], leaf[4])
    parts = []
    for b, n in enumerate(lens):
        r = slice(int(cu[b]), int(cu[b + 1]))
        seen = torch.from_numpy(bounded.sees(n, n, 1, window, sinks))
        k, v = (t[r].repeat_interleave(hq // hkv, 1) for t in (k64, leaf[2]))
        z = torch.einsum("ihd,jhd->hij", q64[r], k) * d ** -0.5
        parts.append(torch.einsum("hij,jhd->ihd", z.masked_fill(~seen, -torch.inf).softmax(-1), v))
    (torch.cat(parts) * dout.double()).sum().backward()
    # the library
    dev = [t.cuda() for t in x]
    tables = dict(rope_cos=cos.cuda(), rope_sin=sin.cuda(), q_weight=wq.cuda(), k_weight=wk.cuda())
    c, codes = ints(cu), torch.ones(4, dtype=torch.uint8, device="cuda")
    q, k = vlp.thd_qk_norm_rope(dev[0], dev[1], c, **tables)
    out, lse = vlp.thd_attn_fwd(q, k, dev[2], c, c, seq_is_causal=codes, window=window, sink_tokens=sinks)
    dq, dk, dv = vlp.thd_attn_bwd(q, k, dev[2], out, lse, dout.cuda(), c, c, seq_is_causal=codes, window=window,
                                  sink_tokens=sinks)
    dq, dk, dwq, dwk = vlp.thd_qk_norm_rope_bwd(dq, dk, dev[0], dev[1], c, **tables)
    # each stage rounds to bf16 (2^-8 relative): q, k, P, dS, out (through D), dq, dk and the output, each relative to terms of
    # the size of the gradients; in the norm over all values they add up as their squares: sqrt(8) 2^-8 = 1.1e-2
    for got, t in zip((dq, dk, dv, dwq, dwk), leaf):
        r = t.grad
        assert (got.double().cpu() - r).norm() <= 8 ** 0.5 * 2.0 ** -8 * r.norm()
