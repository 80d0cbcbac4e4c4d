"""GPU tests of the eviction from a paged cache: bit for bit what the oracle keeps and moves."""
import numpy as np
import pytest
import torch

from oracle import bounded

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")

BF16, FP16 = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def make(keys, keep, page, hkv, d, dtype=BF16, first=False, apart=False, few=False, seed=0, extra=2):
    rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in keys]
    more = [-(-max(0, min(a, b)) // page) for a, b in zip(keep, keys)] if apart else []
    order = rng.permutation(sum(need) + sum(more) + 3)
    at, tables = 0, []
    for want in (need, more):
        table = np.full((len(keys), max(want + [0]) + extra), -1, np.int32)
        for b, n in enumerate(want):
            table[b, :n] = order[at:at + n]
            at += n
        tables.append(table)
    shape = (len(order), hkv, page)
    kv = [torch.randint(-2 ** 15, 2 ** 15, shape + (d,), generator=g, dtype=torch.int16).view(dtype).cuda() for _ in range(2)]
    w = (torch.randint(0, 5, shape, generator=g).float() if few else torch.randn(shape, generator=g).exp()).cuda()
    x = [t.transpose(1, 2) if first else t.transpose(1, 2).contiguous() for t in kv + [w]]
    return dict(kc=x[0], vc=x[1], w=x[2], table=tables[0], new=tables[1] if apart else None, keys=list(keys), keep=list(keep))


def run(x, sinks=0, recent=0, width=None, **over):
    B, hkv = len(x["keys"]), x["kc"].shape[2]
    kept = None if width is None else torch.full((B, hkv, width), 77, dtype=torch.int32, device="cuda")
    kw = dict(new_page_table=None if x["new"] is None else ints(x["new"]), sink_tokens=sinks, recent_tokens=recent, kept=kept)
    kw.update(over)
    lens = vlp.thd_kv_evict(x["kc"], x["vc"], x["w"], ints(x["table"]), ints(x["keys"]), ints(x["keep"]), **kw)
    torch.cuda.synchronize()
    return lens, kw["kept"]


def bits(t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32).cpu().numpy()


def check(x, sinks=0, recent=0, width=None, **over):
    keep = x["keep"] if width is None else [min(n, width) for n in x["keep"]]
    caches = [bits(x["kc"]).copy(), bits(x["vc"]).copy()]
    w = x["w"].cpu().numpy().copy()
    (kc, vc), w_ref, lens_ref, kept_ref = bounded.evict(caches, w, x["table"], x["keys"], keep, x["new"], len(keep), sinks,
                                                        recent)
    lens, kept = run(x, sinks, recent, width, **over)
    assert lens[:len(keep)].tolist() == lens_ref
    if kept is not None:
        for b, heads in enumerate(kept_ref):
            for h, slots in enumerate(heads):
                assert kept[b, h].tolist() == slots + [-1] * (kept.shape[2] - len(slots)), (b, h)
    assert np.array_equal(bits(x["kc"]), kc) and np.array_equal(bits(x["vc"]), vc)
    assert np.array_equal(x["w"].cpu().numpy(), w_ref, equal_nan=True)


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("keys,keep,page,hkv,d,dtype,first,few,sinks,recent", [
    ([1], [1], 16, 1, 8, BF16, False, False, 0, 0),
    ([1, 2, 0, 5], [0, 1, 3, 4], 1, 2, 128, BF16, False, False, 1, 1),
    ([1000], [500], 16, 8, 128, BF16, False, False, 4, 64),
    ([1000, 513, 512, 511, 33], [500, 512, 1, 400, 99], 24, 3, 96, FP16, True, False, 4, 64),
    ([700, 900], [300, 650], 16, 2, 64, BF16, False, True, 0, 0),            # many equal weights
    ([700, 900], [1, 650], 16, 2, 72, BF16, True, True, 0, 200),
    ([700, 900], [100, 650], 64, 2, 40, FP16, False, True, 300, 200),        # the first ones alone, and both ends
    ([5000, 4999], [4998, 4999], 16, 1, 128, BF16, False, False, 0, 0),      # one key goes, and none
    ([4000] * 3, [-5, 0, 2500], 128, 4, 80, BF16, True, True, 7, 9),
    ([60000], [20000], 256, 1, 128, BF16, False, False, 4, 100),             # more weights than shared memory holds
    ([50] * 200, [20] * 200, 8, 2, 32, FP16, False, False, 2, 3),            # more lists than SMs
])
def test_evict_matches_oracle(keys, keep, page, hkv, d, dtype, first, few, sinks, recent, apart):
    x = make(keys, keep, page, hkv, d, dtype, first, apart, few)
    check(x, sinks, recent, width=max(max(keep), 1))


@pytest.mark.parametrize("apart", [False, True])
def test_values_that_are_not_ordinary(apart):
    x = make([600], [250], 16, 2, 64, apart=apart, seed=4)
    rng = np.random.default_rng(4)
    flat = x["w"]
    for value in (float("nan"), float("inf"), -float("inf"), 0.0, -0.0, -1.0, 1e-42, 3.4e38):
        for _ in range(60):
            flat[int(rng.integers(flat.shape[0])), int(rng.integers(16)), int(rng.integers(2))] = value
    check(x, 3, 5, width=250)


def test_all_weights_equal_and_without_kept():
    x = make([900], [300], 16, 2, 64)
    x["w"].zero_()
    check(x, 2, 10, width=300)
    x = make([900, 400], [300, 300], 16, 2, 64, apart=True)
    check(x, 2, 10)


def test_width_bounds_what_is_kept_and_longer_buffers():
    x = make([900, 400], [300, 200], 16, 2, 64)
    check(x, 2, 10, width=123)
    x = make([900, 400], [300, 200], 16, 2, 64)
    lens = torch.full((5,), 9, dtype=torch.int32, device="cuda")
    kept = torch.full((4, 2, 310), 9, dtype=torch.int32, device="cuda")
    check(x, 2, 10, new_lens=lens, kept=kept[:2], batch_size=2)
    assert lens[2:].tolist() == [9] * 3 and torch.all(kept[2:] == 9)


def test_own_table_given_as_the_new_one_is_in_place():
    x, y = make([900], [300], 16, 2, 64), make([900], [300], 16, 2, 64)
    run(x, 2, 10)
    table = ints(y["table"])
    vlp.thd_kv_evict(y["kc"], y["vc"], y["w"], table, ints(y["keys"]), ints(y["keep"]), new_page_table=table,
                     sink_tokens=2, recent_tokens=10)
    assert np.array_equal(bits(x["kc"]), bits(y["kc"])) and torch.equal(x["w"], y["w"])


def test_fewer_columns_of_the_own_table_bound_what_stays():
    x, y = make([900, 700], [300, 290], 16, 2, 64), make([900, 700], [128, 128], 16, 2, 64)
    table = ints(x["table"])
    kept = torch.zeros((2, 2, 400), dtype=torch.int32, device="cuda")
    lens = vlp.thd_kv_evict(x["kc"], x["vc"], x["w"], table, ints(x["keys"]), ints(x["keep"]), new_page_table=table[:, :8],
                            sink_tokens=2, recent_tokens=10, kept=kept)
    run(y, 2, 10)
    assert lens.tolist() == [128, 128] and torch.all(kept[:, :, 128:] == -1)
    assert np.array_equal(bits(x["kc"]), bits(y["kc"])) and torch.equal(x["w"], y["w"])


def test_shared_pages_into_other_pages():
    """Two sequences that share their first pages each keep their own keys."""
    x = make([320, 320], [100, 90], 16, 2, 64, apart=True)
    x["table"][1, :10] = x["table"][0, :10]
    check(x, 1, 20, width=100)


def test_bad_metadata_stays_in_the_buffers():
    x = make([50, 60, 70], [30, 40, 50], 8, 2, 64, apart=True)
    rng = np.random.default_rng(6)
    for new in (None, x["new"]):
        for _ in range(6):
            y = dict(x, table=rng.integers(-5, 60, x["table"].shape), keys=rng.integers(-10, 10**6, 3).tolist(),
                     keep=rng.integers(-10, 10**6, 3).tolist(), new=None if new is None else rng.integers(-5, 60, new.shape))
            run(y, 3, 4)
    x = make([50, 60, 70], [30, 40, 50], 8, 2, 64)
    x["table"][1, 2:4] = (-1, 10 ** 6)
    had = [bits(t).copy() for t in (x["kc"], x["vc"])]
    lens, _ = run(x, 3, 4)
    assert lens.tolist() == [30, 40, 50] and any(not np.array_equal(a, bits(t)) for a, t in zip(had, (x["kc"], x["vc"])))


def test_refusals():
    x = make([50], [30], 8, 2, 64)
    keys = ints(x["keys"])
    args = dict(k_cache=x["kc"], v_cache=x["vc"], key_weights=x["w"], page_table=ints(x["table"]), kv_lens=keys,
                keep_lens=ints(x["keep"]))
    for over, kind in ((dict(k_cache=x["kc"].float()), TypeError), (dict(v_cache=x["vc"][:-1]), ValueError),
                       (dict(key_weights=x["w"][:-1]), ValueError), (dict(key_weights=x["w"].half()), TypeError),
                       (dict(page_table=ints(x["table"]).long()), TypeError), (dict(kv_lens=keys.long()), TypeError),
                       (dict(keep_lens=None), TypeError), (dict(batch_size=2), ValueError),
                       (dict(sink_tokens=-1), ValueError), (dict(recent_tokens=-1), ValueError),
                       (dict(kept=torch.zeros(1, 3, 5, dtype=torch.int32, device="cuda")), ValueError),
                       (dict(new_lens=keys), vlp.ThdError), (dict(new_page_table=ints(x["table"])[0]), ValueError),
                       (dict(k_cache=x["kc"].cpu()), TypeError), (dict(batch_size=-1), ValueError),
                       (dict(k_cache=x["kc"][:1].expand(x["kc"].shape)), ValueError)):
        with pytest.raises(kind):
            vlp.thd_kv_evict(**{**args, **over})
    assert vlp.thd_kv_evict(**{**args, "batch_size": 0}).numel() == 0


@pytest.mark.parametrize("apart", [False, True])
def test_graph_replayed_with_other_lengths_on_two_streams(apart):
    x = make([900, 300], [300, 250], 16, 2, 64, apart=apart)
    table, new = ints(x["table"]), None if x["new"] is None else ints(x["new"])
    keys, keep, lens = ints(x["keys"]), ints(x["keep"]), ints([0, 0])
    kept = torch.zeros(2, 2, 300, dtype=torch.int32, device="cuda")
    fresh = {n: x[n].clone() for n in ("kc", "vc", "w")}
    call = lambda: vlp.thd_kv_evict(x["kc"], x["vc"], x["w"], table, keys, keep, new_page_table=new, sink_tokens=4,  # noqa: E731
                                    recent_tokens=9, new_lens=lens, kept=kept)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for L, K in (([900, 300], [300, 250]), ([500, 20], [100, 30]), ([0, 299], [5, 298])):
        for n, t in fresh.items():
            x[n].copy_(t)
        keys.copy_(ints(L))
        keep.copy_(ints(K))
        y = dict(x, keys=L, keep=K)
        caches = [bits(x["kc"]).copy(), bits(x["vc"]).copy()]
        (kc, vc), w, lens_ref, kept_ref = bounded.evict(caches, x["w"].cpu().numpy(), x["table"], L, K, x["new"], 2, 4, 9)
        graph.replay()
        torch.cuda.synchronize()
        same = [np.array_equal(bits(y["kc"]), kc), np.array_equal(bits(y["vc"]), vc)]
        assert lens.tolist() == lens_ref and same == [True, True]
        assert kept[1, 1].tolist()[:lens_ref[1]] == kept_ref[1][1] and np.array_equal(x["w"].cpu().numpy(), w)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes; the sequence's pages lie at its end, the new ones at its start."""
    page, hkv, d = 16, 1, 128
    pages = (1 << 20) + 100
    kc, vc = (torch.zeros(pages, page, hkv, d, dtype=BF16, device="cuda") for _ in range(2))
    w = torch.zeros(pages, page, hkv, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    at = torch.arange(pages - 64, pages, device="cuda")
    for t in (kc, vc):
        t[at] = torch.randn(64, page, hkv, d, generator=g, device="cuda").to(BF16)
    w[at] = torch.rand(64, page, hkv, generator=g, device="cuda")
    new = torch.arange(32, dtype=torch.int32, device="cuda")[None]
    kept = torch.zeros(1, 1, 400, dtype=torch.int32, device="cuda")
    lens = vlp.thd_kv_evict(kc, vc, w, at.int()[None], ints([1000]), ints([400]), new_page_table=new, kept=kept)
    slots = kept[0, 0].long()
    flat = w[at].flatten()[:1000]
    assert lens.tolist() == [400] and torch.equal(slots, flat.topk(400)[1].sort()[0])
    for t in (kc, vc):
        assert torch.equal(t[new[0].long()].reshape(-1, d)[:400], t[at].reshape(-1, d)[slots])
    assert torch.equal(w[new[0].long()].flatten()[:400], flat[slots])
