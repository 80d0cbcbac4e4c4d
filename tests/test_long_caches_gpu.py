"""Eviction and key weights at the ends of what 32 bits count: lists as wide as they may be, caches of nearly 2^31 keys."""
import numpy as np
import pytest
import torch

from test_evict_gpu import bits, check, ints, make

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")


@pytest.mark.parametrize("keys,keep", [(300, 200), (5000, 0)])
def test_a_list_of_kept_slots_as_wide_as_may_be(keys, keep):
    """Steps behind the end of a list of 2^31 - 1 slots pass 32 bits."""
    x = make([keys], [keep], 16, 1, 8)
    width, guard = 2 ** 31 - 1, 4096
    held = torch.full((width + 2 * guard,), 77, dtype=torch.int32, device="cuda")
    kept = held[guard:guard + width].view(1, 1, width)
    check(x, sinks=2, recent=5)
    y = make([keys], [keep], 16, 1, 8)
    lens = vlp.thd_kv_evict(y["kc"], y["vc"], y["w"], ints(y["table"]), ints([keys]), ints([keep]), sink_tokens=2,
                            recent_tokens=5, kept=kept)
    torch.cuda.synchronize()
    assert lens.tolist() == [keep] and all(np.array_equal(bits(x[n]), bits(y[n])) for n in ("kc", "vc", "w"))
    assert torch.all(held[:guard] == 77) and torch.all(held[guard + width:] == 77)
    slots = kept[0, 0, :keep].tolist()
    assert slots == sorted(set(slots)) and (keep == 0 or (slots[0] >= 0 and slots[-1] == keys - 1))
    for at in range(keep, width, 1 << 28):
        assert torch.all(kept[0, 0, at:at + (1 << 28)] == -1)


@pytest.mark.parametrize("new,left,sinks", [(20, -1, 0), (20, 1000, 3), (130, -1, 0), (1, -1, 0), (1, 1500, 70)])
def test_weights_of_a_cache_of_nearly_2_to_the_31_keys(new, left, sinks):
    """All keys but the last 2048 have no page: the attention reads page 0 for them, zeros here, and they have no weight.
    The last ones score 40 against their 0.  Tolerances as in test_paged_window_gpu; the sum over the zeros is below
    2^31 e^-30 of that over the last keys, its roundings far less."""
    page, d, real = 128, 8, 16
    wide = 2 ** 24 - 1                     # 2^31 - 128 keys
    L, n0 = wide * page, wide * page - real * page
    g = torch.Generator("cuda").manual_seed(new)
    kc = torch.zeros(real + 1, page, 1, d, dtype=torch.bfloat16, device="cuda")
    kc[1:] = 3.5 + 0.25 * torch.randn(real, page, 1, d, generator=g, device="cuda").clamp(-3, 3)
    vc = torch.randn(kc.shape, generator=g, device="cuda").to(torch.bfloat16)
    q = (4 + 0.25 * torch.randn(new, 1, d, generator=g, device="cuda").clamp(-3, 3)).to(torch.bfloat16)
    table = torch.full((1, wide), -1, dtype=torch.int32, device="cuda")
    table[0, -real:] = torch.arange(1, real + 1, device="cuda")
    w = torch.rand(real + 1, page, 1, generator=g, device="cuda")
    had = w.clone()
    _, lse = vlp.thd_attn_paged(q, kc, vc, table, ints([L]), ints([0, new]), window=(left, -1), sink_tokens=sinks,
                                key_weights=w)
    torch.cuda.synchronize()
    # 64 bits: keys n0 .. L - 1, and so many zeros before them
    k, qq = kc[1:].reshape(-1, d).double(), q[:, 0].double()
    own = L - new + torch.arange(new, device="cuda")[:, None]
    key = n0 + torch.arange(real * page, device="cuda")[None]
    see = (key <= own) & (key >= own - left if left >= 0 else True)
    s = (qq @ k.T * d ** -0.5).masked_fill(~see, float("-inf"))
    zeros = n0 if left < 0 else sinks
    want = torch.logaddexp(s.logsumexp(1), torch.full((new,), float(zeros), dtype=torch.float64, device="cuda").log())
    S = float((qq.abs() @ k.abs().T).max()) * d ** -0.5
    e = 136 * 2.0 ** -23 * S + 2.0 ** -21 * (1 + S)
    assert torch.all((lse[0].double() - want).abs() <= e + 4 * 2.0 ** -24 * want.abs())
    added = (s - want[:, None]).exp().sum(0)
    fresh = torch.arange(real * page, device="cuda") >= real * page - new
    expect = torch.where(fresh, 0.0, had[1:].flatten().double()) + added
    share = 2 * e + 2.0 ** -20 * (1 + float(want.abs().max())) + new * 2.0 ** -24
    bound = share * added + 2.0 ** -24 * expect + 2.0 ** -126
    worst = float(((w[1:].flatten().double() - expect).abs() / bound).max())
    print(f"weights: largest share of the bound {worst:.3f}")
    assert worst <= 1.0 and torch.equal(w[0], had[0]) and float(added.max()) > 1e-4
