"""Eviction at the end of what 32 bits count: lists as wide as they may be."""
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
