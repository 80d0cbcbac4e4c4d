"""Sizes and window extents past 32 bits of the packed attention calls (no GPU): refused, not cut to the bits that fit."""
import pytest

torch = pytest.importorskip("torch")

import variable_length_packed_gb300 as vlp  # noqa: E402

BIG = 2 ** 31


def rows(T, heads, d=8):
    return torch.empty(T, heads, d, dtype=torch.bfloat16, device="meta")


def calls(q, k, **over):
    cu = torch.zeros(2, dtype=torch.int32)
    lse = torch.empty(q.shape[1], q.shape[0], device="meta")
    return (lambda: vlp.thd_attn_fwd(q, k, k, cu, cu, **over), lambda: vlp.thd_attn_bwd(q, k, k, q, lse, q, cu, cu, **over))


@pytest.mark.parametrize("window", [(BIG, 0), (0, BIG), (2 ** 32 + 64, 0), (-1, 2 ** 32), (2 ** 40, 2 ** 40)])
def test_window_extents(window):
    q = rows(4, 2)
    for call in calls(q, q, window=window):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    for call in calls(q, q, window=(BIG - 1, BIG - 1)):   # the largest: on to the next check
        with pytest.raises(TypeError, match="CUDA"):
            call()


@pytest.mark.parametrize("T,hq,hkv,d", [(BIG, 1, 1, 8), (2 ** 32 + 5, 1, 1, 8), (1, 2 ** 32 + 2, 1, 8), (1, 2, BIG, 8),
                                        (1, 1, 1, 2 ** 32 + 8)])
def test_sizes(T, hq, hkv, d):
    q, k = rows(T, hq, d), rows(T, hkv, d)
    cu = torch.zeros(2, dtype=torch.int32)
    for call in calls(q, k) + (lambda: vlp.thd_attn_fwd_noalloc(q, k, k, cu, cu, None, None, None, 1, 0, 1.0, q),):
        with pytest.raises(ValueError, match="32 bits"):
            call()
