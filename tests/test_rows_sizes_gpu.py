"""GPU tests: sizes past the library's 32 bits are refused by the bindings."""
import pytest
import torch

from test_paged_gpu import BF16, ints, make, run

pytestmark = pytest.mark.gpu
vlp = pytest.importorskip("variable_length_packed_gb300")


def test_a_head_dim_past_32_bits_is_refused():
    """Not cut to what fits: 2^32 + 64 would pass for 64."""
    wide = 2 ** 32 + 64
    x = torch.empty(wide, dtype=BF16, device="cuda")
    q, c, n, cu = x.view(1, 1, wide), x.view(1, 1, 1, wide), ints([1]), ints([0, 1])
    for call in (lambda: vlp.thd_qk_norm_rope(q, None, cu), lambda: vlp.thd_qk_norm_rope_bwd(q, None, None, None, cu),
                 lambda: vlp.thd_kv_append(q, q, c, c, ints([[0]]), ints([0]), cu),
                 lambda: vlp.thd_attn_paged(q, c, c, ints([[0]]), n, cu)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_a_hint_past_32_bits_is_refused():
    x = make([5], [2], 4, 4, 2, 64, BF16)
    with pytest.raises(ValueError, match="32 bits"):
        run(x, max_seqlen_q=5 - 2 ** 32)   # would pass for 5
