"""Sizes past 32 bits of the row operators' helpers (no GPU): refused, not cut to the bits that fit."""
import pytest

pytest.importorskip("torch")

import variable_length_packed_gb300 as vlp  # noqa: E402
from variable_length_packed_gb300 import build as vbuild  # noqa: E402


@pytest.mark.parametrize("head_dim", [2**32 + 64, -2**32 + 64, 2**31, -8])
def test_workspace_of_a_head_dim_that_does_not_fit(head_dim):
    vbuild.build()
    assert vlp.thd_attn_paged_workspace_size(head_dim) == 0
    assert vlp.thd_qk_norm_rope_bwd_workspace_size(head_dim) == 0
