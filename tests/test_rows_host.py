"""Refusals of the row operators, through the C ABI, before anything is launched (no GPU)."""
import ctypes

import pytest

pytest.importorskip("torch")
import torch  # noqa: E402

import variable_length_packed_gb300 as vlp  # noqa: E402
from variable_length_packed_gb300 import build as vbuild  # noqa: E402

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    vbuild.build()
    return vlp.load_library()


def call(fn, order, base, over):
    unknown = set(over) - set(base)
    assert not unknown, unknown
    args = {**base, **over}
    return fn(*[args[k] for k in order])


ROPE = dict(q=16, qs=256, k=16, ks=128, wq=16, wk=16, w32=0, eps=1e-6, cos=16, sin=16, rows=8, rot=64, inter=0, cu=16,
            pad=None, off=None, B=1, qo=16, ko=16, T=0, hq=4, hkv=2, d=64, dtype=0, stream=None)
BWD = dict(gq=16, gk=16, q=16, qs=256, k=16, ks=128, wq=16, wk=16, w32=0, eps=1e-6, cos=16, sin=16, rows=8, rot=64,
           inter=0, cu=16, pad=None, off=None, B=1, dq=16, dqs=256, dk=16, dks=128, dwq=16, dwk=16, T=8, hq=4, hkv=2,
           d=64, dtype=0, ws=16, wsb=1 << 20, stream=None)
STRIDES = (512, 128, 64, 512, 128, 64)
APPEND = dict(q=16, qs=256, k=16, ks=128, v=16, vs=128, wq=16, wk=16, w32=0, eps=1e-6, cos=16, sin=16, rows=8, rot=64,
              inter=0, pos=None, cu=16, pad=None, lens=16, B=1, qo=16, kc=16, vc=16,
              st=(ctypes.c_int64 * 6)(*STRIDES), pages=4, page=4, table=16, ts=4, wide=4, T=8, hq=4, hkv=2, d=64,
              dtype=0, stream=None)
PAGED = dict(q=16, kc=16, vc=16, st=(ctypes.c_int64 * 6)(*STRIDES), pages=4, page=4, table=16, ts=4, wide=4, lens=16,
             cu=16, pad=None, B=1, longest=0, tree=None, words=0, scale=0.125, out=16, lse=None, T=8, hq=4, hkv=2,
             d=64, dtype=0, ws=16, wsb=1 << 26, stream=None)

COMMON = [(dict(B=-1), -1), (dict(T=-1), -1), (dict(dtype=5), -2), (dict(d=24), -2), (dict(d=144), -2), (dict(d=8), -2),
          (dict(rot=8), -2), (dict(rot=80), -2), (dict(rot=-16), -2), (dict(eps=NAN), -1), (dict(eps=-1.0), -1),
          (dict(eps=INF), -1), (dict(cos=None), -1), (dict(sin=None), -1), (dict(cos=8), -1), (dict(rows=0), -1),
          (dict(wq=8), -1), (dict(wk=4), -1), (dict(w32=2), -1), (dict(cu=None, T=8), -1), (dict(cu=6), -1),
          (dict(pad=6), -1), (dict(hq=-1), -1), (dict(hkv=-1), -1)]


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(T=8, q=None), -1), (dict(T=8, qs=248), -1), (dict(T=8, qs=260), -1), (dict(T=8, ks=120), -1),
    (dict(T=8, q=24), -1), (dict(T=8, qo=None), -1), (dict(T=8, ko=8), -1), (dict(hq=0, hkv=0), -1), (dict(off=2), -1),
    (dict(T=2**31 - 1, hq=128, qs=128 * 64), -2), (dict(), 0), (dict(T=0, q=None, k=None, qo=None, ko=None), 0)])
def test_rope_refusals(lib, over, status):
    assert call(lib.thd_qk_norm_rope, ROPE, ROPE, over) == status


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(gq=None), -1), (dict(gk=24), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(dq=None), -1),
    (dict(dqs=128), -1), (dict(dks=132), -1), (dict(dwq=None), -1), (dict(wk=None), -1), (dict(dwk=2), -1),
    (dict(ws=None), -4), (dict(ws=8), -4), (dict(wsb=1000), -4), (dict(hq=0, hkv=0), -1)])
def test_rope_bwd_refusals(lib, over, status):
    assert call(lib.thd_qk_norm_rope_bwd, BWD, BWD, over) == status


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(hkv=0), -1), (dict(pages=-1), -1), (dict(page=0), -1), (dict(wide=-1), -1), (dict(ts=3), -1),
    (dict(st=None), -1), (dict(st=(ctypes.c_int64 * 6)(512, 128, 60, 512, 128, 64)), -1),
    (dict(st=(ctypes.c_int64 * 6)(512, 128, 64, 512, -128, 64)), -1), (dict(lens=None), -1), (dict(table=None), -1),
    (dict(table=18), -1), (dict(pos=2), -1), (dict(lens=2), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(vs=100), -1), (dict(kc=None), -1), (dict(vc=24), -1), (dict(qo=None), -1),
    (dict(T=0, k=None, v=None, q=None), 0)])
def test_append_refusals(lib, over, status):
    assert call(lib.thd_kv_append, APPEND, APPEND, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), -1), (dict(T=-1), -1), (dict(longest=-1), -1), (dict(hq=0), -1), (dict(hkv=0), -1),
    (dict(hq=3), -2), (dict(d=12), -2), (dict(d=136), -2), (dict(dtype=3), -2), (dict(scale=0.0), -1),
    (dict(scale=NAN), -1), (dict(scale=INF), -1), (dict(pages=-1), -1), (dict(page=0), -1), (dict(wide=-1), -1),
    (dict(ts=2), -1), (dict(st=None), -1), (dict(st=(ctypes.c_int64 * 6)(512, 130, 64, 512, 128, 64)), -1),
    (dict(q=None), -1), (dict(q=8), -1), (dict(out=None), -1), (dict(out=4), -1), (dict(lse=2), -1),
    (dict(kc=None), -1), (dict(vc=8), -1), (dict(table=None), -1), (dict(lens=None), -1), (dict(cu=None), -1),
    (dict(lens=2), -1), (dict(cu=2), -1), (dict(pad=2), -1), (dict(table=2), -1), (dict(tree=12, words=1), -1),
    (dict(tree=16, words=0), -1), (dict(ws=None), -4), (dict(ws=8), -4), (dict(wsb=100), -4),
    (dict(T=2**30, hq=4, hkv=2), -2), (dict(wide=2**20, ts=2**20, page=2**12), -2),
    (dict(T=0, q=None, out=None), 0)])
def test_paged_refusals(lib, over, status):
    assert call(lib.thd_attn_paged, PAGED, PAGED, over) == status


@pytest.mark.parametrize("side", ["hq", "hkv"])
@pytest.mark.parametrize("heads", [2**25, 2**30])
def test_rows_of_too_many_values_are_refused(lib, side, heads):
    over = {side: heads, "qs": heads * 64, "ks": heads * 64}   # 2^31 values of a row and more
    assert call(lib.thd_qk_norm_rope, ROPE, ROPE, {**over, "T": 8}) == -2
    assert call(lib.thd_qk_norm_rope_bwd, BWD, BWD, {**over, "dqs": heads * 64, "dks": heads * 64}) == -2
    assert call(lib.thd_kv_append, APPEND, APPEND, {**over, "vs": heads * 64}) == -2


def test_workspace_sizes(lib):
    assert vlp.thd_qk_norm_rope_bwd_workspace_size(128) > 0 and vlp.thd_qk_norm_rope_bwd_workspace_size(24) == 0
    assert vlp.thd_attn_paged_workspace_size(8) > 0 and vlp.thd_attn_paged_workspace_size(132) == 0


def test_cpu_tensors_are_refused(lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    cache = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)
    for f in (lambda: vlp.thd_qk_norm_rope(x, x, cu), lambda: vlp.thd_qk_norm_rope_bwd(x, x, x, x, cu),
              lambda: vlp.thd_kv_append(x, x, cache, cache, cu[None], cu, cu),
              lambda: vlp.thd_attn_paged(x, cache, cache, cu[None], cu, cu)):
        with pytest.raises(TypeError, match="CUDA"):
            f()
