"""Refusals of the window, sinks, key weights and eviction through the C ABI, before anything is launched (no GPU)."""
import ctypes

import pytest

pytest.importorskip("torch")
from test_rows_host import PAGED, call, lib  # noqa: E402, F401

W3 = (ctypes.c_int64 * 3)(8, 2, 1)
BAD3 = (ctypes.c_int64 * 3)(8, -2, 1)


def _with(base, after, **more):
    out = {}
    for k, v in base.items():
        out[k] = v
        if k == after:
            out.update(more)
    return out


WINDOW = _with(PAGED, "words", left=-1, sinks=0, kw=None, kws=None)
FWD = dict(q=16, k=16, v=16, cuq=16, cuk=16, pq=None, pk=None, causal=None, B=1, longest=0, scale=0.125, out=16, lse=None,
           T=8, hq=4, hkv=2, d=64, dtype=0, left=3, right=0, sinks=1, ws=16, wsb=256, stream=None)
BWD = dict(q=16, k=16, v=16, out=16, lse=16, dout=16, cuq=16, cuk=16, pq=None, pk=None, causal=None, B=1, longest=0,
           scale=0.125, dq=16, dk=16, dv=16, T=8, hq=4, hkv=2, d=64, dtype=0, left=3, right=0, sinks=1, ws=256,
           wsb=1 << 26, stream=None)
EVICT = dict(kc=16, vc=16, st=PAGED["st"], w=16, ws=W3, pages=4, page=4, table=16, ts=4, wide=4, new=None, nts=0, nwide=0,
             lens=64, keep=128, B=1, sinks=1, recent=1, kept=256, width=8, out=192, hkv=2, d=64, dtype=0, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(left=-2), -1), (dict(sinks=-1), -1), (dict(left=3, tree=16, words=1), -2), (dict(kw=16), -1),
    (dict(kw=16, kws=W3), -1), (dict(kw=16, kws=BAD3, lse=16), -1), (dict(kw=18, kws=W3, lse=16), -1),
    (dict(T=0, left=5, sinks=3), 0), (dict(T=0, kw=16, kws=W3, lse=16), 0)])
def test_paged_window_refusals(lib, over, status):  # noqa: F811
    assert call(lib.thd_attn_paged_window, WINDOW, WINDOW, over) == status


@pytest.mark.parametrize("base,fn", [(FWD, "thd_attn_fwd_sinks"), (BWD, "thd_attn_bwd_sinks")])
@pytest.mark.parametrize("over,status", [(dict(sinks=-1), -1), (dict(left=-2), -1), (dict(right=-2), -1),
                                         (dict(T=0), 0), (dict(d=136), -2), (dict(ws=None), -4), (dict(q=8), -1)])
def test_packed_sinks_refusals(lib, base, fn, over, status):  # noqa: F811
    assert call(getattr(lib, fn), base, base, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), -1), (dict(hkv=0), -1), (dict(page=0), -1), (dict(pages=-1), -1), (dict(wide=-1), -1), (dict(ts=3), -1),
    (dict(sinks=-1), -1), (dict(recent=-1), -1), (dict(width=-1), -1), (dict(dtype=2), -2), (dict(d=12), -2),
    (dict(d=136), -2), (dict(d=0), -2), (dict(ws=BAD3), -1), (dict(ws=None), -1), (dict(st=None), -1),
    (dict(st=(ctypes.c_int64 * 6)(512, 128, 64, 512, 124, 64)), -1), (dict(lens=None), -1), (dict(keep=None), -1),
    (dict(out=None), -1), (dict(kept=None), -1), (dict(kc=None), -1), (dict(vc=8), -1), (dict(w=2), -1), (dict(w=None), -1),
    (dict(table=None), -1), (dict(lens=66), -1), (dict(out=64), -1), (dict(out=128), -1), (dict(B=40, out=192), -1),
    (dict(new=16, nwide=-1), -1), (dict(new=16, nwide=4, nts=3), -1), (dict(new=18, nwide=4, nts=4), -1),
    (dict(wide=2 ** 30, ts=2 ** 30), -2), (dict(new=32, nwide=2 ** 30, nts=2 ** 30), -2), (dict(B=2 ** 27, hkv=2), -2),
    (dict(ws=(ctypes.c_int64 * 3)(2 ** 31, 2, 1)), -2),
    (dict(B=0), 0), (dict(B=0, kc=None, w=None, kept=None, lens=None), 0)])
def test_evict_refusals(lib, over, status):  # noqa: F811
    assert call(lib.thd_kv_evict, EVICT, EVICT, over) == status


def test_evict_in_place_takes_the_rows_of_the_table_itself(lib):  # noqa: F811
    """A new table at the old one's address with rows elsewhere is another table over the same pages."""
    assert call(lib.thd_kv_evict, EVICT, EVICT, dict(B=2, new=16, nwide=4, nts=8, keep=160)) == -1
