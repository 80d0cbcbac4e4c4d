"""Bindings of the operators around packed attention: head norm and rotation with its
gradients, appending to a paged key/value cache, and attention over it.

Like the rest of the package these only check and marshal tensors and allocate outputs;
the work is in the library's kernels (include/thd_attn.h states each operator).
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import THD_BF16, THD_FP16, THD_OK, ThdError, _check_metadata, load_library

# the current stream's handle without the Stream object around it (2 us a call)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_F32 = torch.float32
_Places = ctypes.c_int64 * 6
_COUNT_MAX = 2 ** 31 - 1   # the library's counts are C ints, which ctypes would cut to 32 bits without a word
_CODES = {torch.bfloat16: THD_BF16, torch.float16: THD_FP16}


@functools.lru_cache(maxsize=None)
def _workspace_size(name, head_dim):
    size = getattr(load_library(), name)
    return int(size(head_dim)) if abs(head_dim) <= _COUNT_MAX else 0


def thd_qk_norm_rope_bwd_workspace_size(head_dim):
    """Bytes of device workspace thd_qk_norm_rope_bwd needs; 0 for an unsupported head_dim."""
    return _workspace_size("thd_qk_norm_rope_bwd_workspace_size", int(head_dim))


def thd_attn_paged_workspace_size(head_dim):
    """Bytes of device workspace thd_attn_paged needs; 0 for an unsupported head_dim."""
    return _workspace_size("thd_attn_paged_workspace_size", int(head_dim))


def _addr(t):
    return None if t is None else t.data_ptr()


def _too_large(name):
    return ValueError(f"{name}: a size does not fit the library's 32 bits")


def _on(t, name, device):
    """A tensor on `device`, which is a GPU's."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call on {device}")


def _whole(t, name, device, dtype, shape=None):
    """A contiguous tensor of one dtype (and shape) on `device`; None passes."""
    if t is None:
        return
    if (type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == device.index and t.is_contiguous()
            and (shape is None or t.shape == shape)):   # the usual case, without building devices to compare
        return
    _on(t, name, device)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name, device, dtype, shape=None):
    """Row stride of a [T, heads, head_dim] tensor whose rows are whole but may lie apart."""
    if (type(t) is torch.Tensor and t.get_device() == device.index and t.dtype is dtype and t.is_contiguous()
            and (t.shape == shape if shape is not None else t.dim() == 3)):   # the usual case in few steps
        _, h, d = t.shape
        return h * d
    _on(t, name, device)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, heads, head_dim]")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    T, h, d = t.shape
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    row, head, one = t.stride()
    if (d > 1 and one != 1) or (h > 1 and head != d):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if T <= 1:
        return h * d
    if row < h * d:
        raise ValueError(f"{name}: rows overlap (stride {row} for {h * d} values)")
    return row


def _dtype_code(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor (no CPU path exists)")
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bf16 or fp16")
    return code


def _meta(device, batch_size, cu, padded, name, per_seq):
    """Batch size and checks of the int32 metadata; per_seq: a tensor of >= batch_size entries, or None."""
    if cu is None:
        raise TypeError("cu_seqlens must be an int32 tensor")
    _whole(cu, "cu_seqlens", device, torch.int32)
    if batch_size is None:
        batch_size = cu.numel() - 1
    batch_size = int(batch_size)
    if padded is not None:
        _whole(padded, "cu_seqlens_padded", device, torch.int32)
    if batch_size < 0 or cu.numel() <= batch_size or (padded is not None and padded.numel() < batch_size):
        _check_metadata(batch_size, cu, None, padded)
    if per_seq is not None:
        _whole(per_seq, name, device, torch.int32)
        if per_seq.numel() < batch_size:
            raise ValueError(f"{name} holds {per_seq.numel()} entries, batch_size {batch_size} needs as many")
    return batch_size


def _tables(cos, sin, device, d):
    """(rows, rotary_dim) of the angle tables; (0, 0) without them."""
    if cos is None and sin is None:
        return 0, 0
    if cos is None or sin is None:
        raise ValueError("rope_cos and rope_sin come together")
    if type(cos) is torch.Tensor is type(sin):   # the usual case in few steps
        shape, index = cos.shape, device.index
        if (cos.dtype is _F32 is sin.dtype and sin.shape == shape and len(shape) == 2 and shape[0] > 0
                and 2 * shape[1] <= d and cos.get_device() == index == sin.get_device() and cos.is_contiguous()
                and sin.is_contiguous()):
            return shape[0], 2 * shape[1]
    _whole(cos, "rope_cos", device, torch.float32)
    _whole(sin, "rope_sin", device, torch.float32, cos.shape)
    if cos.dim() != 2 or 2 * cos.shape[1] > d:
        raise ValueError("rope_cos and rope_sin must be [positions, rotary_dim / 2] with rotary_dim <= head_dim")
    if cos.shape[0] < 1 and cos.shape[1] > 0:
        raise ValueError("rope_cos and rope_sin hold no position")
    return cos.shape[0], 2 * cos.shape[1]


def _weights(wq, wk, device, d, dtype):
    """1 if the norm weights are fp32, 0 if they are of the rows' dtype."""
    if wq is None and wk is None:
        return 0
    if type(wq) is torch.Tensor is type(wk):   # the usual case in few steps
        kind, index = wq.dtype, device.index
        if (kind is wk.dtype and (kind is dtype or kind is _F32) and wq.shape == (d,) == wk.shape
                and wq.get_device() == index == wk.get_device() and wq.is_contiguous() and wk.is_contiguous()):
            return 1 if kind is _F32 else 0
    fp32 = 0
    for name, w in (("q_weight", wq), ("k_weight", wk)):
        if w is not None:
            if not isinstance(w, torch.Tensor) or (w.dtype is not dtype and w.dtype is not torch.float32):
                raise TypeError(f"{name} must be a float32 or {dtype} tensor")
            _whole(w, name, device, w.dtype, (d,))
            fp32 = int(w.dtype is torch.float32)
    if wq is not None and wk is not None and wq.dtype is not wk.dtype:
        raise TypeError("q_weight and k_weight must share a dtype")
    return fp32


def _call(name, device, *args):
    """The library's entry point on the current stream of `device`."""
    fn = getattr(load_library(), name)
    if torch.cuda.current_device() == device.index:
        st = fn(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device.index))
    if st != THD_OK:
        raise ThdError(st, name)


def thd_qk_norm_rope(q, k, cu_seqlens, rope_cos=None, rope_sin=None, cu_seqlens_padded=None, batch_size=None,
                     position_offsets=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None,
                     k_out=None):
    """RMS norm of each query and key head and the rotation by its row's position, in one pass.

    q: [T, Hq, d], k: [T, Hkv, d] or None (bf16 or fp16; rows may lie apart, as parts of a fused
    projection do).  rope_cos / rope_sin: float32 [positions, rotary_dim / 2] or None (no
    rotation); position i + position_offsets[b] for row i of sequence b.  q_weight / k_weight: [d]
    in q's dtype or float32, or None (that side is not normed).  interleaved: pairs (2c, 2c+1)
    instead of (c, c + rotary_dim / 2).  q_out / k_out may be q / k (contiguous ones).
    Returns (q_out [T, Hq, d], k_out [T, Hkv, d] or None), zeros on rows of no sequence.
    """
    code = _dtype_code(q, "q")
    dev, dtype = q.device, q.dtype
    qs = _rows(q, "q", dev, dtype)
    T, hq, d = q.shape
    hkv, ks = 0, 0
    if k is not None:
        ks = _rows(k, "k", dev, dtype)
        hkv = k.shape[1]
        if k.shape[0] != T or k.shape[2] != d:
            raise ValueError("k must be [T, Hkv, head_dim] with q's T and head_dim")
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    B = _meta(dev, batch_size, cu_seqlens, cu_seqlens_padded, "position_offsets", position_offsets)
    rows, rot = _tables(rope_cos, rope_sin, dev, d)
    fp32 = _weights(q_weight, k_weight, dev, d, dtype)
    if q_out is None:
        q_out = torch.empty((T, hq, d), dtype=dtype, device=dev)
    else:
        _whole(q_out, "q_out", dev, dtype, q.shape)
    if k is not None:
        if k_out is None:
            k_out = torch.empty((T, hkv, d), dtype=dtype, device=dev)
        else:
            _whole(k_out, "k_out", dev, dtype, k.shape)
    if (T | hq | hkv | d | rows | B) > _COUNT_MAX:   # the or of sizes in range is in range
        raise _too_large("thd_qk_norm_rope")
    _call("thd_qk_norm_rope", dev, _addr(q), qs, _addr(k), ks, _addr(q_weight), _addr(k_weight), fp32, float(eps),
          _addr(rope_cos), _addr(rope_sin), rows, rot, int(bool(interleaved)), cu_seqlens.data_ptr(),
          _addr(cu_seqlens_padded), _addr(position_offsets), B, _addr(q_out), _addr(k_out), T, hq, hkv, d, code)
    return q_out, k_out


def thd_qk_norm_rope_bwd(grad_q, grad_k, q, k, cu_seqlens, rope_cos=None, rope_sin=None, cu_seqlens_padded=None,
                         batch_size=None, position_offsets=None, q_weight=None, k_weight=None, eps=1e-6,
                         interleaved=False, dq=None, dk=None, dq_weight=None, dk_weight=None, workspace=None):
    """Gradients of thd_qk_norm_rope: (dq, dk, dq_weight, dk_weight), the weights' float32 [d] and
    None where there is no weight.  grad_q / grad_k: gradients of q_out / k_out, contiguous; q / k:
    the forward's inputs (where no weight is given they may be None).  dq / dk may be parts of
    a fused gradient (rows apart), or grad_q / grad_k themselves."""
    code = _dtype_code(grad_q, "grad_q")
    dev, dtype = grad_q.device, grad_q.dtype
    _whole(grad_q, "grad_q", dev, dtype)
    if grad_q.dim() != 3:
        raise ValueError("grad_q must be [T, heads, head_dim]")
    T, hq, d = grad_q.shape
    hkv = 0
    if grad_k is not None:
        _whole(grad_k, "grad_k", dev, dtype)
        if grad_k.dim() != 3 or grad_k.shape[0] != T or grad_k.shape[2] != d:
            raise ValueError("grad_k must be [T, Hkv, head_dim] with grad_q's T and head_dim")
        hkv = grad_k.shape[1]
    elif dk is not None or k_weight is not None or dk_weight is not None:
        raise ValueError("dk, k_weight and dk_weight need grad_k")
    fp32 = _weights(q_weight, k_weight, dev, d, dtype)
    qs = ks = 0
    if q_weight is not None:
        qs = _rows(q, "q", dev, dtype, grad_q.shape)
    if k_weight is not None:
        ks = _rows(k, "k", dev, dtype, grad_k.shape)
    B = _meta(dev, batch_size, cu_seqlens, cu_seqlens_padded, "position_offsets", position_offsets)
    rows, rot = _tables(rope_cos, rope_sin, dev, d)
    if dq is None:
        dq = torch.empty((T, hq, d), dtype=dtype, device=dev)
    dqs = _rows(dq, "dq", dev, dtype, grad_q.shape)
    dks = 0
    if grad_k is not None:
        if dk is None:
            dk = torch.empty((T, hkv, d), dtype=dtype, device=dev)
        dks = _rows(dk, "dk", dev, dtype, grad_k.shape)
    grads = []
    for name, w, g in (("dq_weight", q_weight, dq_weight), ("dk_weight", k_weight, dk_weight)):
        if w is None and g is not None:
            raise ValueError(f"{name} needs its weight")
        if w is not None and g is None:
            g = torch.empty(d, dtype=torch.float32, device=dev)
        _whole(g, name, dev, torch.float32, (d,))
        grads.append(g)
    size = 0
    if q_weight is not None or k_weight is not None:
        if workspace is None:
            workspace = torch.empty(_workspace_size("thd_qk_norm_rope_bwd_workspace_size", d), dtype=torch.uint8,
                                    device=dev)
        else:
            _whole(workspace, "workspace", dev, torch.uint8)
        size = workspace.numel()
    if (T | hq | hkv | d | rows | B) > _COUNT_MAX:
        raise _too_large("thd_qk_norm_rope_bwd")
    _call("thd_qk_norm_rope_bwd", dev, grad_q.data_ptr(), _addr(grad_k), _addr(q), qs, _addr(k), ks, _addr(q_weight),
          _addr(k_weight), fp32, float(eps), _addr(rope_cos), _addr(rope_sin), rows, rot, int(bool(interleaved)),
          cu_seqlens.data_ptr(), _addr(cu_seqlens_padded), _addr(position_offsets), B, dq.data_ptr(), dqs, _addr(dk), dks,
          _addr(grads[0]), _addr(grads[1]), T, hq, hkv, d, code, _addr(workspace), size)
    return dq, dk, grads[0], grads[1]


def _caches(k_cache, v_cache, device, dtype, page_table, batch_size, writes):
    """Strides of the two caches (ctypes int64[6]: page, token, head of each), and the table's."""
    if (type(k_cache) is torch.Tensor is type(v_cache) and k_cache.is_contiguous() and v_cache.is_contiguous()
            and k_cache.dtype is dtype is v_cache.dtype and type(page_table) is torch.Tensor
            and page_table.is_contiguous() and page_table.dtype is torch.int32
            and k_cache.get_device() == device.index == v_cache.get_device() == page_table.get_device()):
        # the usual case in few steps
        shape, table = k_cache.shape, page_table.shape
        if len(shape) == 4 and shape == v_cache.shape and len(table) == 2 and table[0] >= batch_size:
            _, size, heads, d = shape
            page = size * heads * d
            return shape, _Places(page, heads * d, d, page, heads * d, d), table[1], table[1]
    shape = k_cache.shape if isinstance(k_cache, torch.Tensor) else None
    places = []
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        if type(c) is not torch.Tensor or c.get_device() != device.index:
            _on(c, name, device)
        if c.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}")
        if c.dim() != 4 or c.shape != shape:
            raise ValueError("k_cache and v_cache must both be [pages, page_size, Hkv, head_dim]")
        pages, size, heads, d = shape
        page, token, head, one = c.stride()
        if d > 1 and one != 1:
            raise ValueError(f"{name}: the values of a head must be contiguous")
        if writes and not c.is_contiguous():
            need = d
            for step, n in sorted((s, n) for s, n in ((page, pages), (token, size), (head, heads)) if n > 1):
                if step < need:
                    raise ValueError(f"{name}: places overlap")
                need = step * n
        places += (page if pages > 1 else 0, token if size > 1 else 0, head if heads > 1 else 0)
    if type(page_table) is not torch.Tensor or page_table.get_device() != device.index:
        _on(page_table, "page_table", device)
    if page_table.dtype is not torch.int32:
        raise TypeError("page_table must be int32")
    if page_table.dim() != 2 or page_table.shape[0] < batch_size:
        raise ValueError("page_table must be [>= batch_size, pages]")
    wide = page_table.shape[1]
    if wide > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table: the entries of a sequence must be contiguous")
    step = page_table.stride(0) if page_table.shape[0] > 1 else wide
    if step < wide:
        raise ValueError("page_table: rows overlap")
    return shape, _Places(*places), wide, step


def thd_kv_append(k, v, k_cache, v_cache, page_table, cache_lens, cu_seqlens, cu_seqlens_padded=None,
                  batch_size=None, q=None, rope_cos=None, rope_sin=None, positions=None, q_weight=None, k_weight=None,
                  eps=1e-6, interleaved=False, q_out=None):
    """New keys and values of a packed batch into a paged cache; keys (and q, where given) are
    normed and rotated on the way as by thd_qk_norm_rope.  Returns q_out, or None without q.

    k, v: [T, Hkv, d], q: [T, Hq, d] (rows may lie apart).  k_cache / v_cache: [pages, page_size,
    Hkv, d], in any order of pages, tokens and heads in memory.  page_table: int32 [B, pages of a
    sequence].  cache_lens: int32 [B], keys already cached; row i of sequence b goes to slot
    cache_lens[b] + i, and is not written if the table names no page of the cache for it.
    positions: int32 [T], the rows' rotary positions, or None: their slots.  cache_lens is
    not changed.
    """
    code = _dtype_code(k, "k")
    dev, dtype = k.device, k.dtype
    ks = _rows(k, "k", dev, dtype)
    vs = _rows(v, "v", dev, dtype, k.shape)
    T, hkv, d = k.shape
    hq, qs = 0, 0
    if q is not None:
        qs = _rows(q, "q", dev, dtype)
        hq = q.shape[1]
        if q.shape[0] != T or q.shape[2] != d:
            raise ValueError("q must be [T, Hq, head_dim] with k's T and head_dim")
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out and q_weight need q")
    if cache_lens is None:
        raise TypeError("cache_lens must be an int32 tensor")
    B = _meta(dev, batch_size, cu_seqlens, cu_seqlens_padded, "cache_lens", cache_lens)
    rows, rot = _tables(rope_cos, rope_sin, dev, d)
    fp32 = _weights(q_weight, k_weight, dev, d, dtype)
    if positions is not None:
        _whole(positions, "positions", dev, torch.int32, (T,))
    shape, strides, wide, step = _caches(k_cache, v_cache, dev, dtype, page_table, B, True)
    if shape[2] != hkv or shape[3] != d:
        raise ValueError("the caches must have k's heads and head_dim")
    if shape[1] < 1:
        raise ValueError("a page must hold a token")
    if q is not None:
        if q_out is None:
            q_out = torch.empty((T, hq, d), dtype=dtype, device=dev)
        else:
            _whole(q_out, "q_out", dev, dtype, q.shape)
    if (T | hq | hkv | d | rows | B | shape[0] | shape[1] | wide) > _COUNT_MAX:
        raise _too_large("thd_kv_append")
    _call("thd_kv_append", dev, _addr(q), qs, _addr(k), ks, v.data_ptr(), vs, _addr(q_weight), _addr(k_weight), fp32,
          float(eps), _addr(rope_cos), _addr(rope_sin), rows, rot, int(bool(interleaved)), _addr(positions),
          cu_seqlens.data_ptr(), _addr(cu_seqlens_padded), cache_lens.data_ptr(), B, _addr(q_out), k_cache.data_ptr(),
          v_cache.data_ptr(), strides, shape[0], shape[1], page_table.data_ptr(), step, wide, T, hq, hkv, d, code)
    return q_out


def thd_attn_paged(q, k_cache, v_cache, page_table, kv_lens, cu_seqlens_q, cu_seqlens_q_padded=None, batch_size=None,
                   max_seqlen_q=0, tree_mask=None, softmax_scale=None, out=None, lse=None, return_lse=True,
                   workspace=None):
    """Attention of packed new tokens over a paged cache: decoding steps, chunks, drafted trees.

    q: [T, Hq, d] (bf16 or fp16, contiguous).  k_cache / v_cache / page_table: as in thd_kv_append,
    the new tokens' own keys already in them.  kv_lens: int32 [B], keys of each sequence with the
    new ones.  New token i of n sees key j iff j <= kv_len - n + i; with tree_mask (int64
    [T, words]) iff j < kv_len - n or bit j - (kv_len - n) of its mask is set.  max_seqlen_q: a
    hint, the most new tokens of a sequence (0: unknown).  Returns (out [T, Hq, d], lse [Hq, T]
    float32 or None); rows of no sequence and rows that see no key are 0 with lse -inf.
    """
    code = _dtype_code(q, "q")
    dev, dtype = q.device, q.dtype
    _whole(q, "q", dev, dtype)
    if q.dim() != 3:
        raise ValueError("q must be [T, heads, head_dim]")
    T, hq, d = q.shape
    if kv_lens is None:
        raise TypeError("kv_lens must be an int32 tensor")
    B = _meta(dev, batch_size, cu_seqlens_q, cu_seqlens_q_padded, "kv_lens", kv_lens)
    shape, strides, wide, step = _caches(k_cache, v_cache, dev, dtype, page_table, B, False)
    if shape[3] != d:
        raise ValueError("the caches must have q's head_dim")
    if shape[1] < 1:
        raise ValueError("a page must hold a token")
    words = 0
    if tree_mask is not None:
        _whole(tree_mask, "tree_mask", dev, torch.int64)
        if tree_mask.dim() != 2 or tree_mask.shape[0] != T or tree_mask.shape[1] < 1:
            raise ValueError("tree_mask must be [T, words]")
        words = tree_mask.shape[1]
    if out is None:
        out = torch.empty((T, hq, d), dtype=dtype, device=dev)
    else:
        _whole(out, "out", dev, dtype, q.shape)
    if lse is None and return_lse:
        lse = torch.empty((hq, T), dtype=torch.float32, device=dev)
    else:
        _whole(lse, "lse", dev, torch.float32, (hq, T))
    if workspace is None:
        workspace = torch.empty(_workspace_size("thd_attn_paged_workspace_size", d), dtype=torch.uint8, device=dev)
    else:
        _whole(workspace, "workspace", dev, torch.uint8)
    max_seqlen_q = int(max_seqlen_q)
    if (T | hq | shape[2] | d | B | shape[0] | shape[1] | wide | words | abs(max_seqlen_q)) > _COUNT_MAX:
        raise _too_large("thd_attn_paged")
    _call("thd_attn_paged", dev, _addr(q), k_cache.data_ptr(), v_cache.data_ptr(), strides, shape[0], shape[1],
          page_table.data_ptr(), step, wide, kv_lens.data_ptr(), cu_seqlens_q.data_ptr(), _addr(cu_seqlens_q_padded), B,
          max_seqlen_q, _addr(tree_mask), words, 1.0 / math.sqrt(d) if softmax_scale is None else
          float(softmax_scale), out.data_ptr(), _addr(lse), T, hq, shape[2], d, code, _addr(workspace), workspace.numel())
    return out, lse
