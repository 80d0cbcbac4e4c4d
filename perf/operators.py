"""Measured workloads of the operators around packed attention.

Four operators, each with its cases, its plain form in torch operations and its
definition in 64 bits:

* ``rope``      norm of every query and key head and the position rotation, packed rows
* ``rope_bwd``  its gradients, those of the norm weights among them
* ``append``    new keys and values (normed, rotated) into a paged cache, queries rotated
* ``paged``     attention of packed new tokens over a paged cache: one token, several, or a tree

``own`` picks the side: False computes the plain form, True calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------------------ cases
def _rope(name, op, seqs, tokens, hq, hkv, d, dtype="bf16", norm=True, rotary=None, interleaved=False, gap=0,
          fused=False, base=10000.0):
    return {"name": name, "op": op, "seqs": seqs, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype,
            "norm": norm, "rotary": d if rotary is None else rotary, "interleaved": interleaved, "gap": gap,
            "fused": fused, "base": base}


def _append(name, seqs, tokens, cached, page, hq, hkv, d, dtype="bf16", norm=False, rotary=None, interleaved=False,
            gap=0, fused=False, tree=False, heads_first=False, base=500000.0):
    return {"name": name, "op": "append", "seqs": seqs, "tokens": tokens, "cached": cached, "page": page, "hq": hq,
            "hkv": hkv, "d": d, "dtype": dtype, "norm": norm, "rotary": d if rotary is None else rotary,
            "interleaved": interleaved, "gap": gap, "fused": fused, "tree": tree, "heads_first": heads_first,
            "base": base}


def _paged(name, seqs, keys, new, page, hq, hkv, d, dtype="bf16", tree=False, ragged=False, gap=0,
           heads_first=False):
    return {"name": name, "op": "paged", "seqs": seqs, "keys": keys, "new": new, "page": page, "hq": hq, "hkv": hkv,
            "d": d, "dtype": dtype, "tree": tree, "ragged": ragged, "gap": gap, "heads_first": heads_first}


def listed():
    return [
        # the step of a small decoding batch: one row for each of 16 sequences, latency alone
        _rope("rope 16 rows", "rope", 16, 16, 32, 8, 128),
        # a packed training batch with grouped heads and gaps, read out of the fused projection
        _rope("rope packed gqa", "rope", 64, 65536, 32, 8, 128, gap=31, fused=True),
        # the long-context batch, rotation alone (models without the norm)
        _rope("rope long context", "rope", 8, 131072, 16, 16, 128, norm=False, base=500000.0),
        # gradients of a short odd-sized batch: 9 sequences, 1001 rows
        _rope("rope_bwd 1001 rows", "rope_bwd", 9, 1001, 16, 2, 128, gap=5),
        # gradients of the packed training batch
        _rope("rope_bwd packed gqa", "rope_bwd", 64, 65536, 32, 8, 128, gap=31, fused=True),
        # gradients of many short sequences in fp16, half of each head rotated, pairs side by side
        _rope("rope_bwd many short", "rope_bwd", 4096, 200000, 32, 32, 64, dtype="fp16", rotary=32,
              interleaved=True, gap=15),
        # one new token for each of 64 sequences
        _append("append decode", 64, 64, 1000, 16, 32, 8, 128),
        # a chunk of prompt tokens for a few sequences, queries and keys normed, out of the fused projection
        _append("append prefill", 7, 16384, 5000, 64, 32, 8, 128, norm=True, fused=True, gap=9),
        # one sequence, one token, a short cache: latency alone
        _paged("paged one short", 1, 777, 1, 16, 32, 8, 128),
        # a decoding batch of uneven lengths
        _paged("paged decode batch", 64, 500000, 1, 16, 32, 8, 128),
        # one long sequence without grouped heads, fp16
        _paged("paged one long fp16", 1, 262144, 1, 64, 16, 16, 64, dtype="fp16"),
        # trees of 27 drafted tokens
        _paged("paged tree", 16, 120000, 27, 32, 32, 8, 128, tree=True),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "paged", "paged"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    d = rng.choice([32, 64, 80, 96, 128, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    group = rng.choice([1, 2, 4, 4, 5, 8])
    hq = hkv * group
    rotary = rng.choice([0, 16, 32, d, d, d]) if d > 32 else rng.choice([16, d])
    inter = rng.random() < 0.3
    gap = rng.choice([0, 0, 3, 17])
    fused = rng.random() < 0.5
    if op in ("rope", "rope_bwd"):
        rows = _spread(rng, 1, min(200000, 2.0e8 / ((hq + hkv) * d)))
        return _strip(_rope("", op, min(rows, _spread(rng, 1, 3000)), rows, hq, hkv, d, dtype,
                            rng.random() < 0.7 or rotary == 0, rotary, inter, gap, fused,
                            rng.choice([10000.0, 500000.0])))
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 256])
    order = rng.random() < 0.3
    if op == "append":
        seqs = _spread(rng, 1, 300)
        tokens = max(seqs, _spread(rng, 1, 16000))
        return _strip(_append("", seqs, tokens, _spread(rng, 1, 2000), page, hq, hkv, d, dtype, rng.random() < 0.4,
                              rotary, inter, gap, fused, rng.random() < 0.3, order))
    seqs = _spread(rng, 1, 130)
    new = rng.choice([1, 1, 1, _spread(rng, 2, 64)])
    most = 120000 if new > 1 else min(260000, 500000 * 8 * 128 / (hkv * d) / 2)
    keys = max(seqs * new, min(seqs * 16000, _spread(rng, 64, most)))
    # the plain form holds [sequences, heads, new, keys] scores: keep within the listed cases' work
    if new > 1:
        keys = max(seqs * new, min(keys, int(2.5e8 / (hq * new))))
    return _strip(_paged("", seqs, keys, new, page, hq, hkv, d, dtype, new > 1 and rng.random() < 0.7,
                         new > 1 and rng.random() < 0.4, gap, order))


def _strip(case):
    del case["name"]
    return case


# ------------------------------------------------------------------------------ inputs
def _lengths(rng, seqs, total):
    """`seqs` uneven lengths of at least 1 that sum to `total` (shares within a factor of 4)."""
    share = [math.exp(rng.uniform(0.0, math.log(4.0))) for _ in range(seqs)]
    left, scale = total - seqs, (total - seqs) / sum(share)
    got = [int(s * scale) for s in share]
    for i in range(left - sum(got)):
        got[i % seqs] += 1
    return [1 + g for g in got]


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _packed(rng, state, lens, gap, rows):
    """cu_seqlens, slot starts with gaps of 0..gap rows, and a buffer for `rows` rows and all gaps."""
    cu, starts, at = [0], [], 0
    for n in lens:
        at += rng.randint(0, gap)
        starts.append(at)
        at += n
        cu.append(cu[-1] + n)
    state["cu"] = _int(cu)
    state["padded"] = _int(starts) if gap else None
    state["rows"] = rows + (len(lens) + 1) * gap
    state["seqs"], state["tokens"], state["longest"] = len(lens), cu[-1], max(lens)


def _rand(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _tables(positions, rotary, base):
    """cos and sin of position * base^(-2i/rotary), computed in 64 bits, held in fp32."""
    freq = base ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return angle.cos().float().contiguous(), angle.sin().float().contiguous()


def _qkv(g, s, c, heads, dtype):
    """Row tensors of the given head counts: views of one fused projection, or each its own."""
    if c["fused"]:
        x = _rand(g, (s["rows"], sum(heads) * c["d"]), dtype)
        return [p.unflatten(1, (h, c["d"])) for p, h in zip(x.split([h * c["d"] for h in heads], 1), heads)]
    return [_rand(g, (s["rows"], h, c["d"]), dtype) for h in heads]


def _weights(g, s, c, dtype):
    s["wq"] = s["wk"] = None
    if c["norm"]:
        s["wq"] = (1 + _rand(g, (c["d"],), torch.float32, 0.2)).to(dtype)
        s["wk"] = (1 + _rand(g, (c["d"],), torch.float32, 0.2)).to(dtype)


def _cache(rng, g, s, c, lens, most, dtype):
    """A paged cache that holds `lens` keys of each sequence (`most` at the most in all) at pages in no order; unused
    table entries hold -1."""
    page = c["page"]
    need = [-(-n // page) for n in lens]
    pages = most // page + len(lens) + 3
    order = list(range(pages))
    rng.shuffle(order)
    wide, at, table = max(need) + 1, 0, []
    for n in need:
        table.append(order[at:at + n] + [-1] * (wide - n))
        at += n
    s["table"], s["page"], s["wide"] = _int(table), page, wide
    for name in ("kc", "vc"):
        shape = (pages, c["hkv"], page, c["d"]) if c["heads_first"] else (pages, page, c["hkv"], c["d"])
        x = torch.empty(shape, device="cuda", dtype=dtype)
        x.normal_(generator=g)
        s[name] = x.transpose(1, 2) if c["heads_first"] else x


def _parents(rng, new):
    """The parent of each drafted token of a tree but its root, token 0."""
    return [rng.randint(max(0, i - 9), i - 1) for i in range(1, new)]


def _depths(parents):
    """The depth of each token of the tree."""
    depth = [0]
    for p in parents:
        depth.append(depth[p] + 1)
    return depth


def _sees(parents):
    """The tokens that each token of a tree of up to 64 sees (itself and those above it), as signed 64-bit words."""
    sees = [1]
    for i, p in enumerate(parents, 1):
        sees.append(sees[p] | 1 << i)
    return [x - (1 << 64) if x >> 63 else x for x in sees]


def prepare(case, seed):
    c, rng = case, random.Random(seed)
    g = torch.Generator("cuda").manual_seed(seed)
    dtype = _DTYPES[c["dtype"]]
    s = {"case": c, "dtype": dtype}
    if c["op"] in ("rope", "rope_bwd"):
        _packed(rng, s, _lengths(rng, c["seqs"], c["tokens"]), c["gap"], c["tokens"])
        s["q"], s["k"] = _qkv(g, s, c, [c["hq"], c["hkv"], c["hkv"]] if c["fused"] else [c["hq"], c["hkv"]], dtype)[:2]
        _weights(g, s, c, dtype)
        s["cos"], s["sin"] = _tables(s["longest"], c["rotary"], c["base"]) if c["rotary"] else (None, None)
        if c["op"] == "rope_bwd":
            s["gq"], s["gk"] = _rand(g, s["q"].shape, dtype), _rand(g, s["k"].shape, dtype)
        return s
    if c["op"] == "append":
        lens = _lengths(rng, c["seqs"], c["tokens"])
        _packed(rng, s, lens, c["gap"], c["tokens"])
        s["q"], s["k"], s["v"] = _qkv(g, s, c, [c["hq"], c["hkv"], c["hkv"]], dtype)
        _weights(g, s, c, dtype)
        before = [rng.randint(c["cached"] // 2, c["cached"]) for _ in lens]
        s["before"] = _int(before)
        _cache(rng, g, s, c, [a + b for a, b in zip(before, lens)], c["seqs"] * c["cached"] + c["tokens"], dtype)
        s["cos"], s["sin"] = _tables(c["cached"] + max(lens), c["rotary"], c["base"]) if c["rotary"] else (None, None)
        s["positions"] = None
        if c["tree"]:
            at, pos = s["padded"].tolist() if c["gap"] else s["cu"].tolist(), [0] * s["rows"]
            for b, n in enumerate(lens):
                pos[at[b]:at[b] + n] = [before[b] + x for x in _depths(_parents(rng, n))]
            s["positions"] = _int(pos)
        return s
    new = [rng.randint(1, c["new"]) if c["ragged"] else c["new"] for _ in range(c["seqs"])]
    _packed(rng, s, new, c["gap"], c["seqs"] * c["new"])
    keys = [max(a, b) for a, b in zip(_lengths(rng, c["seqs"], c["keys"]), new)]
    s["keys"], s["most"] = _int(keys), max(keys)
    _cache(rng, g, s, c, keys, c["keys"] + c["seqs"] * c["new"], dtype)
    s["q"] = _rand(g, (s["rows"], c["hq"], c["d"]), dtype)
    s["tree"] = None
    if c["tree"]:
        at, words = s["padded"].tolist() if c["gap"] else s["cu"].tolist(), [0] * s["rows"]
        for b, n in enumerate(new):
            words[at[b]:at[b] + n] = _sees(_parents(rng, n))
        s["tree"] = torch.tensor(words, dtype=torch.int64, device="cuda")[:, None]
    s["scale"] = 1.0 / math.sqrt(c["d"])
    return s


# ------------------------------------------------------------------------------ plain forms
def _places(s):
    """Sequence, position in it and buffer row of each valid token."""
    cu = s["cu"].long()
    seq = torch.repeat_interleave(torch.arange(s["seqs"], device="cuda"), cu[1:] - cu[:-1], output_size=s["tokens"])
    pos = torch.arange(s["tokens"], device="cuda") - cu[seq]
    start = cu if s["padded"] is None else s["padded"].long()
    return seq, pos, start[seq] + pos


def _norm(x, w):
    """(normed x, x / rms) in 32 bits."""
    if w is None:
        return x, x
    unit = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return unit * w.float(), unit


def _turn(x, cos, sin, interleaved, back=False):
    """The rotation of the first 2 * cos.shape[1] values of each head by the rows' angles."""
    if cos is None:
        return x
    half = cos.shape[1]
    c, n = cos[:, None, :], -sin[:, None, :] if back else sin[:, None, :]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * n, b * c + a * n
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * n, b * c + a * n
    return y


def _angles(s, pos):
    return (None, None) if s["cos"] is None else (s["cos"][pos], s["sin"][pos])


def _run_rope(s):
    c = s["case"]
    _, pos, rows = _places(s)
    cos, sin = _angles(s, pos)
    outs = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = torch.zeros(x.shape, dtype=x.dtype, device="cuda")
        y[rows] = _turn(_norm(x[rows].float(), w)[0], cos, sin, c["interleaved"]).to(x.dtype)
        outs.append(y)
    return outs


def _run_rope_bwd(s):
    c = s["case"]
    _, pos, rows = _places(s)
    cos, sin = _angles(s, pos)
    grads, weights = [], []
    for g, x, w in ((s["gq"], s["q"], s["wq"]), (s["gk"], s["k"], s["wk"])):
        h = _turn(g[rows].float(), cos, sin, c["interleaved"], back=True)
        if w is not None:
            v = x[rows].float()
            r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
            unit = v * r
            weights.append((h * unit).sum((0, 1), dtype=torch.float64).float())
            h = h * w.float()
            h = r * (h - unit * (h * unit).mean(-1, keepdim=True))
        dx = torch.zeros(x.shape, dtype=x.dtype, device="cuda")
        dx[rows] = h.to(x.dtype)
        grads.append(dx)
    return grads + weights


def _run_append(s):
    c = s["case"]
    seq, pos, rows = _places(s)
    slot = s["before"].long()[seq] + pos
    cos, sin = _angles(s, slot if s["positions"] is None else s["positions"].long()[rows])
    q = torch.zeros(s["q"].shape, dtype=s["dtype"], device="cuda")
    q[rows] = _turn(_norm(s["q"][rows].float(), s["wq"])[0], cos, sin, c["interleaved"]).to(s["dtype"])
    page, at = s["table"].long()[seq, slot // s["page"]], slot % s["page"]
    s["kc"][page, at] = _turn(_norm(s["k"][rows].float(), s["wk"])[0], cos, sin, c["interleaved"]).to(s["dtype"])
    s["vc"][page, at] = s["v"][rows]
    return [q, s["kc"], s["vc"]]


def _run_paged(s):
    c = s["case"]
    hkv, group, d, most, longest = c["hkv"], c["hq"] // c["hkv"], c["d"], s["most"], s["longest"]
    cu, keys = s["cu"].long(), s["keys"].long()
    new = cu[1:] - cu[:-1]
    at = torch.arange(most, device="cuda")
    page = s["table"].long()[:, at // s["page"]].clamp_min(0)
    k = s["kc"][page, at % s["page"]].permute(0, 2, 3, 1).float()         # [B, Hkv, d, S]
    v = s["vc"][page, at % s["page"]].permute(0, 2, 1, 3).float()         # [B, Hkv, S, d]
    start = cu[:-1] if s["padded"] is None else s["padded"].long()
    i = torch.arange(longest, device="cuda")
    row = (start[:, None] + i).clamp_max(s["rows"] - 1)                   # [B, L]
    q = s["q"][row].float().unflatten(2, (hkv, group)).permute(0, 2, 1, 3, 4).reshape(-1, hkv, longest * group, d)
    past = (keys - new)[:, None, None]
    j = at[None, None, :] - past                                          # index among the new tokens, < 0: cached
    if s["tree"] is None:
        seen = j <= i[None, :, None]
    else:
        seen = (j < 0) | ((s["tree"][row] >> j.clamp(0, 63)) & 1).bool() & (j < 64)
    seen = seen & (at[None, None, :] < keys[:, None, None])
    x = torch.matmul(q, k) * s["scale"]
    x = x.view(-1, hkv, longest, group, most).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    e = (x - top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(-1, hkv, longest * group, most), v).view(-1, hkv, longest, group, d) / total
    o = torch.where(total > 0, o, 0.0).permute(0, 2, 1, 3, 4).reshape(-1, longest, c["hq"], d)
    lse = (top + total.log())[..., 0].permute(1, 3, 0, 2).reshape(c["hq"], -1, longest)
    seq, pos, rows = _places(s)
    out = torch.zeros(s["q"].shape, dtype=s["dtype"], device="cuda")
    out[rows] = o[seq, pos].to(s["dtype"])
    full = torch.full((c["hq"], s["rows"]), -math.inf, device="cuda")
    full[:, rows] = lse[:, seq, pos]
    return [out, full]


# ------------------------------------------------------------------------------ the library's calls
def _own_rope(s):
    import variable_length_packed_gb300 as thd
    return list(thd.thd_qk_norm_rope(s["q"], s["k"], s["cu"], s["cos"], s["sin"], cu_seqlens_padded=s["padded"],
                                     batch_size=s["seqs"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                                     interleaved=s["case"]["interleaved"]))


def _own_rope_bwd(s):
    import variable_length_packed_gb300 as thd
    dq, dk, dwq, dwk = thd.thd_qk_norm_rope_bwd(
        s["gq"], s["gk"], s["q"], s["k"], s["cu"], s["cos"], s["sin"], cu_seqlens_padded=s["padded"],
        batch_size=s["seqs"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS, interleaved=s["case"]["interleaved"])
    return [dq, dk] if dwq is None else [dq, dk, dwq, dwk]


def _own_append(s):
    import variable_length_packed_gb300 as thd
    q = thd.thd_kv_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["before"], s["cu"],
                          cu_seqlens_padded=s["padded"], batch_size=s["seqs"], q=s["q"], rope_cos=s["cos"],
                          rope_sin=s["sin"], positions=s["positions"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                          interleaved=s["case"]["interleaved"])
    return [q, s["kc"], s["vc"]]


def _own_paged(s):
    import variable_length_packed_gb300 as thd
    return list(thd.thd_attn_paged(s["q"], s["kc"], s["vc"], s["table"], s["keys"], s["cu"],
                                   cu_seqlens_q_padded=s["padded"], batch_size=s["seqs"],
                                   max_seqlen_q=s["longest"], tree_mask=s["tree"], softmax_scale=s["scale"]))


_PLAIN = {"rope": _run_rope, "rope_bwd": _run_rope_bwd, "append": _run_append, "paged": _run_paged}
_OWN = {"rope": _own_rope, "rope_bwd": _own_rope_bwd, "append": _own_append, "paged": _own_paged}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ least work
def work(case):
    c = case
    heads = c["hq"] + c["hkv"]
    if c["op"] in ("rope", "rope_bwd"):
        rows = c["tokens"] * heads
        table = 8 * (c["rotary"] // 2) * min(c["tokens"], 4 * -(-c["tokens"] // c["seqs"]))
        passes = 2 if c["op"] == "rope" else 3
        per = 4 * (3 if c["op"] == "rope" else 8)
        return {"bytes": 2 * passes * rows * c["d"] + table, "flops": per * rows * c["d"] / 4}
    if c["op"] == "append":
        rows = c["tokens"] * (heads + c["hkv"])
        return {"bytes": 4 * rows * c["d"] + 8 * (c["rotary"] // 2) * c["tokens"], "flops": 3 * rows * c["d"]}
    new = c["seqs"] * (c["new"] + 1) // 2 if c["ragged"] else c["seqs"] * c["new"]
    pairs = c["keys"] * new / c["seqs"]
    return {"bytes": 4 * c["keys"] * c["hkv"] * c["d"] + 4 * new * c["hq"] * c["d"] + 4 * new * c["hq"],
            "flops": 4 * pairs * c["hq"] * c["d"]}


# ------------------------------------------------------------------------------ definitions in 64 bits
def _exact_places(s):
    """The same as _places, sequence by sequence on the host."""
    cu = s["cu"].tolist()
    at = s["padded"].tolist() if s["padded"] is not None else cu
    return [(b, at[b], cu[b + 1] - cu[b]) for b in range(s["seqs"])]


def _exact_rows(s):
    """Row of each valid token and its position, from the host's lists."""
    rows, pos = [], []
    for _, start, n in _exact_places(s):
        rows += range(start, start + n)
        pos += range(n)
    return torch.tensor(rows, device="cuda"), torch.tensor(pos, device="cuda")


def _exact_matrix(s, c, pos):
    """Each row's cos and sin spread over the head's d places, and each place's partner and its sign."""
    d, rot, inter = c["d"], c["rotary"], c["interleaved"]
    place = torch.arange(d, device="cuda")
    if inter:
        index, partner, first = place // 2, place ^ 1, place % 2 == 0
    else:
        index, partner, first = place % max(rot // 2, 1), (place + rot // 2) % max(rot, 1), place < rot // 2
    turned = place < rot
    partner = torch.where(turned, partner, place)
    index = torch.where(turned, index, 0)
    if rot:
        cos = torch.where(turned, s["cos"].double()[pos][:, index], 1.0)
        sin = torch.where(turned, s["sin"].double()[pos][:, index], 0.0) * torch.where(first, -1.0, 1.0)
    else:
        cos = torch.ones((len(pos), d), dtype=torch.float64, device="cuda")
        sin = torch.zeros_like(cos)
    return cos[:, None, :], sin[:, None, :], partner


def _exact_forward(x, w, turn):
    cos, sin, partner = turn
    n = x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    return n * cos + n[..., partner] * sin


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] in ("rope", "rope_bwd"):
        rows, pos = _exact_rows(s)
        turn = _exact_matrix(s, c, pos)
        outs, weights = [], []
        for x, w, g in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
            v = x[rows].double()
            y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
            if g is None:
                y[rows] = _exact_forward(v, w, turn)
            else:
                # of y_i = n_i cos_i + n_p(i) sin_i: dn_i = g_i cos_i + g_p(i) sin_p(i)
                cos, sin, partner = turn
                h = g[rows].double()
                h = h * cos + (h * sin)[..., partner]
                if w is not None:
                    ms = v.pow(2).sum(-1, keepdim=True) / c["d"] + EPS
                    weights.append((h * v / ms.sqrt()).sum((0, 1)))
                    h = h * w.double()
                    h = h / ms.sqrt() - v * (h * v).sum(-1, keepdim=True) / (c["d"] * ms * ms.sqrt())
                y[rows] = h
            outs.append(y)
        return outs + weights
    if c["op"] == "append":
        rows, pos = _exact_rows(s)
        before, table = s["before"].tolist(), s["table"].tolist()
        slots = [(b, before[b] + i) for b, _, n in _exact_places(s) for i in range(n)]
        where = torch.tensor([[table[b][i // s["page"]], i % s["page"]] for b, i in slots], device="cuda")
        angle = torch.tensor([i for _, i in slots], device="cuda") if s["positions"] is None else s["positions"].long()[rows]
        turn = _exact_matrix(s, c, angle)
        q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        q[rows] = _exact_forward(s["q"][rows].double(), s["wq"], turn)
        kc, vc = s["kc"].double(), s["vc"].double()
        kc[where[:, 0], where[:, 1]] = _exact_forward(s["k"][rows].double(), s["wk"], turn)
        vc[where[:, 0], where[:, 1]] = s["v"][rows].double()
        return [q, kc, vc]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((c["hq"], s["rows"]), -math.inf, dtype=torch.float64, device="cuda")
    keys, group = s["keys"].tolist(), c["hq"] // c["hkv"]
    bit = torch.arange(64, device="cuda")
    for b, start, n in _exact_places(s):
        pages = s["table"][b, :-(-keys[b] // s["page"])].long()
        seen = torch.ones((n, keys[b]), dtype=torch.bool, device="cuda")
        if s["tree"] is None:
            seen[:, keys[b] - n:] = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
        else:
            seen[:, keys[b] - n:] = ((s["tree"][start:start + n] >> bit) & 1).bool()[:, :n]
        for h in range(c["hkv"]):
            k = s["kc"][pages, :, h].reshape(-1, c["d"])[:keys[b]].double()
            v = s["vc"][pages, :, h].reshape(-1, c["d"])[:keys[b]].double()
            for x in range(h * group, (h + 1) * group):
                z = (s["q"][start:start + n, x].double() @ k.T * s["scale"]).masked_fill(~seen, -math.inf)
                lse[x, start:start + n] = z.logsumexp(-1)
                out[start:start + n, x] = z.softmax(-1) @ v
    return [out, lse]
