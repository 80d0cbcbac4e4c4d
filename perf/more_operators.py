"""Measured workloads of the operators that bound what a long sequence costs.

Five operators, each with its cases, its plain form in torch operations and its definition in
64 bits:

* ``fwd``      packed attention with a sliding window and first tokens that stay visible (sinks)
* ``bwd``      its gradients
* ``paged``    the same window and sinks over a paged cache: single tokens and chunks
* ``weights``  attention over a paged cache that adds up the weight each cached key got
* ``evict``    the keys of a paged cache with the most weight kept, the others dropped

``own`` picks the side: False computes the plain form, True calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------ cases
def _packed(name, op, seqs, tokens, hq, hkv, d, left, right, sinks, policy="causal", dtype="bf16", gap=0):
    return {"name": name, "op": op, "seqs": seqs, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "left": left,
            "right": right, "sinks": sinks, "policy": policy, "dtype": dtype, "gap": gap}


def _paged(name, op, seqs, keys, new, page, hq, hkv, d, left=-1, sinks=0, dtype="bf16", ragged=False, gap=0,
           heads_first=False):
    return {"name": name, "op": op, "seqs": seqs, "keys": keys, "new": new, "page": page, "hq": hq, "hkv": hkv, "d": d,
            "left": left, "sinks": sinks, "dtype": dtype, "ragged": ragged, "gap": gap, "heads_first": heads_first}


def _evict(name, seqs, keys, keep, page, hkv, d, sinks, recent, dtype="bf16", in_place=False, heads_first=False):
    return {"name": name, "op": "evict", "seqs": seqs, "keys": keys, "keep": keep, "page": page, "hkv": hkv, "d": d,
            "sinks": sinks, "recent": recent, "dtype": dtype, "in_place": in_place, "heads_first": heads_first}


def listed():
    return [
        # a handful of short prompts: latency alone
        _packed("sinks fwd 16 short", "fwd", 16, 2000, 32, 8, 128, 64, 0, 4),
        # a packed training batch with grouped heads, gaps and mask types of each sequence's own
        _packed("sinks fwd packed gqa", "fwd", 64, 65536, 32, 8, 128, 511, 511, 4, policy="mixed", gap=31),
        # the long-context batch with the window that the benchmark times, and sinks
        _packed("sinks fwd long context", "fwd", 8, 131072, 16, 16, 128, 2048, 0, 64),
        # gradients of a short odd-sized batch: 9 sequences, 1001 rows
        _packed("sinks bwd 1001 rows", "bwd", 9, 1001, 16, 2, 128, 100, 30, 3, policy="mixed", gap=5),
        # gradients of the packed training batch
        _packed("sinks bwd packed gqa", "bwd", 64, 65536, 32, 8, 128, 511, 511, 4, policy="mixed", gap=31),
        # gradients of one long sequence in fp16: its sinks are seen by every row behind them
        _packed("sinks bwd one long", "bwd", 1, 65536, 16, 4, 64, 1023, 0, 16, dtype="fp16"),
        # one new token for each sequence of a decoding batch, each looking back over 2048 keys
        _paged("window decode batch", "paged", 64, 500000, 1, 16, 32, 8, 128, left=2047, sinks=4),
        # chunks of a prompt over what is cached of it
        _paged("window chunk", "paged", 8, 100000, 512, 32, 32, 8, 128, left=1023, sinks=16),
        # a decoding batch whose keys' weights are added up
        _paged("weights decode batch", "weights", 64, 500000, 1, 16, 32, 8, 128),
        # the last chunk of a few prompts, after which keys are dropped by their weight
        _paged("weights chunk", "weights", 4, 60000, 1024, 32, 32, 8, 128),
        # one short sequence cut to half: latency alone
        _evict("evict one short", 1, 1000, 500, 16, 8, 128, 4, 64),
        # a decoding batch of uneven lengths cut to a common bound, into other pages
        _evict("evict batch", 32, 500000, 8000, 16, 8, 128, 4, 256),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "paged", "weights", "evict"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    group = rng.choice([1, 2, 4, 4, 5, 8])
    hq = hkv * group
    gap = rng.choice([0, 0, 3, 17])
    if op in ("fwd", "bwd"):
        d = rng.choice([40, 64, 96, 128, 128]) if op == "fwd" else rng.choice([64, 128, 128])
        left, sinks = _spread(rng, 1, 4000) - 1, _spread(rng, 1, 200)
        policy = rng.choice(["causal", "causal", "mixed", "full"])
        right = 0 if policy == "causal" else _spread(rng, 1, 1000) - 1
        # the plain form holds [tokens, heads, keys of a block] scores: keep within the listed cases' work
        most = (5.0e9 if op == "fwd" else 2.5e9) / (hq * (left + right + sinks + 256))
        # a row that sees itself alone has no gradients but of its value: sequences of some rows there
        tokens, rows = (_spread(rng, 1, min(120000, most)), 1) if op == "fwd" else (_spread(rng, 8, min(120000, most)), 8)
        return _strip(_packed("", op, min(tokens // rows, _spread(rng, 1, 300)), tokens, hq, hkv, d, left, right, sinks,
                              policy, dtype, gap))
    d = rng.choice([32, 64, 80, 96, 128, 128, 128])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 256])
    order = rng.random() < 0.3
    seqs = _spread(rng, 1, 130)
    if op == "evict":
        keys = max(seqs, min(seqs * 16000, _spread(rng, 64, min(260000, 500000 * 8 * 128 / (hkv * d) / 2))))
        return _strip(_evict("", seqs, keys, _spread(rng, 1, 2 * keys // seqs + 1), page, hkv, d, rng.choice([0, 1, 4, 70]),
                             rng.choice([0, 16, 200]), dtype, rng.random() < 0.4, order))
    new = rng.choice([1, 1, 1, _spread(rng, 2, 300)])
    most = 120000 if new > 1 else min(260000, 500000 * 8 * 128 / (hkv * d) / 2)
    keys = max(seqs * new, min(seqs * 16000, _spread(rng, 64, most)))
    if new > 1:
        keys = max(seqs * new, min(keys, int(2.5e8 / (hq * new))))
    left, sinks = -1, 0
    if op == "paged" or rng.random() < 0.3:
        left, sinks = _spread(rng, 1, 6000) - 1, rng.choice([0, 1, 4, 70])
    return _strip(_paged("", op, seqs, keys, new, page, hq, hkv, d, left, sinks, dtype, new > 1 and rng.random() < 0.4,
                         gap, order))


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


def _rows(rng, state, lens, gap, rows):
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


def _pages(rng, g, s, c, lens, most, dtype, other=None):
    """A paged cache that holds `lens` keys of each sequence (`most` at the most in all, `other` included) at pages in no
    order; unused table entries hold -1.  other: keys of each sequence that a second table of pages has room for."""
    page = c["page"]
    need = [-(-n // page) for n in lens]
    more = [-(-n // page) for n in other or []]
    pages = most // page + len(lens) * (2 if other else 1) + 3
    order = list(range(pages))
    rng.shuffle(order)
    at, tables = 0, []
    for want in (need, more):
        table, wide = [], max(want or [0]) + 1
        for n in want:
            table.append(order[at:at + n] + [-1] * (wide - n))
            at += n
        tables.append(table)
    s["table"], s["new_table"] = _int(tables[0]), _int(tables[1]) if other else None
    for name in ("kc", "vc"):
        shape = (pages, c["hkv"], page, c["d"]) if c["heads_first"] else (pages, page, c["hkv"], c["d"])
        x = torch.empty(shape, device="cuda", dtype=dtype)
        x.normal_(generator=g)
        s[name] = x.transpose(1, 2) if c["heads_first"] else x
    # weights lie head by head within a page; many keys never got any
    w = torch.randn((pages, c["hkv"], page), generator=g, device="cuda").mul_(2.0).exp_()
    s["weights"] = w.masked_fill_(torch.rand(w.shape, generator=g, device="cuda") < 0.1, 0.0).transpose(1, 2)


def prepare(case, seed):
    c, rng = case, random.Random(seed)
    g = torch.Generator("cuda").manual_seed(seed)
    dtype = _DTYPES[c["dtype"]]
    s = {"case": c, "dtype": dtype, "scale": 1.0 / math.sqrt(c["d"])}
    if c["op"] in ("fwd", "bwd"):
        _rows(rng, s, _lengths(rng, c["seqs"], c["tokens"]), c["gap"], c["tokens"])
        for name, h in (("q", c["hq"]), ("k", c["hkv"]), ("v", c["hkv"])):
            s[name] = _rand(g, (s["rows"], h, c["d"]), dtype)
        kind = {"causal": [1], "full": [0], "mixed": [0, 1, 2]}[c["policy"]]
        s["causal"] = torch.tensor([rng.choice(kind) for _ in range(c["seqs"])], dtype=torch.uint8, device="cuda")
        if c["op"] == "bwd":   # the forward's results, as the training step has them in hand
            s["out"], s["lse"] = _plain_fwd(s)
            s["dout"] = _rand(g, s["q"].shape, dtype)
        return s
    if c["op"] == "evict":
        lens = _lengths(rng, c["seqs"], c["keys"])
        keep = [rng.randint(c["keep"] // 2, c["keep"]) if c["seqs"] > 1 else c["keep"] for _ in lens]
        _pages(rng, g, s, c, lens, c["keys"] + c["seqs"] * c["keep"], dtype, None if c["in_place"] else [min(a, b) for a, b in zip(keep, lens)])
        s["keys"], s["keep"], s["most"] = _int(lens), _int(keep), max(lens)
        s["seqs"] = c["seqs"]
        return s
    new = [rng.randint(1, c["new"]) if c["ragged"] else c["new"] for _ in range(c["seqs"])]
    _rows(rng, s, new, c["gap"], c["seqs"] * c["new"])
    keys = [max(a, b) for a, b in zip(_lengths(rng, c["seqs"], c["keys"]), new)]
    s["keys"], s["most"] = _int(keys), max(keys)
    _pages(rng, g, s, c, keys, c["keys"] + c["seqs"] * c["new"], dtype)
    s["q"] = _rand(g, (s["rows"], c["hq"], c["d"]), dtype)
    return s


# ------------------------------------------------------------------------------ plain forms
def _places(s):
    """Sequence, position in it and buffer row of each valid token."""
    cu = s["cu"].long()
    seq = torch.repeat_interleave(torch.arange(s["seqs"], device="cuda"), cu[1:] - cu[:-1], output_size=s["tokens"])
    pos = torch.arange(s["tokens"], device="cuda") - cu[seq]
    start = cu if s["padded"] is None else s["padded"].long()
    return seq, pos, start[seq] + pos


_BLOCK = 256


def _blocks(s):
    """The batch in blocks of 256 rows of one sequence, each with the keys that its window may reach and the
    sinks: buffer rows of the queries [N, R] and keys [N, K], what each query sees [N, R, K], which
    queries exist [N, R]."""
    c = s["case"]
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    start = cu[:-1] if s["padded"] is None else s["padded"].long()
    per = (lens + _BLOCK - 1) // _BLOCK
    seq = torch.repeat_interleave(torch.arange(s["seqs"], device="cuda"), per)
    q0 = (torch.arange(len(seq), device="cuda") - (per.cumsum(0) - per)[seq]) * _BLOCK
    n, code = lens[seq][:, None], s["causal"][seq][:, None, None]
    i = q0[:, None] + torch.arange(_BLOCK, device="cuda")
    near = q0[:, None] - c["left"] + torch.arange(c["left"] + _BLOCK + c["right"], device="cuda")
    first = torch.arange(c["sinks"], device="cuda").expand(len(seq), -1)
    ii = i[:, :, None]
    in_window = lambda j: (j >= ii - c["left"]) & (j <= ii + c["right"])  # noqa: E731
    allowed = lambda j: (j >= 0) & (j < n[:, :, None]) & ((code == 0) | (j <= ii))  # noqa: E731
    sees = torch.cat([allowed(near[:, None, :]) & in_window(near[:, None, :]),
                      allowed(first[:, None, :]) & ~in_window(first[:, None, :])], -1)
    j = torch.cat([near, first], 1)
    j = torch.minimum(j.clamp_min(0), n - 1)
    return start[seq][:, None] + torch.minimum(i, n - 1), start[seq][:, None] + j, sees, i < n


def _heads(x, rows, hkv):
    """Rows [N, R] of x [T, heads, d] in 32 bits: [N, hkv, R * group, d]."""
    y = x[rows].float().unflatten(2, (hkv, -1))                                  # [N, R, hkv, group, d]
    return y.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _back(y, group):
    """[N, hkv, R * group, ...] as [N, R, heads, ...]."""
    y = y.unflatten(2, (-1, group))
    return y.transpose(1, 2).flatten(2, 3)


def _scores(s, rows, keys, sees):
    c = s["case"]
    x = torch.matmul(_heads(s["q"], rows, c["hkv"]), _heads(s["k"], keys, c["hkv"]).transpose(2, 3)).mul_(s["scale"])
    group = c["hq"] // c["hkv"]
    return x.unflatten(2, (-1, group)).masked_fill_(~sees[:, None, :, None, :], -math.inf).flatten(2, 3)


def _plain_fwd(s):
    c = s["case"]
    group = c["hq"] // c["hkv"]
    rows, keys, sees, real = _blocks(s)
    x = _scores(s, rows, keys, sees)
    top = x.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    e = x.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, _heads(s["v"], keys, c["hkv"])) / total
    o = _back(torch.where(total > 0, o, 0.0), group)
    lse = _back(top + total.log(), group)[..., 0]
    out = torch.zeros(s["q"].shape, dtype=s["dtype"], device="cuda")
    out[rows[real]] = o[real].to(s["dtype"])
    full = torch.full((s["rows"], c["hq"]), -math.inf, device="cuda")
    full[rows[real]] = lse[real]
    return [out, full.t().contiguous()]


def _plain_bwd(s):
    c = s["case"]
    hkv, group = c["hkv"], c["hq"] // c["hkv"]
    rows, keys, sees, real = _blocks(s)
    real_rows = real[:, None, :, None].expand(-1, hkv, -1, group).flatten(2)[..., None]
    x = _scores(s, rows, keys, sees)
    lse = _heads(s["lse"].t()[..., None], rows, hkv)
    p = x.sub_(lse.masked_fill(lse == -math.inf, 0.0)).exp_().mul_(real_rows)
    go, o = _heads(s["dout"], rows, hkv), _heads(s["out"], rows, hkv)
    dv = torch.matmul(p.transpose(2, 3), go)
    ds = torch.matmul(go, _heads(s["v"], keys, hkv).transpose(2, 3)).sub_((go * o).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, _heads(s["k"], keys, hkv)).mul_(s["scale"])
    dk = torch.matmul(ds.transpose(2, 3), _heads(s["q"], rows, hkv)).mul_(s["scale"])
    grads = [torch.zeros(s["q"].shape, dtype=s["dtype"], device="cuda")]
    grads[0][rows[real]] = _back(dq, group)[real].to(s["dtype"])
    for part in (dk, dv):
        total = torch.zeros(s["k"].shape, device="cuda")
        total.index_add_(0, keys.flatten(), part.transpose(1, 2).flatten(0, 1))
        grads.append(total.to(s["dtype"]))
    return grads


def _plain_paged(s):
    c = s["case"]
    hkv, group, d, most, longest = c["hkv"], c["hq"] // c["hkv"], c["d"], s["most"], s["longest"]
    cu, keys = s["cu"].long(), s["keys"].long()
    new = cu[1:] - cu[:-1]
    at = torch.arange(most, device="cuda")
    page, place = s["table"].long()[:, at // c["page"]].clamp_min(0), at % c["page"]
    k = s["kc"][page, place].permute(0, 2, 3, 1).float()                  # [B, Hkv, d, S]
    v = s["vc"][page, place].permute(0, 2, 1, 3).float()                  # [B, Hkv, S, d]
    start = cu[:-1] if s["padded"] is None else s["padded"].long()
    i = torch.arange(longest, device="cuda")
    row = (start[:, None] + i).clamp_max(s["rows"] - 1)                   # [B, L]
    q = s["q"][row].float().unflatten(2, (hkv, group)).permute(0, 2, 1, 3, 4).reshape(-1, hkv, longest * group, d)
    end = ((keys - new)[:, None] + i)[:, :, None]                         # each token's own slot
    seen = (at <= end) & (at < keys[:, None, None]) & (i < new[:, None])[:, :, None]
    if c["left"] >= 0:
        seen = seen & ((at >= end - c["left"]) | (at < c["sinks"]))
    x = torch.matmul(q, k).mul_(s["scale"])
    x = x.view(-1, hkv, longest, group, most).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    e = x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(-1, hkv, longest * group, most), v).view(-1, hkv, longest, group, d) / total
    o = torch.where(total > 0, o, 0.0).permute(0, 2, 1, 3, 4).reshape(-1, longest, c["hq"], d)
    lse = (top + total.log())[..., 0].permute(1, 3, 0, 2).reshape(c["hq"], -1, longest)
    seq, pos, rows = _places(s)
    out = torch.zeros(s["q"].shape, dtype=s["dtype"], device="cuda")
    out[rows] = o[seq, pos].to(s["dtype"])
    full = torch.full((c["hq"], s["rows"]), -math.inf, device="cuda")
    full[:, rows] = lse[:, seq, pos]
    if c["op"] == "paged":
        return [out, full]
    got = e.div_(torch.where(total > 0, total, 1.0)).sum((2, 3)).transpose(1, 2)   # [B, S, Hkv]
    real, fresh = at < keys[:, None], at >= (keys - new)[:, None]
    place = place.expand_as(page)
    had = s["weights"][page, place].masked_fill_(fresh[..., None], 0.0)
    s["weights"][page[real], place[real]] = (had + got)[real]
    return [out, full, s["weights"]]


def _plain_evict(s):
    c = s["case"]
    keys, most = s["keys"].long()[:, None, None], s["most"]
    keep = torch.minimum(s["keep"].long()[:, None, None], keys)
    at = torch.arange(most, device="cuda")
    page, place = s["table"].long()[:, at // c["page"]].clamp_min(0), at % c["page"]
    w = s["weights"][page, place].transpose(1, 2)                         # [B, Hkv, S]
    sinks = keep.clamp_max(c["sinks"])
    recent = torch.minimum(keep - sinks, torch.full_like(keep, c["recent"]))
    w = w.masked_fill((at < sinks) | (at >= keys - recent), math.inf).masked_fill(at >= keys, -math.inf)
    order = w.sort(dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(-1, order, at.expand_as(order))
    kept = rank < keep
    # the kept slots in their order, then the others
    slots = (~kept).to(torch.int8).sort(dim=-1, stable=True)[1]
    slots = torch.nn.functional.pad(slots, (0, c["keep"]))[..., :c["keep"]]                # [B, Hkv, K]
    to = torch.arange(c["keep"], device="cuda")
    real = (to < keep).expand(-1, c["hkv"], -1)
    head = torch.arange(c["hkv"], device="cuda")[:, None].expand_as(slots)
    seq = torch.arange(s["seqs"], device="cuda")[:, None, None].expand_as(slots)
    old, new = s["table"].long(), (s["table"] if s["new_table"] is None else s["new_table"]).long()
    src = (old[seq, slots // c["page"]][real], (slots % c["page"])[real], head[real])
    to = to.expand_as(slots)
    dst = (new[seq, (to // c["page"]).clamp_max(new.shape[1] - 1)][real], (to % c["page"])[real], head[real])
    for name in ("kc", "vc", "weights"):
        s[name][dst] = s[name][src]
    return [s["kc"], s["vc"], s["weights"], keep.flatten().int(), slots.masked_fill(~real, -1).int()]


# ------------------------------------------------------------------------------ the library's calls
def _own_fwd(s):
    import variable_length_packed_gb300 as thd
    c = s["case"]
    return list(thd.thd_attn_fwd(s["q"], s["k"], s["v"], s["cu"], s["cu"], s["padded"], s["padded"], s["causal"], s["seqs"],
                                 s["longest"], s["scale"], window=(c["left"], c["right"]), sink_tokens=c["sinks"]))


def _own_bwd(s):
    import variable_length_packed_gb300 as thd
    c = s["case"]
    return list(thd.thd_attn_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["cu"], s["cu"], s["padded"],
                                 s["padded"], s["causal"], s["seqs"], s["longest"], s["scale"],
                                 window=(c["left"], c["right"]), sink_tokens=c["sinks"]))


def _own_paged(s):
    import variable_length_packed_gb300 as thd
    c = s["case"]
    more = {} if c["op"] == "paged" else {"key_weights": s["weights"]}
    got = thd.thd_attn_paged(s["q"], s["kc"], s["vc"], s["table"], s["keys"], s["cu"], cu_seqlens_q_padded=s["padded"],
                             batch_size=s["seqs"], max_seqlen_q=s["longest"], softmax_scale=s["scale"],
                             window=(c["left"], 0 if c["left"] >= 0 else -1), sink_tokens=c["sinks"], **more)
    return list(got) + list(more.values())


def _own_evict(s):
    import variable_length_packed_gb300 as thd
    c = s["case"]
    kept = torch.empty((s["seqs"], c["hkv"], c["keep"]), dtype=torch.int32, device="cuda")
    lens = thd.thd_kv_evict(s["kc"], s["vc"], s["weights"], s["table"], s["keys"], s["keep"], batch_size=s["seqs"],
                            new_page_table=s["new_table"], sink_tokens=c["sinks"], recent_tokens=c["recent"], kept=kept)
    return [s["kc"], s["vc"], s["weights"], lens, kept]


_PLAIN = {"fwd": _plain_fwd, "bwd": _plain_bwd, "paged": _plain_paged, "weights": _plain_paged, "evict": _plain_evict}
_OWN = {"fwd": _own_fwd, "bwd": _own_bwd, "paged": _own_paged, "weights": _own_paged, "evict": _own_evict}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ least work
def _pairs(n, left, right, sinks, causal):
    """Pairs of a query and a key that it sees, in one sequence of n rows."""
    if causal:
        return sum(min(i + 1, left + 1 + min(sinks, max(0, i - left))) for i in range(n))
    return sum(min(n, i + right + 1) - max(0, i - left) + min(sinks, max(0, i - left)) +
               max(0, min(sinks, n) - (i + right + 1)) for i in range(n))


def work(case):
    c = case
    if c["op"] == "evict":
        keep = min(c["keys"], c["seqs"] * c["keep"] * (0.75 if c["seqs"] > 1 else 1.0))
        return {"bytes": c["hkv"] * (4 * c["keys"] + keep * (8 * c["d"] + 12)), "flops": 0}
    if c["op"] in ("fwd", "bwd"):
        n = -(-c["tokens"] // c["seqs"])
        share = {"causal": 1.0, "full": 0.0, "mixed": 2 / 3}[c["policy"]]
        pairs = c["tokens"] / n * sum(x * _pairs(n, c["left"], c["right"], c["sinks"], k)
                                      for x, k in ((share, True), (1 - share, False)) if x)
        rows = c["tokens"] * c["d"] * (c["hq"] + c["hkv"])
        if c["op"] == "fwd":
            return {"bytes": 4 * rows + 4 * c["tokens"] * c["hq"], "flops": 4 * pairs * c["hq"] * c["d"]}
        return {"bytes": 8 * rows + 4 * c["tokens"] * c["hq"], "flops": 10 * pairs * c["hq"] * c["d"]}
    new = (c["new"] + 1) / 2 if c["ragged"] else c["new"]
    each = c["keys"] / c["seqs"]
    seen, span = each, each
    if c["left"] >= 0:
        seen, span = min(each, c["left"] + 1 + c["sinks"]), min(each, c["left"] + new + c["sinks"])
    size = 4 * span * c["hkv"] * c["d"] + 4 * new * c["hq"] * (c["d"] + 1)
    if c["op"] == "weights":
        size += 8 * span * c["hkv"]
    return {"bytes": c["seqs"] * size, "flops": 4 * c["seqs"] * seen * new * c["hq"] * c["d"]}


# ------------------------------------------------------------------------------ definitions in 64 bits
def _exact_spans(s):
    cu = s["cu"].tolist()
    at = s["padded"].tolist() if s["padded"] is not None else cu
    return [(b, at[b], cu[b + 1] - cu[b]) for b in range(s["seqs"])]


def _exact_sees(c, code, rows, cols, n):
    """Whether query `rows` sees key `cols` of a sequence of n."""
    i, j = rows[:, None], cols[None, :]
    near = (i - j <= c["left"]) & (j - i <= c["right"])
    return (near | (j < c["sinks"])) & ((j <= i) if code else (j < n))


def _exact_packed(s, c):
    """Every (sequence, head, run of rows): the rows of the buffer, its keys' and what is seen of them."""
    codes = s["causal"].tolist()
    for b, start, n in _exact_spans(s):
        for i0 in range(0, n, 2048):
            i = torch.arange(i0, min(n, i0 + 2048), device="cuda")
            low = max(0, i0 - c["left"])
            high = min(n, max(i0 + 2048 + c["right"], c["sinks"]))
            j = torch.arange(low, high, device="cuda")
            few = torch.arange(min(c["sinks"], low), device="cuda")
            j = torch.cat([few, j])
            yield start + i, start + j, _exact_sees(c, codes[b], i, j, n)


def exact(case, seed):
    c = case
    if c["op"] in ("fwd", "bwd") and work(c)["flops"] > 2.5e12:
        return None
    s = prepare(c, seed)
    if c["op"] == "fwd":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full((c["hq"], s["rows"]), -math.inf, dtype=torch.float64, device="cuda")
        for rows, cols, seen in _exact_packed(s, c):
            for h in range(c["hq"]):
                k, v = (s[x][cols, h * c["hkv"] // c["hq"]].double() for x in "kv")
                z = (s["q"][rows, h].double() @ k.T * s["scale"]).masked_fill_(~seen, -math.inf)
                lse[h, rows] = z.logsumexp(-1)
                out[rows, h] = z.softmax(-1).nan_to_num(nan=0.0) @ v
        return [out, lse]
    if c["op"] == "bwd":
        grads = [torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in "qkv"]
        for rows, cols, seen in _exact_packed(s, c):
            for h in range(c["hq"]):
                m = h * c["hkv"] // c["hq"]
                q, go, o = (s[x][rows, h].double() for x in ("q", "dout", "out"))
                k, v = (s[x][cols, m].double() for x in "kv")
                z = q @ k.T * s["scale"] - s["lse"][h, rows].double()[:, None]
                p = torch.where(seen, z, -math.inf).exp()
                ds = p * (go @ v.T - (go * o).sum(1, keepdim=True))
                grads[0][rows, h] = ds @ k * s["scale"]
                grads[1][cols, m] += ds.T @ q * s["scale"]
                grads[2][cols, m] += p.T @ go
        return grads
    if c["op"] == "evict":
        caches = [s[x].clone() for x in ("kc", "vc", "weights")]
        keys, keep, old = s["keys"].tolist(), s["keep"].tolist(), s["table"].tolist()
        new = old if s["new_table"] is None else s["new_table"].tolist()
        lens = [min(a, b) for a, b in zip(keys, keep)]
        kept = torch.full((s["seqs"], c["hkv"], c["keep"]), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            first = min(c["sinks"], n)
            last = min(c["recent"], n - first)
            where = torch.tensor([[old[b][i // c["page"]], i % c["page"]] for i in range(keys[b])], device="cuda")
            to = torch.tensor([[new[b][i // c["page"]], i % c["page"]] for i in range(n)], dtype=torch.long,
                              device="cuda").view(-1, 2)
            for h in range(c["hkv"]):
                w = s["weights"][where[:, 0], where[:, 1], h].tolist()
                middle = sorted(range(first, keys[b] - last), key=lambda i: (-w[i], i))[:n - first - last]
                got = list(range(first)) + sorted(middle) + list(range(keys[b] - last, keys[b]))
                kept[b, h, :n] = torch.tensor(got, dtype=torch.int32)
                src = where[torch.tensor(got, device="cuda").long()]
                for x, y in zip(caches, ("kc", "vc", "weights")):
                    x[to[:, 0], to[:, 1], h] = s[y][src[:, 0], src[:, 1], h]
        return [x.double() for x in caches] + [_int(lens), kept.cuda()]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((c["hq"], s["rows"]), -math.inf, dtype=torch.float64, device="cuda")
    weights = s["weights"].double()
    keys, group = s["keys"].tolist(), c["hq"] // c["hkv"]
    for b, start, n in _exact_spans(s):
        slots = torch.arange(keys[b], device="cuda")
        page, at = s["table"][b, slots // c["page"]].long(), slots % c["page"]
        mine = keys[b] - n + torch.arange(n, device="cuda")[:, None]
        seen = slots <= mine
        if c["left"] >= 0:
            seen &= (mine - slots <= c["left"]) | (slots < c["sinks"])
        for h in range(c["hkv"]):
            k, v = s["kc"][page, at, h].double(), s["vc"][page, at, h].double()
            weights[page[keys[b] - n:], at[keys[b] - n:], h] = 0.0
            for x in range(h * group, (h + 1) * group):
                z = (s["q"][start:start + n, x].double() @ k.T * s["scale"]).masked_fill(~seen, -math.inf)
                lse[x, start:start + n] = z.logsumexp(-1)
                p = z.softmax(-1)
                out[start:start + n, x] = p @ v
                weights[page, at, h] += p.sum(0)
    return [out, lse] if c["op"] == "paged" else [out, lse, weights]
