"""The cases that the serving operators around the quantized projections are
measured on: rotary positions with the append to a paged cache, attention of
new tokens over that cache, and the pages' own bookkeeping (free, fork,
reserve, copy, compact).

Where ``own`` is false, ``run`` computes an operator in elementary torch
operations; where it is true, it calls the library.  ``exact`` computes the
same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def qmm():
    from block_quantized_weight_matmulnbits_amd import qmm as q
    return q


# -- the cases ---------------------------------------------------------------

def rope(name, **kw):
    c = dict(op="rope", name=name, dtype="bf16", q_heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, scaling="none", factor=1.0, base=500000.0, seqs=1, tokens=1,
             context=0, page=16, token_major=False, shift=0)
    c.update(kw)
    return c


def attend(name, **kw):
    c = dict(op="attend", name=name, dtype="bf16", q_heads=32, kv_heads=8, dim=128, seqs=1,
             new=1, singles=0, longest=1024, shortest=1, page=16, token_major=False, causal=True,
             window=0, cap=0.0)
    c.update(kw)
    return c


def pages(name, op, **kw):
    c = dict(op=op, name=name, planes=64, pages=1024, page=16, elems=16384, count=16, longest=512,
             grow=1, share=0.5)
    c.update(kw)
    return c


def listed():
    return [
        # One decode step of 8 sequences, a token each: pairs of neighbours
        # over half the head, frequencies stretched for a long context and
        # positions near a million.
        rope("rope_decode_8", dtype="f16", q_heads=28, kv_heads=4, rot=64, interleaved=True,
             scaling="yarn", factor=16.0, base=10000.0, seqs=8, tokens=8, context=1400, page=64,
             token_major=True, shift=1000000),
        # A prefill of 16384 tokens, five prompts of uneven length, the heads
        # of the 4096-wide layer (32 query, 8 key/value heads of 128).
        rope("rope_prefill_16384", seqs=5, tokens=16384),
        # One user waiting for the next token: latency.
        attend("attend_decode_1", dtype="f16", longest=1037, shortest=1037),
        # A batch of 64 chats at uneven lengths: the ordinary decode step.
        attend("attend_decode_64", seqs=64, longest=8191, shortest=17),
        # Two long documents, a token each: work has to be split along the keys.
        attend("attend_decode_long_2", seqs=2, longest=131071, shortest=90001, page=64,
               token_major=True),
        # Checking five guessed tokens each in 32 bits, 7 query heads to a
        # key/value head, a head of 80, a sliding window and a capped score.
        attend("attend_verify_f32", dtype="f32", q_heads=28, kv_heads=4, dim=80, seqs=7, new=5,
               longest=2500, shortest=3, page=32, window=1024, cap=30.0),
        # A chunked prefill between decodes: three chunks and six single tokens.
        attend("attend_chunks_mixed", seqs=9, new=509, singles=6, longest=9001, shortest=400),
        # The largest: 4096 new tokens after 12288 cached ones.
        attend("attend_prefill_4096", new=4096, longest=16384, shortest=16384, page=32),
        # A beam search turns over: 4 beams dropped, their slots forked anew,
        # one layer's keys and values.
        pages("fork_beams_4", "fork", planes=2, pages=200, count=4, longest=700),
        # 48 samples started from shared prompts, 32 layers' keys and values.
        pages("fork_samples_48", "fork", pages=1536, count=48, longest=380, grow=33),
        # A small pool with holes, closed up before it shrinks.
        pages("compact_small", "compact", planes=4, pages=257, count=12, longest=200),
        # The whole cache of 32 layers, half of it holes; 2 MiB a page.
        pages("compact_large", "compact", pages=1000, count=60, longest=250),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        c = drawn(rng, spread)
        w = work(c)
        scores = c["op"] == "attend" and c["seqs"] * c["new"] * c["q_heads"] * c["longest"]
        if w["bytes"] <= 1e9 and w["flops"] <= 9e11 and scores <= 2e9:
            del c["name"]
            return c


def drawn(rng, spread):
    kind = rng.choice(["rope", "attend", "attend", "attend", "fork", "compact", "copy"])
    if kind == "rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        kv = rng.choice([1, 2, 4, 8])
        c = rope("", dtype=rng.choice(["bf16", "f16", "f32"]), q_heads=kv * rng.randint(1, 8),
                 kv_heads=kv, dim=dim, rot=rng.choice([dim, dim // 2, dim // 4 * 2]),
                 interleaved=rng.random() < 0.4,
                 scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                 factor=rng.choice([2.0, 4.0, 8.0, 32.0]), base=rng.choice([1e4, 5e5, 1e6]),
                 tokens=spread(1, 6000), context=spread(1, 4000),
                 page=rng.choice([1, 8, 16, 32, 64, 128]), token_major=rng.random() < 0.5,
                 shift=rng.choice([0, 0, 1000, 2000000]))
        c["seqs"] = rng.randint(1, min(c["tokens"], 24))
    elif kind == "attend":
        kv = rng.choice([1, 2, 4, 8])
        c = attend("", dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                   q_heads=kv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), kv_heads=kv,
                   dim=rng.choice([64, 80, 96, 128, 128, 192, 256]), page=rng.choice([8, 16, 32, 64, 128]),
                   token_major=rng.random() < 0.5, causal=rng.random() < 0.85,
                   window=rng.choice([0, 0, 0, spread(1, 3000)]),
                   cap=rng.choice([0.0, 0.0, 0.0, 50.0]))
        style = rng.choice(["decode", "guess", "chunk", "chunk"])
        if style == "chunk":
            c.update(seqs=rng.randint(1, 6), new=spread(17, 700))
            c["singles"] = rng.randint(0, c["seqs"] - 1)
            c["longest"] = max(c["new"] + 1, spread(20, 5000))
        else:
            c.update(seqs=spread(1, 80), new=1 if style == "decode" else rng.randint(2, 12))
            c["longest"] = max(c["new"] + 1, min(spread(20, 60000), 200000 // c["seqs"]))
        c["shortest"] = rng.randint(1, c["longest"])
    else:
        c = pages("", kind, planes=2 * spread(1, 32), pages=spread(40, 900),
                  page=rng.choice([8, 16, 32]), elems=rng.choice([1024, 4096, 8 * 1160, 16384]),
                  longest=spread(9, 400), grow=rng.randint(0, 40), share=rng.choice([0.0, 0.5, 0.9]))
        # A third of the pool is room for the forks and their next tokens.
        c["count"] = spread(1, max(1, min(40, c["pages"] // (3 * (3 + c["grow"] // c["page"])))))
    return c


# -- inputs ------------------------------------------------------------------

def frequencies(c):
    """Radians a position turns each pair by, in 64 bits, and the factor on
    cosine and sine, for the plain and the stretched forms."""
    d, base, f = c["rot"], c["base"], c["factor"]
    i = np.arange(0, d, 2, dtype=np.float64)
    if c["scaling"] == "ntk":
        base = base * f ** (d / (d - 2)) if d > 2 else base
    w = base ** (-i / d)
    if c["scaling"] == "linear":
        w = w / f
    if c["scaling"] == "yarn":
        turns = 4096 * w / (2 * math.pi)            # over the context trained on
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        w = w * keep + w / f * (1 - keep)
        return w, 0.1 * math.log(f) + 1.0
    return w, 1.0


def layout(c, rng):
    """Lengths, tables and the number of pages of a batch (host arrays).  The
    lengths are the case's own, so that its outputs keep their shapes; which
    pages hold them is drawn."""
    S, order_rng = c["seqs"], rng
    rng = np.random.default_rng(7)
    if c["op"] == "rope":
        cut = np.sort(rng.choice(np.arange(1, c["tokens"]), S - 1, replace=False)) if S > 1 else []
        new = np.diff(np.concatenate([[0], cut, [c["tokens"]]])).astype(np.int64)
        lens = new + (rng.integers(0, c["context"] + 1, S) if c["context"] else 0)
    else:
        lens = rng.integers(c["shortest"], c["longest"] + 1, S)
        lens[0] = c["longest"]
        lens[-1] = c["shortest"] if S > 1 else lens[-1]
        new = np.full(S, c["new"], dtype=np.int64)
        if c["singles"]:
            new[S - c["singles"]:] = 1
        new = np.minimum(new, lens)
    per = -(-lens // c["page"])
    total = int(per.sum()) + 3
    order = order_rng.permutation(total)
    width = int(per.max()) + 1
    table = np.full((S, width), -1, dtype=np.int32)
    at = 0
    for s in range(S):
        table[s, :per[s]] = order[at:at + per[s]]
        at += per[s]
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return starts, lens.astype(np.int32), table, total


def cache(c, total, dtype, g):
    """Pages [pages, kv_heads, page, dim], either head by head or token by
    token in memory."""
    shape = (total, c["page"], c["kv_heads"], c["dim"]) if c["token_major"] else \
        (total, c["kv_heads"], c["page"], c["dim"])
    t = torch.randn(shape, device=DEV, generator=g, dtype=torch.float32).to(dtype)
    return t.transpose(1, 2) if c["token_major"] else t


def prepare(case, seed):
    c = dict(case)
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("rope", "attend"):
        dtype = TYPES[c["dtype"]]
        starts, lens, table, total = layout(c, rng)
        T, H, KV, D = int(starts[-1]), c["q_heads"], c["kv_heads"], c["dim"]
        s["starts"], s["lens"], s["table"] = (torch.from_numpy(a).to(DEV) for a in (starts, lens, table))
        s["max_new"], s["max_len"] = int(np.diff(starts).max()), int(lens.max())
        s["k_pages"], s["v_pages"] = cache(c, total, dtype, g), cache(c, total, dtype, g)
        # One row a token, query, key and value heads side by side, as the
        # stacked projection writes it.
        if c["op"] == "rope":
            qkv = torch.randn(T, H + 2 * KV, D, device=DEV, generator=g).to(dtype)
            s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
            w, s["factor"] = frequencies(c)
            s["inv_freq"] = torch.from_numpy(w).to(DEV)
            s["positions"] = None
            if c["shift"]:
                pos = np.concatenate([np.arange(l - n, l) for n, l in zip(np.diff(starts), lens)])
                s["positions"] = torch.from_numpy((pos + c["shift"]).astype(np.int32)).to(DEV)
            s["out"] = torch.empty(T, H, D, dtype=dtype, device=DEV)
        else:
            # Scores of a few units, so that some keys stand out.
            s["q"] = (1.7 * torch.randn(T, H, D, device=DEV, generator=g)).to(dtype)
            s["out"] = torch.empty(T, H, D, dtype=dtype, device=DEV)
            s["lse"] = torch.empty(T, H, dtype=torch.float32, device=DEV)
        if own:
            q = qmm()
            s["kv"] = q.PagedKV(s["k_pages"], s["v_pages"])
            s["batch"] = q.PagedBatch(s["starts"], s["lens"], s["table"], T, s["max_new"], s["max_len"])
            if c["op"] == "attend":
                n = q.qmm_paged_attention_workspace_size(s["batch"], H, KV, D)
                s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
        return s

    P, n, ps = c["pages"], c["count"], c["page"]
    s["data"] = torch.empty(c["planes"], P, c["elems"], dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    if c["op"] == "copy":
        m = min(n * 4, P // 2)
        order = rng.permutation(P).astype(np.int32)
        s["src"], s["dst"] = (torch.from_numpy(order[a:a + m].copy()).to(DEV) for a in (0, m))
        if own:
            s["pool"] = qmm().PagePool(s["data"])
        return s
    # n sequences, some starting with the pages of the one before, and for a
    # fork n beams that are about to be dropped, each with pages of its own.
    free = list(rng.permutation(P if c["op"] == "compact" else P * 2 // 3))
    width = -(-(c["longest"] + c["grow"]) // ps) + 2
    slots = 2 * n + 1
    table, lens, refs = np.full((slots, width), -1, np.int32), np.zeros(slots, np.int32), np.zeros(P, np.int32)
    spare = len(free) // 2
    for i in range(n if c["op"] == "compact" else 2 * n):
        length = int(rng.integers(1, c["longest"] + 1))
        full, need = length // ps, -(-length // ps)
        shared = min(full, int(lens[i - 1]) // ps) if i and i < n and rng.random() < c["share"] else 0
        if need - shared > len(free) - spare:
            # No pages left for it: the first page of the one before, shared.
            length, need, shared = ps, 1, 1
        row = [int(table[i - 1, j]) for j in range(shared)] + [int(free.pop()) for _ in range(need - shared)]
        table[i, :need], lens[i] = row, length
        np.add.at(refs, row, 1)
    s["table"], s["lens"], s["refs"] = (torch.from_numpy(a).to(DEV) for a in (table, lens, refs))
    if c["op"] == "fork":
        s["parents"] = torch.from_numpy(rng.integers(0, n, n).astype(np.int32)).to(DEV)
        s["children"] = torch.from_numpy((n + rng.permutation(n)).astype(np.int32)).to(DEV)
        s["grow"] = torch.full((n,), c["grow"], dtype=torch.int32, device=DEV)
        s["status"] = torch.zeros(2, dtype=torch.int32, device=DEV)
    else:
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        s["live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if own:
        q = qmm()
        s["pool"] = q.PagePool(s["data"], s["refs"], s["table"], s["lens"], ps)
        s["workspace"] = torch.zeros(q.qmm_pages_workspace_size(s["pool"], n), dtype=torch.uint8, device=DEV)
    return s


# -- one pass ----------------------------------------------------------------

def plain_rope(s):
    c = s["case"]
    T = s["q"].shape[0]
    token = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["starts"][1:].contiguous(), token, right=True)
    slot = s["lens"][seq].long() - s["starts"][1:][seq].long() + token
    pos = slot if s["positions"] is None else s["positions"].long()
    angle = pos.double()[:, None] * s["inv_freq"]
    cos = (torch.cos(angle) * s["factor"]).float()[:, None]
    sin = (torch.sin(angle) * s["factor"]).float()[:, None]
    rot = c["rot"]

    def turn(x):
        x = x.float()
        a, b = (x[..., :rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        u, w = a * cos - b * sin, b * cos + a * sin
        y = torch.stack([u, w], -1).flatten(-2) if c["interleaved"] else torch.cat([u, w], -1)
        return torch.cat([y, x[..., rot:]], -1).to(s["q"].dtype)

    page = s["table"][seq, torch.div(slot, c["page"], rounding_mode="floor")].long()
    s["out"].copy_(turn(s["q"]))
    s["k_pages"][page, :, slot % c["page"]] = turn(s["k"])
    s["v_pages"][page, :, slot % c["page"]] = s["v"]
    return s["out"], s["k_pages"], s["v_pages"]


def plain_attend(s):
    c = s["case"]
    T, H, D = s["q"].shape
    KV, ps, S, n, L = c["kv_heads"], c["page"], c["seqs"], s["max_new"], s["max_len"]
    G = H // KV
    used = s["table"][:, :-(-L // ps)].long().clamp(min=0)
    k, v = (t[used].transpose(1, 2).reshape(S, KV, -1, D)[:, :, :L].float() for t in (s["k_pages"], s["v_pages"]))
    # Queries padded to the longest chunk, [S, KV, n * G, D].
    count = s["starts"][1:] - s["starts"][:-1]
    i = torch.arange(n, device=DEV)
    at = (s["starts"][:-1, None] + i).clamp(max=T - 1)
    q = s["q"][at].float().view(S, n, KV, G, D).permute(0, 2, 1, 3, 4).reshape(S, KV, n * G, D)
    score = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    if c["cap"]:
        score = c["cap"] * torch.tanh(score / c["cap"])
    j = torch.arange(L, device=DEV)
    pos = (s["lens"] - count)[:, None] + i
    see = (j < s["lens"][:, None, None]).expand(S, n, L)
    if c["causal"]:
        see = see & (j <= pos[:, :, None])
    if c["window"]:
        see = see & (j > pos[:, :, None] - c["window"])
    see = see[:, None, :, None, :].expand(S, KV, n, G, L).reshape(S, KV, n * G, L)
    score.masked_fill_(~see, -math.inf)
    m = score.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp_(score.sub_(m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = torch.log(total) + m
    o = o.view(S, KV, n, G, D).permute(0, 2, 1, 3, 4).reshape(S * n, H, D)
    lse = lse.view(S, KV, n, G).permute(0, 2, 1, 3).reshape(S * n, H)
    token = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["starts"][1:].contiguous(), token, right=True)
    back = seq * n + token - s["starts"][seq]
    s["out"].copy_(o[back])
    s["lse"].copy_(lse[back])
    return s["out"], s["lse"]


def plain_fork(s):
    c = s["case"]
    ps, table, lens, refs, data = c["page"], s["table"], s["lens"], s["refs"], s["data"]
    parents, children = s["parents"].long(), s["children"].long()
    col = torch.arange(table.shape[1], device=DEV)
    # The dropped beams give their pages back.
    rows = table[children]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), -(rows >= 0).flatten().int())
    table[children], lens[children] = -1, 0
    # Full pages are shared, a part-filled last one is copied; then room for
    # the tokens to come.  New pages are the lowest free ones, in list order.
    rows, length = table[parents], lens[parents]
    full, part = length // ps, (length % ps != 0).int()
    share = col < full[:, None]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), share.flatten().int())
    lowest = torch.argsort((refs > 0).int(), stable=True)
    fresh = lowest[torch.cumsum(part, 0) - part]
    last = rows.gather(1, full[:, None].long().clamp(max=table.shape[1] - 1))[:, 0].clamp(min=0).long()
    src = torch.where(part > 0, last, rows[:, 0].long())
    data[:, torch.where(part > 0, fresh, src)] = data[:, src]
    refs.index_add_(0, fresh, part)
    rows = torch.where(share, rows, -1)
    rows = torch.where((col == full[:, None]) & (part[:, None] > 0), fresh[:, None].int(), rows)
    have, length = full + part, length + s["grow"]
    need = (length + ps - 1) // ps
    more = (need - have).clamp(min=0)
    first = torch.cumsum(more, 0) - more
    lowest = torch.argsort((refs > 0).int(), stable=True)
    take = (col >= have[:, None]) & (col < need[:, None])
    rank = torch.where(take, first[:, None] + col - have[:, None], 0)
    rows = torch.where(take, lowest[rank].int(), rows)
    refs.index_add_(0, lowest[rank].flatten(), take.flatten().int())
    table[children], lens[children] = rows, length.int()
    return data, refs, table, lens


def plain_compact(s):
    refs, data = s["refs"], s["data"]
    used = refs > 0
    live = used.sum()
    P = refs.numel()
    at = torch.arange(P, device=DEV)
    hole, move = ~used & (at < live), used & (at >= live)
    # The k-th used page past the end goes to the k-th hole.
    holes = torch.argsort((~hole).int(), stable=True)
    to = torch.where(move, holes[(torch.cumsum(move, 0) - 1).clamp(min=0)], at)
    order = torch.argsort((~move).int(), stable=True)[:P // 2 + 1]
    order = torch.where(at[:P // 2 + 1] < move.sum(), order, order[0])
    data[:, to[order]] = data[:, order]
    s["refs_out"].zero_()
    s["refs_out"].index_add_(0, to, refs)
    s["table_out"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()].int(), s["table"]))
    s["live"].copy_(live)
    return data, s["refs_out"], s["table_out"], s["live"]


def plain_copy(s):
    s["data"][:, s["dst"].long()] = s["data"][:, s["src"].long()]
    return s["data"]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"rope": plain_rope, "attend": plain_attend, "fork": plain_fork, "compact": plain_compact,
                "copy": plain_copy}[op](s)
    q = qmm()
    if op == "rope":
        q.qmm_rope_append(s["q"], s["k"], s["v"], s["out"], s["kv"], s["batch"], s["inv_freq"],
                          interleaved=c["interleaved"], factor=s["factor"], positions=s["positions"])
        return s["out"], s["k_pages"], s["v_pages"]
    if op == "attend":
        q.qmm_paged_attention(s["q"], s["kv"], s["batch"], s["out"], s["workspace"],
                              scale=1.0 / math.sqrt(c["dim"]), causal=c["causal"], window=c["window"],
                              softcap=c["cap"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "fork":
        q.qmm_pages_free(s["pool"], s["children"])
        q.qmm_pages_fork(s["pool"], s["parents"], s["children"], s["status"], s["workspace"])
        q.qmm_pages_reserve(s["pool"], s["children"], s["grow"], s["status"], s["workspace"])
        return s["data"], s["refs"], s["table"], s["lens"]
    if op == "compact":
        q.qmm_pages_compact(s["pool"], s["refs_out"], s["table_out"], s["live"], s["workspace"])
        return s["data"], s["refs_out"], s["table_out"], s["live"]
    q.qmm_pages_copy(s["pool"], s["src"], s["dst"])
    return s["data"]


# -- what a pass cannot do without -------------------------------------------

def work(case):
    c = case
    rng = np.random.default_rng(1)
    if c["op"] in ("rope", "attend"):
        starts, lens, _, _ = layout(c, rng)
        size = 4 if c["dtype"] == "f32" else 2
        T, H, KV, D = int(starts[-1]), c["q_heads"], c["kv_heads"], c["dim"]
        if c["op"] == "rope":
            return {"bytes": 2 * T * (H + 2 * KV) * D * size, "flops": 3 * T * (H + KV) * c["rot"]}
        pairs, keys = 0, 0
        for n, l in zip(np.diff(starts).astype(int), lens.astype(int)):
            pos = np.arange(l - n, l)
            hi = pos + 1 if c["causal"] else np.full(n, l)
            lo = np.maximum(0, pos - c["window"] + 1) if c["window"] else np.zeros(n, int)
            pairs += int((hi - lo).sum())
            keys += int(hi.max() - lo.min())
        return {"bytes": 2 * keys * KV * D * size + 2 * T * H * D * size + 4 * T * H,
                "flops": 4 * pairs * H * D}
    page = c["planes"] * c["elems"] * 2
    if c["op"] == "copy":
        return {"bytes": 2 * page * min(c["count"] * 4, c["pages"] // 2), "flops": 0}
    if c["op"] == "fork":
        # A last page is part-filled in all but one of `page` lengths.
        return {"bytes": 2 * page * c["count"] * (c["page"] - 1) / c["page"] + 8 * c["pages"], "flops": 0}
    # About half of the pool is live, half of that past the end.
    held = c["count"] * (c["longest"] / 2 / c["page"] + 1) * (1 - 0.4 * c["share"])
    live = min(c["pages"] / 2, held)
    return {"bytes": 2 * page * live * (1 - live / c["pages"]) + 8 * c["pages"], "flops": 0}


# -- from the definitions, in 64 bits ----------------------------------------

def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "rope":
        w, factor = frequencies(c)
        starts, lens, table = (s[n].cpu().numpy() for n in ("starts", "lens", "table"))
        out = s["q"].double().clone()
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        half = c["rot"] // 2
        at = np.arange(half)
        one, two = (2 * at, 2 * at + 1) if c["interleaved"] else (at, at + half)
        one, two = (torch.from_numpy(a).to(DEV) for a in (one, two))
        for i in range(c["seqs"]):
            t = torch.arange(int(starts[i]), int(starts[i + 1]), device=DEV)
            slot = np.arange(lens[i] - len(t), lens[i])
            turn = torch.polar(torch.full((len(t), half), factor, dtype=torch.float64, device=DEV),
                               torch.from_numpy(np.outer((slot + c["shift"]).astype(np.float64), w)).to(DEV))[:, None]
            # A pair is a complex number; a position turns it.
            for x, y in ((s["q"][t], "q"), (s["k"][t], "k")):
                x = x.double()
                z = torch.complex(x[..., one], x[..., two]) * turn
                x[..., one], x[..., two] = z.real, z.imag
                if y == "q":
                    out[t] = x
                else:
                    page = torch.from_numpy(table[i, slot // c["page"]].astype(np.int64)).to(DEV)
                    place = torch.from_numpy(slot % c["page"]).to(DEV)
                    kp[page, :, place] = x
                    vp[page, :, place] = s["v"][t].double()
        return out, kp, vp
    if c["op"] == "attend":
        starts, lens, table = (s[n].cpu().numpy() for n in ("starts", "lens", "table"))
        T, H, D = s["q"].shape
        G = H // c["kv_heads"]
        out = torch.zeros(T, H, D, dtype=torch.float64, device=DEV)
        lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=DEV)
        for i in range(c["seqs"]):
            n, l = int(starts[i + 1] - starts[i]), int(lens[i])
            ids = torch.from_numpy(table[i, np.arange(l) // c["page"]].astype(np.int64)).to(DEV)
            place = torch.from_numpy(np.arange(l) % c["page"]).to(DEV)
            for h in range(c["kv_heads"]):
                k, v = (t[ids, h, place].double() for t in (s["k_pages"], s["v_pages"]))
                for a in range(0, n, 256):
                    b = min(n, a + 256)
                    q = s["q"][starts[i] + a:starts[i] + b, h * G:(h + 1) * G].double().reshape(-1, D)
                    z = q @ k.T.contiguous() / math.sqrt(D)
                    if c["cap"]:
                        z = torch.tanh(z / c["cap"]) * c["cap"]
                    place_q = torch.arange(l - n + a, l - n + b, device=DEV).repeat_interleave(G)[:, None]
                    key = torch.arange(l, device=DEV)[None]
                    hide = torch.zeros(z.shape, dtype=torch.bool, device=DEV)
                    if c["causal"]:
                        hide |= key > place_q
                    if c["window"]:
                        hide |= key <= place_q - c["window"]
                    z[hide] = -math.inf
                    e = torch.logsumexp(z, -1)
                    prob = torch.exp(z - torch.where(e == -math.inf, 0.0, e)[:, None])
                    lse[starts[i] + a:starts[i] + b, h * G:(h + 1) * G] = e.view(-1, G)
                    out[starts[i] + a:starts[i] + b, h * G:(h + 1) * G] = (prob @ v).view(-1, G, D)
        return out, lse
    # The pages' tables are whole numbers and their contents are copied.
    return None
