"""Timed cases of the key/value-cache operators that surround block verification.

A verify pass runs the target model on a block (or a tree) of drafted tokens, each layer
attending from the drafted tokens to a paged cache and to one another; once the block is
verified the accepted tokens' keys and values join the cache, and a cache that has outgrown
its budget keeps the positions that attention weighs most.  Four operators:

  attention  drafted tokens over the cache and over their own tree
  commit     the accepted path's keys and values into the cache
  scores     attention weight received by each cached position, accumulated
  evict      selection by accumulated weight, and the kept rows into fresh pages

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is set,
through the package's entry points.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def _attention(name, B, T, heads, kv_heads, dim, length, page, tree=False, ragged=False, fused=False):
    return {"name": name, "op": "attention", "B": B, "T": T, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "length": length, "page": page, "tree": tree, "ragged": ragged, "fused": fused}


def listed():
    return [
        # one token of one short conversation, pages of 16: the smallest call, where latency counts
        _attention("attention_1x1_len500", 1, 1, 32, 8, 128, 500, 16),
        # a block of 16 drafts after the last verified token, one sequence, a few thousand cached tokens
        _attention("attention_1x17_len8191", 1, 17, 32, 8, 128, 8191, 64, fused=True),
        # single-token decoding over two very long contexts in one contiguous buffer each
        _attention("attention_2x1_len131072", 2, 1, 64, 8, 128, 131072, 0),
        # a serving batch of blocks, ragged lengths, the drafts' projections in one fused tensor
        _attention("attention_64x17_ragged", 64, 17, 64, 8, 128, 12000, 64, ragged=True, fused=True),
        # trees of 64 nodes: 512 query rows per key/value head
        _attention("attention_8x64_tree", 8, 64, 64, 8, 128, 16384, 128, tree=True),
        # narrow heads in groups of 6, odd lengths, small pages, a small tree
        _attention("attention_24x9_d64", 24, 9, 24, 4, 64, 3001, 32, tree=True, ragged=True),
        # the accepted tokens of one sequence
        {"name": "commit_1x17", "op": "commit", "B": 1, "T": 17, "kv_heads": 8, "dim": 128, "length": 8191, "page": 64,
         "tree": False},
        # the accepted paths of a large batch of trees
        {"name": "commit_256x64_tree", "op": "commit", "B": 256, "T": 64, "kv_heads": 8, "dim": 128, "length": 1000,
         "page": 16, "tree": True},
        # weights of one accepted block over a short cache
        {"name": "scores_1x17_len4000", "op": "scores", "B": 1, "T": 17, "heads": 32, "kv_heads": 8, "dim": 128,
         "length": 4000, "page": 64, "tree": False, "ragged": False},
        # weights of a batch of blocks over long caches
        {"name": "scores_16x17_len32768", "op": "scores", "B": 16, "T": 17, "heads": 64, "kv_heads": 8, "dim": 128,
         "length": 32768, "page": 64, "tree": False, "ragged": True},
        # one sequence shrinks to a quarter
        {"name": "evict_1_4096_to_1024", "op": "evict", "B": 1, "kv_heads": 8, "dim": 128, "length": 4096, "page": 64,
         "keep": 1024, "recent": 128, "ragged": False},
        # a batch of long sequences shrinks to an odd budget
        {"name": "evict_16_32768_to_8001", "op": "evict", "B": 16, "kv_heads": 8, "dim": 128, "length": 32768,
         "page": 64, "keep": 8001, "recent": 500, "ragged": True},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "commit", "scores", "evict"])
    kv_heads = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128])
    page = rng.choice([0, 16, 32, 64, 128, 256])
    if op == "commit":
        return {"op": op, "B": _logint(rng, 1, 256), "T": _logint(rng, 1, 128), "kv_heads": kv_heads, "dim": dim,
                "length": _logint(rng, 1, 1000), "page": page, "tree": rng.random() < 0.5}
    if op == "evict":
        B = _logint(rng, 1, 32)
        length = _logint(rng, 16, min(131072, 500000 // B))
        keep = max(1, int(length * rng.uniform(0.1, 0.9)))
        return {"op": op, "B": B, "kv_heads": kv_heads, "dim": dim, "length": length, "page": page, "keep": keep,
                "recent": int(keep * rng.uniform(0.0, 0.3)), "ragged": rng.random() < 0.5}
    group = rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
    B, T = _logint(rng, 1, 64), _logint(rng, 1, 128)
    # no more query rows x keys than the largest tree, no more cached bytes than the largest batch
    most = min(131072, 400000 // B, 1 << 26, (8 * 512 * 8 * 16384) // (B * T * group * kv_heads))
    case = {"op": op, "B": B, "T": T, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
            "length": _logint(rng, 1, max(1, most)), "page": page, "tree": rng.random() < 0.5,
            "ragged": rng.random() < 0.5}
    if op == "attention":
        case["fused"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _lengths(case, rng):
    B, n = case["B"], case["length"]
    if not case.get("ragged", op_ragged(case)):
        return np.full(B, n, np.int32)
    lens = rng.integers(n // 8, n + 1, B).astype(np.int32)
    lens[0] = n
    return lens


def op_ragged(case):
    return case["op"] == "commit" and case["B"] > 1


def _normal(gen, shape, std=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return x.normal_(0.0, std, generator=gen)


def _pool(case, capacity, gen, rng, blank=False):
    """Keys and values [pages, page, kv_heads, dim] and the block table (None: sequence b is page b)."""
    B, H, D, page = case["B"], case["kv_heads"], case["dim"], case["page"]
    if page == 0:
        shape, table = (B, capacity, H, D), None
    else:
        per = -(-capacity // page)
        shape = (B * per + 3, page, H, D)
        table = torch.from_numpy(rng.permutation(B * per + 3)[:B * per].reshape(B, per).astype(np.int32)).cuda()
    if blank:
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), \
            torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), table
    k, v = _normal(gen, shape), _normal(gen, shape)
    # a few positions of every page draw much more attention than the rest, as they do in trained models
    k[:, :: max(1, shape[1] // 2)] *= 2.0
    return k, v, table


def _tree(case, rng):
    """ancestors-or-self [B, T, T] of random trees whose nodes follow their parents, and each node's depth."""
    B, T = case["B"], case["T"]
    sees = np.zeros((B, T, T), bool)
    depth = np.zeros((B, T), np.int64)
    parent = np.zeros((B, T), np.int64)
    every = np.arange(B)
    for t in range(T):
        if t:
            p = t - 1 - np.minimum(rng.integers(0, 6, B), t - 1)
            parent[:, t], depth[:, t] = p, depth[every, p] + 1
            sees[:, t] = sees[every, p]
        sees[:, t, t] = True
    return sees, parent, depth


def _mask_words(sees):
    B, T, _ = sees.shape
    words = (T + 63) // 64
    bits = np.zeros((B, T, words * 64), np.uint8)
    bits[:, :, :T] = sees
    return torch.from_numpy(np.packbits(bits, axis=-1, bitorder="little").view(np.int64).copy()).cuda()


def _path(case, rng):
    """The accepted path of each sequence: its node ids (-1 after the end) and its length."""
    B, T = case["B"], case["T"]
    if not case["tree"]:
        return None, rng.integers(1, T + 1, B).astype(np.int32)
    _, parent, depth = _tree(case, rng)
    path, count = np.full((B, T), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        node = int(rng.integers(0, T))
        count[b] = depth[b, node] + 1
        for i in range(int(count[b]) - 1, -1, -1):
            path[b, i], node = node, parent[b, node]
    return torch.from_numpy(path).cuda(), count


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, B, H, D = case["op"], case["B"], case["kv_heads"], case["dim"]
    T = case.get("T", 0)
    lens = _lengths(case, rng)
    capacity = case["length"] + T
    st = {"case": case, "capacity": capacity, "scale": 1.0 / math.sqrt(D)}
    st["k"], st["v"], st["table"] = _pool(case, capacity, gen, rng)
    st["len"] = torch.from_numpy(lens).cuda()
    if op in ("attention", "commit"):
        heads = case.get("heads", 0)
        if case.get("fused"):
            qkv = _normal(gen, (B, T, heads + 2 * H, D))
            st["q"], st["k_new"], st["v_new"] = qkv[:, :, :heads], qkv[:, :, heads:heads + H], qkv[:, :, heads + H:]
        else:
            st["q"] = _normal(gen, (B, T, heads, D)) if heads else None
            st["k_new"], st["v_new"] = _normal(gen, (B, T, H, D)), _normal(gen, (B, T, H, D))
    if op == "attention":
        st["mask"] = _mask_words(_tree(case, rng)[0]) if case["tree"] else None
        st["out"] = torch.empty((B, T, heads, D), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty((B, T, heads), dtype=torch.float32, device="cuda")
    if op in ("commit", "scores"):
        path, count = _path(case, rng)
        st["path"], st["count"] = path, torch.from_numpy(count).cuda()
    if op != "attention":
        st["scores"] = torch.empty((B, H, capacity), dtype=torch.float32, device="cuda").exponential_(generator=gen)
    if op in ("commit", "evict"):
        st["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if op == "scores":
        st["q"] = _normal(gen, (B, T, case["heads"], D))
        # the statistics that the attention pass over the same cache leaves
        st["lse"] = torch.logsumexp(_logits(st), -1).permute(0, 3, 1, 2).reshape(B, T, case["heads"]).contiguous()
    if op == "evict":
        st["dst_k"], st["dst_v"], st["dst_table"] = _pool(case, case["keep"], gen, rng, blank=True)
        st["kept"] = torch.empty((B, H, case["keep"]), dtype=torch.int32, device="cuda")
        st["dst_scores"] = torch.zeros((B, H, case["keep"]), dtype=torch.float32, device="cuda")
    if own:
        from draft_selection_dflash2_gb300 import api
        h = st["handle"] = _handle(api)
        st["cache"] = api.KVCache(st["k"], st["v"], st["table"])
        if op == "attention":
            st["workspace"] = _bytes(api.tree_attention_workspace(h, B, T, case["heads"], H, D))
        if op == "evict":
            st["dst"] = api.KVCache(st["dst_k"], st["dst_v"], st["dst_table"])
    return st


_handles = {}


def _handle(api):
    device = torch.cuda.current_device()
    if device not in _handles:
        _handles[device] = api.Handle(device)
    return _handles[device]


def _bytes(n):
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------
def _rows(x, table, n):
    """The first n positions of every sequence: [B, n, kv_heads, dim]."""
    if table is None:
        return x[:, :n]
    B, page = table.shape[0], x.shape[1]
    return x[table[:, :-(-n // page)].long()].reshape(B, -1, *x.shape[2:])[:, :n]


def _logits(st):
    """Scaled products of every query with every cached key, -inf past the sequence's end: [B, kv_heads, group, T, n]."""
    c, n = st["case"], st["case"]["length"]
    q = st["q"].float().reshape(c["B"], c["T"], c["kv_heads"], -1, c["dim"])
    keys = _rows(st["k"], st["table"], n).float()
    s = torch.einsum("bthgd,bshd->bhgts", q, keys).mul_(st["scale"])
    past = torch.arange(n, device="cuda")[None] >= st["len"][:, None]
    return s.masked_fill_(past[:, None, None, None], -math.inf)


def _attention_plain(st):
    c = st["case"]
    B, T, H, D, n = c["B"], c["T"], c["kv_heads"], c["dim"], c["length"]
    q = st["q"].float().reshape(B, T, H, -1, D)
    s_new = torch.einsum("bthgd,bshd->bhgts", q, st["k_new"].float()) * st["scale"]
    node = torch.arange(T, device="cuda")
    if st["mask"] is None:
        sees = (node[None] <= node[:, None])[None]
    else:
        sees = ((st["mask"][:, :, node // 64] >> (node % 64)) & 1).bool()
    s_new = s_new.masked_fill(~sees[:, None, None], -math.inf)
    s = torch.cat([_logits(st), s_new], -1)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    past = torch.arange(n, device="cuda")[None] >= st["len"][:, None]
    values = _rows(st["v"], st["table"], n).float().masked_fill(past[:, :, None, None], 0.0)
    values = torch.cat([values, st["v_new"].float()], 1)
    o = torch.einsum("bhgts,bshd->bhgtd", p, values) / torch.where(total == 0.0, 1.0, total)
    out = o.permute(0, 3, 1, 2, 4).reshape(B, T, -1, D).to(torch.bfloat16)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, T, -1)
    return {"out": out, "lse": lse}


def _commit_plain(st):
    c = st["case"]
    B, T, H = c["B"], c["T"], c["kv_heads"]
    i = torch.arange(T, device="cuda")[None].expand(B, T)
    taken = i < st["count"][:, None]
    node = i if st["path"] is None else torch.where(taken, st["path"], 0).long()
    at = (st["len"][:, None] + i).long()
    if st["table"] is None:
        page, off = torch.arange(B, device="cuda")[:, None].expand(B, T), at
    else:
        size = st["k"].shape[1]
        page, off = torch.gather(st["table"].long(), 1, at // size), at % size
    which = node[:, :, None, None].expand(B, T, H, c["dim"])
    for new, x in ((st["k_new"], st["k"]), (st["v_new"], st["v"])):
        x[page, off] = torch.where(taken[:, :, None, None], torch.gather(new, 1, which), x[page, off])
    where = at[:, None].expand(B, H, T)
    old = torch.gather(st["scores"], 2, where)
    st["scores"].scatter_(2, where, torch.where(taken[:, None], 0.0, old))
    return {"k": st["k"], "v": st["v"], "scores": st["scores"], "new_len": st["len"] + st["count"]}


def _scores_plain(st):
    c = st["case"]
    B, T, H, n = c["B"], c["T"], c["kv_heads"], c["length"]
    lse = st["lse"].reshape(B, T, H, -1).permute(0, 2, 3, 1)
    p = _logits(st).sub_(lse[..., None]).exp_()
    i = torch.arange(T, device="cuda")
    if st["path"] is None:
        counts = i[None] < st["count"][:, None]
    else:
        counts = torch.zeros((B, T + 1), dtype=torch.bool, device="cuda")
        counts = counts.scatter_(1, torch.where(st["path"] < 0, T, st["path"]).long(), True)[:, :T]
    w = (p * counts[:, None, None, :, None]).sum((2, 3))
    st["scores"][:, :, :n] += w
    return {"scores": st["scores"]}


def _evict_plain(st):
    c = st["case"]
    B, H, D, n, keep = c["B"], c["kv_heads"], c["dim"], c["length"], c["keep"]
    at = torch.arange(n, device="cuda")[None]
    end = st["len"][:, None]
    rank = st["scores"][:, :, :n].masked_fill((at >= end - c["recent"])[:, None], math.inf)
    rank = rank.masked_fill((at >= end)[:, None], -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :, :keep]
    new_len = torch.minimum(st["len"], torch.tensor(keep, device="cuda", dtype=torch.int32))
    live = (torch.arange(keep, device="cuda")[None] < new_len[:, None])[:, None]
    kept = torch.where(live, order, n).sort(dim=-1).values
    first = torch.where(live, kept, 0)
    slot = torch.arange(keep, device="cuda")[None].expand(B, keep)
    if st["dst_table"] is None:
        page, off = torch.arange(B, device="cuda")[:, None].expand(B, keep), slot
    else:
        size = st["dst_k"].shape[1]
        page, off = torch.gather(st["dst_table"].long(), 1, slot // size), slot % size
    which = first.permute(0, 2, 1)[..., None].expand(B, keep, H, D)
    for x, y in ((st["k"], st["dst_k"]), (st["v"], st["dst_v"])):
        rows = torch.gather(_rows(x, st["table"], n), 1, which)
        y[page, off] = torch.where(live.permute(0, 2, 1)[..., None], rows, y[page, off])
    st["dst_scores"].copy_(torch.where(live, torch.gather(st["scores"], 2, first), st["dst_scores"]))
    return {"kept": torch.where(live, kept, -1).to(torch.int32), "new_len": new_len, "k": st["dst_k"],
            "v": st["dst_v"], "scores": st["dst_scores"]}


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"attention": _attention_plain, "commit": _commit_plain, "scores": _scores_plain,
                "evict": _evict_plain}[op](st)
    from draft_selection_dflash2_gb300 import api
    h, cache = st["handle"], st["cache"]
    if op == "attention":
        out, lse = api.tree_attention(h, st["q"], cache, st["len"], st["k_new"], st["v_new"], tree_mask=st["mask"],
                                      scale=st["scale"], out=st["out"], lse=st["lse"], workspace=st["workspace"])
        return {"out": out, "lse": lse}
    if op == "commit":
        new_len = api.cache_commit(h, st["k_new"], st["v_new"], cache, st["len"], st["count"], path=st["path"],
                                   scores=st["scores"], new_len=st["new_len"])
        return {"k": st["k"], "v": st["v"], "scores": st["scores"], "new_len": new_len}
    if op == "scores":
        return {"scores": api.cache_scores(h, st["q"], st["lse"], cache, st["len"], st["scores"], count=st["count"],
                                           path=st["path"], scale=st["scale"])}
    kept, new_len, scores = api.cache_evict(h, st["scores"], cache, st["len"], st["dst"], st["case"]["keep"],
                                            st["case"]["recent"], kept=st["kept"], new_len=st["new_len"],
                                            dst_scores=st["dst_scores"])
    return {"kept": kept, "new_len": new_len, "k": st["dst_k"], "v": st["dst_v"], "scores": scores}


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    op, B, H, D = case["op"], case["B"], case["kv_heads"], case["dim"]
    n = float(case["length"])
    if case.get("ragged", op_ragged(case)):
        n *= 9.0 / 16.0            # lengths are uniform over [n/8, n]
    T = case.get("T", 0)
    row = 2.0 * D                  # bytes of one bf16 row
    if op == "attention":
        q = B * T * case["heads"]
        seen = n + (T / 4.0 if case["tree"] else (T + 1) / 2.0)
        return {"bytes": 2 * q * row + 4 * q + 2 * B * H * (n + T) * row, "flops": 4.0 * q * seen * D}
    accepted = T / 4.0 if case.get("tree") else (T + 1) / 2.0
    if op == "commit":
        return {"bytes": 4 * B * accepted * H * row + 4 * B * accepted * H + 12 * B, "flops": 0}
    if op == "scores":
        q = B * accepted * case["heads"]
        return {"bytes": q * row + 4 * q + B * H * n * (row + 8), "flops": 2.0 * q * n * D}
    kept = min(float(case["keep"]), n)
    return {"bytes": B * H * (4 * n + 12 * kept + 4 * kept * row), "flops": 0}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _sequence(x, table, b, n):
    """Positions 0..n-1 of sequence b, [n, kv_heads, dim] in 64 bits."""
    pages = x[b] if table is None else x[table[b].long()].flatten(0, 1)
    return pages[:n].double()


def exact(case, seed):
    op = case["op"]
    if op not in ("attention", "scores"):
        return None                # rows are moved, not computed
    st = prepare(case, seed)
    B, T, H, D = case["B"], case["T"], case["kv_heads"], case["dim"]
    G = case["heads"] // H
    if 4.0 * B * T * case["heads"] * case["length"] * D > 4e12:
        return None
    if op == "scores":
        want = st["scores"].double()
        for b in range(B):
            n, m = int(st["len"][b]), int(st["count"][b])
            nodes = list(range(m)) if st["path"] is None else st["path"][b, :m].tolist()
            keys = _sequence(st["k"], st["table"], b, n)
            for head in range(H):
                rows = st["q"][b, nodes, head * G:(head + 1) * G].double().reshape(-1, D)
                lse = st["lse"][b, nodes, head * G:(head + 1) * G].double().reshape(-1, 1)
                want[b, head, :n] += torch.exp(rows @ keys[:, head].T * st["scale"] - lse).sum(0)
        return {"scores": want}
    out = torch.empty((B, T, case["heads"], D), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, T, case["heads"]), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(st["len"][b])
        if st["mask"] is None:
            sees = torch.ones((T, T), dtype=torch.bool, device="cuda").tril()
        else:
            words = st["mask"][b].cpu().numpy().view(np.uint64)
            sees = np.array([[(int(words[t, s // 64]) >> (s % 64)) & 1 for s in range(T)] for t in range(T)], bool)
            sees = torch.from_numpy(sees).cuda()
        keys = torch.cat([_sequence(st["k"], st["table"], b, n), st["k_new"][b].double()])
        values = torch.cat([_sequence(st["v"], st["table"], b, n), st["v_new"][b].double()])
        hidden = torch.cat([torch.zeros((T, n), dtype=torch.bool, device="cuda"), ~sees], 1)
        for head in range(case["heads"]):
            z = st["q"][b, :, head].double() @ keys[:, head // G].T * st["scale"]
            z[hidden] = -math.inf
            lse[b, :, head] = torch.logsumexp(z, 1)
            out[b, :, head] = torch.softmax(z, 1) @ values[:, head // G]
    return {"out": out, "lse": lse}
