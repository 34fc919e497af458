"""Timed cases of the operators that a served model runs around the cache and the verification.

A batch of requests often shares its beginning (a system prompt, several answers to one
question), and every token that enters the cache carries its position in its key.  Before a
block is verified, the target's logits take the request's penalties, biases and grammar into
account, position by position.  Five operators:

  prefix   attention of drafted tokens over a cache whose first positions a group of sequences
           shares, those computed once for the group
  rope     rotary positions: half or interleaved layout, part of the head, scaled frequencies
  append   keys (rotated) and values into the paged cache, the queries rotated along
  logits   penalties for repeated tokens, biases and allowed tokens, per node of a block or tree
  counts   how often each sequence has emitted each token, kept up to date

``run`` computes them with elementary torch operations in 32 bits (the angles in 64), or, where
``own`` is set, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def _prefix(name, B, groups, T, heads, kv_heads, dim, prefix, own_len, page, uneven=False, tree=False):
    return {"name": name, "op": "prefix", "B": B, "groups": groups, "T": T, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "prefix": prefix, "own_len": own_len, "page": page, "uneven": uneven, "tree": tree}


def _rotary(kind="none", rotary=128, interleaved=False, theta=10000.0, factor=1.0):
    return {"kind": kind, "rotary": rotary, "interleaved": interleaved, "theta": theta, "factor": factor}


def listed():
    return [
        # four answers to one question, one token each: the smallest call, where latency counts
        _prefix("prefix_4x1_1000", 4, 1, 1, 32, 8, 128, 1008, 200, 16),
        # a serving batch behind one long system prompt, one token each
        _prefix("prefix_64x1_8192", 64, 1, 1, 64, 8, 128, 8192, 1000, 64),
        # blocks of 16 drafts behind four long documents
        _prefix("prefix_32x17_16384", 32, 4, 17, 64, 8, 128, 16384, 2000, 128),
        # small trees, narrow heads in groups of 6, uneven groups, odd lengths, every sequence in a buffer of its own
        _prefix("prefix_50x9_tree_d64", 50, 7, 9, 24, 4, 64, 4001, 777, 0, uneven=True, tree=True),
        # the queries and keys of one drafted tree far into a context, frequencies scaled by ramps
        {"name": "rope_1x17_tree", "op": "rope", "B": 1, "T": 17, "heads": 40, "extra": 8, "dim": 128, "far": 131072,
         "tree": True, **_rotary("yarn", 128, False, 10000.0, 4.0)},
        # the queries and keys of long prompts, half of each head rotated, interleaved
        {"name": "rope_16x4096_part", "op": "rope", "B": 16, "T": 4096, "heads": 72, "extra": 8, "dim": 128, "far": 1,
         "tree": False, **_rotary("none", 64, True, 500000.0)},
        # a decoding batch: one token each, its query rotated in the same call
        {"name": "append_256x1", "op": "append", "B": 256, "T": 1, "heads": 64, "kv_heads": 8, "dim": 128,
         "length": 1000, "page": 16, "shifted": True, **_rotary("wavelength", 128, False, 500000.0, 8.0)},
        # prompts of ragged lengths
        {"name": "append_8x4096", "op": "append", "B": 8, "T": 4096, "heads": 64, "kv_heads": 8, "dim": 128,
         "length": 1, "page": 64, "shifted": False, **_rotary()},
        # four requests of one token each, out of place
        {"name": "logits_4x1", "op": "logits", "B": 4, "T": 1, "V": 151936, "tree": False, "penalties": True,
         "bias": "none", "allowed": False, "inplace": False, "history": 1000},
        # a batch of drafted blocks, half of the requests bound by a grammar, in place
        {"name": "logits_128x17_grammar", "op": "logits", "B": 128, "T": 17, "V": 151936, "tree": False,
         "penalties": True, "bias": "shared", "allowed": True, "inplace": True, "history": 2000},
        # accepted paths of a batch of drafted trees
        {"name": "counts_128x17", "op": "counts", "B": 128, "N": 17, "V": 151936, "tree": True, "prompt": False},
        # long prompts of a batch
        {"name": "counts_32x32768", "op": "counts", "B": 32, "N": 32768, "V": 151936, "tree": False, "prompt": True},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rotary(rng, dim):
    kind = rng.choice(["none", "none", "linear", "ntk", "yarn", "wavelength"])
    return _rotary(kind, rng.choice([dim, dim // 2, dim // 4]), rng.random() < 0.5,
                   rng.choice([10000.0, 500000.0, 1000000.0]), 1.0 if kind == "none" else rng.choice([2.0, 4.0, 8.0]))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "prefix", "rope", "append", "logits", "counts"])
    if op == "prefix":
        kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        group = rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
        B, T = _logint(rng, 1, 128), _logint(rng, 1, 64)
        # no more query rows x keys than the largest, no more cached keys than fit comfortably
        most = min(32768, (32 * 17 * 64 * 18384) // (B * T * group * kv_heads), 1000000 // B)
        own_len = _logint(rng, 1, max(1, min(4000, most // 2)))
        case = _prefix("", B, rng.randint(1, min(B, 8)), T, kv_heads * group, kv_heads, dim,
                       _logint(rng, 16, max(16, most - own_len)), own_len, rng.choice([0, 16, 32, 64, 128, 256]),
                       rng.random() < 0.5, rng.random() < 0.4)
        del case["name"]
        return case
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 256])
        B, heads = _logint(rng, 1, 64), _logint(rng, 1, 80)
        T = _logint(rng, 1, max(1, min(8192, (16 * 4096 * 72 * 128) // (B * heads * dim))))
        return {"op": op, "B": B, "T": T, "heads": heads, "extra": rng.choice([0, 1, 8]), "dim": dim,
                "far": _logint(rng, 1, 1000000), "tree": T <= 128 and rng.random() < 0.5, **_draw_rotary(rng, dim)}
    if op == "append":
        kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        B = _logint(rng, 1, 256)
        T = _logint(rng, 1, max(1, min(4096, 8 * 4096 // B)))
        return {"op": op, "B": B, "T": T, "heads": kv_heads * rng.choice([0, 1, 2, 4, 7, 8]), "kv_heads": kv_heads,
                "dim": dim, "length": _logint(rng, 1, 4000), "page": rng.choice([0, 16, 32, 64, 128, 256]),
                "shifted": rng.random() < 0.5, **_draw_rotary(rng, dim)}
    V = _logint(rng, 1000, 151936)
    if op == "counts":
        tree = rng.random() < 0.5
        return {"op": op, "B": _logint(rng, 1, 128), "N": _logint(rng, 1, 128 if tree else 8192), "V": V, "tree": tree,
                "prompt": not tree and rng.random() < 0.5}
    B = _logint(rng, 1, 128)
    T = _logint(rng, 1, min(64, 2176 // B))
    return {"op": op, "B": B, "T": T, "V": V, "tree": rng.random() < 0.5, "penalties": rng.random() < 0.8,
            "bias": rng.choice(["none", "shared", "each"]), "allowed": rng.random() < 0.5,
            "inplace": rng.random() < 0.5, "history": _logint(rng, 1, 8000)}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _normal(gen, shape, std=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return x.normal_(0.0, std, generator=gen)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _tree(B, T, rng):
    """ancestors-or-self [B, T, T] of random trees whose nodes follow their parents, parents and depths."""
    sees, depth, parent = np.zeros((B, T, T), bool), np.zeros((B, T), np.int64), np.zeros((B, T), np.int64)
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


def _starts(case, rng):
    """First sequence of each group, and B."""
    B, G = case["B"], case["groups"]
    if case["uneven"]:
        cuts = np.sort(rng.choice(np.arange(1, B), G - 1, replace=False)) if G > 1 else np.zeros(0, np.int64)
    else:
        cuts = np.arange(1, G) * B // G
    return np.concatenate([[0], cuts, [B]]).astype(np.int32)


def _prepare_prefix(case, rng, gen, st):
    B, T, H, D, page = case["B"], case["T"], case["kv_heads"], case["dim"], case["page"]
    starts = _starts(case, rng)
    G = len(starts) - 1
    shared = rng.integers(case["prefix"] // 2, case["prefix"] + 1, G)
    shared[0] = case["prefix"]
    if page:
        shared = shared // page * page            # whole pages are shared
    group = np.repeat(np.arange(G), np.diff(starts))
    mine = rng.integers(case["own_len"] // 8, case["own_len"] + 1, B)
    mine[0] = case["own_len"]
    capacity = case["prefix"] + case["own_len"] + T
    st["starts"], st["shared"] = _i32(starts), _i32(shared)
    st["len"] = _i32(shared[group] + mine)
    st["host"] = {"starts": starts, "shared": shared, "len": shared[group] + mine}
    if page:
        per = -(-capacity // page)
        own_pages = -(-(case["own_len"] + T) // page) + 1
        pages = int((shared // page).sum()) + B * own_pages + 1
        ids = rng.permutation(pages)
        table, at = np.zeros((B, per), np.int64), 0
        for g in range(G):
            n = shared[g] // page
            table[starts[g]:starts[g + 1], :n] = ids[at:at + n]
            at += n
        for b in range(B):
            n = shared[group[b]] // page
            m = min(own_pages, per - n)
            table[b, n:n + m] = ids[at:at + m]
            at += m
        shape, st["table"] = (pages, page, H, D), _i32(table)
    else:
        shape, st["table"] = (B, capacity, H, D), None
    st["k"], st["v"] = _normal(gen, shape), _normal(gen, shape)
    st["k"][:, :: max(1, shape[1] // 2)] *= 2.0   # a few positions draw much more attention, as in trained models
    if not page:
        for g in range(G):
            for x in (st["k"], st["v"]):
                x[starts[g]:starts[g + 1], :shared[g]] = x[starts[g], :shared[g]].clone()
    qkv = _normal(gen, (B, T, case["heads"] + 2 * H, D))
    st["q"], st["k_new"], st["v_new"] = qkv.split([case["heads"], H, H], 2)
    st["mask"] = _mask_words(_tree(B, T, rng)[0]) if case["tree"] else None
    st["scale"] = 1.0 / math.sqrt(D)
    st["out"] = torch.empty((B, T, case["heads"], D), dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.empty((B, T, case["heads"]), dtype=torch.float32, device="cuda")


def _prepare_rope(case, rng, gen, st):
    B, T = case["B"], case["T"]
    x = _normal(gen, (B, T, case["heads"] + case["extra"], case["dim"]))
    st["x"] = x[:, :, :case["heads"]]              # queries and keys of a fused projection
    st["base"] = _i32(rng.integers(0, case["far"], B))
    st["depth"] = _i32(_tree(B, T, rng)[2]) if case["tree"] else None
    st["out"] = torch.empty((B, T, case["heads"], case["dim"]), dtype=torch.bfloat16, device="cuda")


def _prepare_append(case, rng, gen, st):
    B, T, H, D, page, heads = (case[k] for k in ("B", "T", "kv_heads", "dim", "page", "heads"))
    lens = rng.integers(case["length"] // 2, case["length"] + 1, B)
    capacity = case["length"] + T
    if page:
        per = -(-capacity // page)
        shape = (B * per + 3, page, H, D)
        st["table"] = _i32(rng.permutation(B * per + 3)[:B * per].reshape(B, per))
    else:
        shape, st["table"] = (B, capacity, H, D), None
    st["k"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    st["v"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    qkv = _normal(gen, (B, T, heads + 2 * H, D))
    st["q"], st["k_new"], st["v_new"] = qkv.split([heads, H, H], 2)
    st["len"] = _i32(lens)
    st["count"] = _i32(rng.integers((T + 1) // 2, T + 1, B))
    # sequences that were shortened before hold fewer positions than they have seen
    st["position"] = _i32(lens + rng.integers(0, 100000, B)) if case["shifted"] else None
    st["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    st["q_out"] = torch.zeros((B, T, heads, D), dtype=torch.bfloat16, device="cuda") if heads else None


def _zipf(rng, shape, V):
    """Token ids, common ones far more often than rare ones, spread over the vocabulary."""
    rank = np.floor(np.exp(rng.random(shape) * math.log(V))).astype(np.int64) - 1
    return (np.clip(rank, 0, V - 1) * 7919 + 13) % V


def _padded(n):
    return -(-n // 8) * 8


def _prepare_logits(case, rng, gen, st):
    B, T, V = case["B"], case["T"], case["V"]
    st["logits"] = _normal(gen, (B, T, _padded(V)), 3.0)[..., :V]
    st["tokens"] = st["mask"] = st["counts"] = st["bias"] = st["allowed"] = None
    st["repetition"] = st["frequency"] = st["presence"] = None
    if case["penalties"]:
        counts = torch.zeros((B, _padded(V)), dtype=torch.int32, device="cuda")
        emitted = torch.from_numpy(_zipf(rng, (B, case["history"]), V)).cuda()
        prompt = torch.from_numpy(_zipf(rng, (B, case["history"]), V)).cuda()
        counts.scatter_add_(1, emitted, torch.ones_like(emitted, dtype=torch.int32))
        flags = torch.zeros_like(counts).scatter_(1, prompt, -2 ** 31)
        st["counts"] = (counts | flags)[:, :V]
        st["tokens"] = _i32(_zipf(rng, (B, T), V))
        if case["tree"]:
            st["mask"] = _mask_words(_tree(B, T, rng)[0])
        for name, lo, hi in (("repetition", 1.0, 1.3), ("frequency", 0.0, 0.5), ("presence", 0.0, 0.5)):
            st[name] = torch.from_numpy(rng.uniform(lo, hi, B).astype(np.float32)).cuda()
    if case["bias"] != "none":
        rows = 1 if case["bias"] == "shared" else B
        bias = torch.zeros((rows, _padded(V)), dtype=torch.float32, device="cuda")
        at = torch.from_numpy(rng.integers(0, V, (rows, min(V, 300)))).cuda()
        bias.scatter_(1, at, torch.from_numpy(rng.normal(0.0, 5.0, tuple(at.shape)).astype(np.float32)).cuda())
        st["bias"] = bias[:, :V]
    if case["allowed"]:
        words = (V + 31) // 32
        allowed = torch.full((B, T, words), -1, dtype=torch.int32, device="cuda")
        for b in range(0, B, 2):                   # every second request follows a grammar: some hundred tokens a node
            bits = np.zeros((T, words * 32), np.uint8)
            bits[np.arange(T)[:, None], rng.integers(0, V, (T, 200))] = 1
            allowed[b] = torch.from_numpy(np.packbits(bits, axis=-1, bitorder="little").view(np.int32)).cuda()
        st["allowed"] = allowed
    st["out"] = st["logits"] if case["inplace"] else \
        torch.zeros((B, T, _padded(V)), dtype=torch.bfloat16, device="cuda")[..., :V]


def _prepare_counts(case, rng, gen, st):
    B, N, V = case["B"], case["N"], case["V"]
    st["tokens"] = _i32(_zipf(rng, (B, N), V))
    st["counts"] = torch.zeros((B, _padded(V)), dtype=torch.int32, device="cuda")[:, :V]
    st["path"], count = None, rng.integers((N + 1) // 2, N + 1, B)
    if case["tree"]:
        _, parent, depth = _tree(B, N, rng)
        path = np.full((B, N), -1, np.int32)
        for b in range(B):
            node = int(rng.integers(0, N))
            count[b] = depth[b, node] + 1
            for i in range(int(count[b]) - 1, -1, -1):
                path[b, i], node = node, parent[b, node]
        st["path"] = _i32(path)
    st["count"] = _i32(count)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    {"prefix": _prepare_prefix, "rope": _prepare_rope, "append": _prepare_append, "logits": _prepare_logits,
     "counts": _prepare_counts}[op](case, rng, gen, st)
    if own:
        from draft_selection_dflash2_gb300 import api
        h = st["handle"] = _handle(api)
        if op in ("prefix", "append"):
            st["cache"] = api.KVCache(st["k"], st["v"], st["table"])
        if op == "prefix":
            n = api.prefix_attention_workspace(h, case["B"], case["T"], case["heads"], case["kv_heads"], case["dim"])
            st["workspace"] = torch.empty(max(int(n), 256), dtype=torch.uint8, device="cuda")
        if op in ("rope", "append"):
            st["rope"] = api.Rope(case["rotary"], theta=case["theta"], interleaved=case["interleaved"],
                                  scaling=_scaling(case))
    return st


_handles = {}


def _handle(api):
    device = torch.cuda.current_device()
    if device not in _handles:
        _handles[device] = api.Handle(device)
    return _handles[device]


def _scaling(case):
    """The scaled frequencies of longer contexts than trained on, as Rope takes them."""
    kind, factor = case["kind"], case["factor"]
    return {"none": None, "linear": {"kind": "linear", "factor": factor}, "ntk": {"kind": "ntk", "factor": factor},
            "yarn": {"kind": "yarn", "factor": factor, "original": 4096, "fast": 32.0, "slow": 1.0},
            "wavelength": {"kind": "wavelength", "factor": factor, "original": 8192, "low": 1.0, "high": 4.0}}[kind]


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------
def _positions_of(x, table, b0, b1, first, n):
    """Positions first .. first + n - 1 of sequences b0 .. b1 - 1 (clamped at the capacity): [b1 - b0, n, kv_heads, dim]."""
    page = x.shape[1]
    capacity = page if table is None else page * table.shape[1]
    at = (first + torch.arange(n, device="cuda")).clamp_(max=capacity - 1)
    if table is None:
        return x[b0:b1, at]
    return x[table[b0:b1][:, at // page].long(), at % page]


def _sees_plain(mask, T):
    node = torch.arange(T, device="cuda")
    if mask is None:
        return (node[None] <= node[:, None])[None]
    return ((mask[:, :, node // 64] >> (node % 64)) & 1).bool()


def _prefix_plain(st):
    c = st["case"]
    B, T, H, D, n = c["B"], c["T"], c["kv_heads"], c["dim"], c["own_len"]
    starts, shared = st["host"]["starts"], st["host"]["shared"]
    out = torch.empty((B, T, c["heads"], D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, T, c["heads"]), dtype=torch.float32, device="cuda")
    sees = _sees_plain(st["mask"], T)
    for g, P in enumerate(shared):
        b0, b1, P = int(starts[g]), int(starts[g + 1]), int(P)
        S = b1 - b0
        q = st["q"][b0:b1].float().reshape(S, T, H, -1, D)
        keys = _positions_of(st["k"], st["table"], b0, b0 + 1, 0, P)[0].float()
        s_shared = torch.einsum("bthgd,shd->bhgts", q, keys)
        mine = _positions_of(st["k"], st["table"], b0, b1, P, n).float()
        past = P + torch.arange(n, device="cuda")[None] >= st["len"][b0:b1, None]
        s_own = torch.einsum("bthgd,bshd->bhgts", q, mine).masked_fill_(past[:, None, None, None], -math.inf)
        s_new = torch.einsum("bthgd,bshd->bhgts", q, st["k_new"][b0:b1].float())
        seen = sees[b0:b1] if st["mask"] is not None else sees
        s_new = s_new.masked_fill(~seen[:, None, None], -math.inf)
        s = torch.cat([s_shared, s_own, s_new], -1).mul_(st["scale"])
        top = s.amax(-1, keepdim=True)
        p = s.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.einsum("bhgts,shd->bhgtd", p[..., :P], _positions_of(st["v"], st["table"], b0, b0 + 1, 0, P)[0].float())
        values = _positions_of(st["v"], st["table"], b0, b1, P, n).float().masked_fill_(past[:, :, None, None], 0.0)
        o += torch.einsum("bhgts,bshd->bhgtd", p[..., P:P + n], values)
        o += torch.einsum("bhgts,bshd->bhgtd", p[..., P + n:], st["v_new"][b0:b1].float())
        out[b0:b1] = (o / total).permute(0, 3, 1, 2, 4).reshape(S, T, -1, D)
        lse[b0:b1] = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(S, T, -1)
    return {"out": out, "lse": lse}


def _frequencies(case):
    """Radians per position of each rotated pair (64 bits), and the factor of cos and sin."""
    rd, theta, s = case["rotary"], case["theta"], _scaling(case)
    i = torch.arange(rd // 2, dtype=torch.float64, device="cuda")
    if s is None:
        return theta ** (-2.0 * i / rd), 1.0
    if s["kind"] == "ntk":
        return (theta * s["factor"] ** (rd / (rd - 2.0))) ** (-2.0 * i / rd), 1.0
    f = theta ** (-2.0 * i / rd)
    if s["kind"] == "linear":
        return f / s["factor"], 1.0
    if s["kind"] == "yarn":
        at = [rd * math.log(s["original"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))
              for turns in (s["fast"], s["slow"])]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp_(0.0, 1.0)
        return f / s["factor"] * ramp + f * (1.0 - ramp), 0.1 * math.log(s["factor"]) + 1.0
    smooth = (s["original"] * f / (2.0 * math.pi) - s["low"]) / (s["high"] - s["low"])
    smooth = smooth.clamp_(0.0, 1.0)
    return f / s["factor"] * (1.0 - smooth) + f * smooth, 1.0


def _rotate_plain(case, x, position):
    """x [B, T, heads, dim] rotated by its positions [B, T], in 32 bits."""
    rd, half = case["rotary"], case["rotary"] // 2
    f, factor = _frequencies(case)
    angle = position[:, :, None].double() * f
    cos, sin = (angle.cos() * factor).float()[:, :, None], (angle.sin() * factor).float()[:, :, None]
    x = x.float()
    y = x.clone()
    if case["interleaved"]:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y[..., 0:rd:2], y[..., 1:rd:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:rd]
        y[..., :half], y[..., half:rd] = a * cos - b * sin, b * cos + a * sin
    return y


def _rope_positions(st):
    T = st["case"]["T"]
    depth = torch.arange(T, device="cuda")[None] if st["depth"] is None else st["depth"]
    return st["base"][:, None] + depth


def _rope_plain(st):
    return {"out": _rotate_plain(st["case"], st["x"], _rope_positions(st)).to(torch.bfloat16)}


def _append_plain(st):
    c = st["case"]
    B, T = c["B"], c["T"]
    i = torch.arange(T, device="cuda")[None].expand(B, T)
    taken = i < st["count"][:, None]
    position = (st["len"] if st["position"] is None else st["position"])[:, None] + i
    at = (st["len"][:, None] + i).long()
    if st["table"] is None:
        page, off = torch.arange(B, device="cuda")[:, None].expand(B, T), at
    else:
        size = st["k"].shape[1]
        page, off = torch.gather(st["table"].long(), 1, at // size), at % size
    keys = _rotate_plain(c, st["k_new"], position).to(torch.bfloat16)
    page, off = page[taken], off[taken]
    st["k"][page, off] = keys[taken]
    st["v"][page, off] = st["v_new"][taken]
    new_len = st["len"] + st["count"]
    if st["q_out"] is not None:
        q = _rotate_plain(c, st["q"], position).to(torch.bfloat16)
        st["q_out"].copy_(torch.where(taken[:, :, None, None], q, st["q_out"]))
        return {"k": st["k"], "v": st["v"], "q": st["q_out"], "new_len": new_len}
    return {"k": st["k"], "v": st["v"], "new_len": new_len}


def _logits_plain(st):
    c = st["case"]
    B, T, V = c["B"], c["T"], c["V"]
    x = st["logits"].float()
    if st["counts"] is not None:
        sees = _sees_plain(st["mask"], T).expand(B, T, T)
        n = (st["counts"] & 0x7FFFFFFF)[:, None].repeat(1, T, 1)
        n.scatter_add_(2, st["tokens"].long()[:, None].expand(B, T, T), sees.int())
        known = (n > 0) | (st["counts"] < 0)[:, None]
        r = st["repetition"][:, None, None]
        x = torch.where(known, torch.where(x > 0.0, x / r, x * r), x)
        x -= n * st["frequency"][:, None, None]
        x -= (n > 0) * st["presence"][:, None, None]
    if st["bias"] is not None:
        x += st["bias"][:, None]
    if st["allowed"] is not None:
        at = torch.arange(V, device="cuda")
        x.masked_fill_(((st["allowed"][:, :, at // 32] >> (at % 32)) & 1) == 0, -math.inf)
    return {"logits": st["out"].copy_(x)}


def _counts_plain(st):
    c = st["case"]
    B, N = c["B"], c["N"]
    taken = torch.arange(N, device="cuda")[None] < st["count"][:, None]
    tokens = st["tokens"].long()
    if st["path"] is not None:
        tokens = torch.gather(tokens, 1, st["path"].clamp(min=0).long())
    if c["prompt"]:
        row = torch.arange(B, device="cuda")[:, None].expand(B, N)[taken]
        st["counts"][row, tokens[taken]] = st["counts"][row, tokens[taken]] | -2 ** 31
    else:
        st["counts"].scatter_add_(1, tokens, taken.int())
    return {"counts": st["counts"]}


def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        return {"prefix": _prefix_plain, "rope": _rope_plain, "append": _append_plain, "logits": _logits_plain,
                "counts": _counts_plain}[op](st)
    from draft_selection_dflash2_gb300 import api
    h = st["handle"]
    if op == "prefix":
        out, lse = api.prefix_attention(h, st["q"], st["cache"], st["len"], st["shared"], st["starts"], st["k_new"],
                                        st["v_new"], tree_mask=st["mask"], scale=st["scale"], out=st["out"],
                                        lse=st["lse"], workspace=st["workspace"])
        return {"out": out, "lse": lse}
    if op == "rope":
        return {"out": api.rope(h, st["x"], st["rope"], base=st["base"], depth=st["depth"], out=st["out"])}
    if op == "append":
        new_len, q = api.cache_append(h, st["k_new"], st["v_new"], st["cache"], st["len"], rope=st["rope"],
                                      count=st["count"], position=st["position"],
                                      q=None if st["q_out"] is None else st["q"], q_out=st["q_out"],
                                      new_len=st["new_len"])
        got = {"k": st["k"], "v": st["v"], "new_len": new_len}
        if q is not None:
            got["q"] = q
        return got
    if op == "logits":
        return {"logits": api.logits_adjust(h, st["logits"], counts=st["counts"], tokens=st["tokens"],
                                            tree_mask=st["mask"], repetition=st["repetition"],
                                            frequency=st["frequency"], presence=st["presence"], bias=st["bias"],
                                            allowed=st["allowed"], out=st["out"])}
    return {"counts": api.token_counts(h, st["tokens"], st["counts"], count=st["count"], path=st["path"],
                                       prompt=c["prompt"])}


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    op, B = case["op"], case["B"]
    if op == "prefix":
        T, H, D = case["T"], case["kv_heads"], case["dim"]
        row = 2.0 * D                                                   # bytes of one bf16 row
        G = case["groups"]
        shared = case["prefix"] * (0.25 / G + 0.75)                     # the first as long as it gets, others from half
        mine = case["own_len"] * 9.0 / 16.0
        q = B * T * case["heads"]
        seen = shared + mine + (T / 4.0 if case["tree"] else (T + 1) / 2.0)
        return {"bytes": 2 * q * row + 4 * q + 2 * H * (G * shared + B * (mine + T)) * row, "flops": 4.0 * q * seen * D}
    if op == "rope":
        rows = B * case["T"] * case["heads"]
        return {"bytes": 4.0 * rows * case["dim"] + 4 * B, "flops": 3.0 * rows * case["rotary"]}
    if op == "append":
        tokens = 0.75 * B * case["T"] if case["T"] > 1 else B
        rows = case["heads"] + 2 * case["kv_heads"]
        return {"bytes": 4.0 * tokens * rows * case["dim"] + 16 * B,
                "flops": 3.0 * tokens * (case["heads"] + case["kv_heads"]) * case["rotary"]}
    V = case["V"]
    if op == "counts":
        tokens = B * (min(case["N"], 8) if case["tree"] else 0.75 * case["N"])
        return {"bytes": 12.0 * tokens + 4 * B, "flops": 0}
    T = case["T"]
    rows = float(B * T)
    most = {"none": 0.0, "shared": 4.0 * V, "each": 4.0 * B * V}[case["bias"]]
    most += 4.0 * B * V if case["penalties"] else 0.0
    most += rows * V / 8.0 if case["allowed"] else 0.0
    if case["inplace"]:            # what stays as it is need not be read; what is not allowed is only written
        touched = min(V, case["history"]) * rows if case["penalties"] else 0.0
        return {"bytes": most + (rows * V if case["allowed"] else 0.0) + 2.0 * touched, "flops": rows * V}
    return {"bytes": most + 4.0 * rows * V, "flops": rows * V}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _exact_prefix(case, st):
    B, T, H, D = case["B"], case["T"], case["kv_heads"], case["dim"]
    if 4.0 * B * T * case["heads"] * (case["prefix"] + case["own_len"] + T) * D > 4e12:
        return None
    G = case["heads"] // H
    out = torch.empty((B, T, case["heads"], D), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, T, case["heads"]), dtype=torch.float64, device="cuda")
    words = None if st["mask"] is None else st["mask"].cpu().numpy().view(np.uint64)
    page = st["k"].shape[1]
    for b in range(B):
        n = int(st["host"]["len"][b])
        hidden = torch.ones((T, T), dtype=torch.bool, device="cuda").triu(1)
        if words is not None:
            hidden = torch.tensor([[not (int(words[b, t, s // 64]) >> (s % 64)) & 1 for s in range(T)] for t in range(T)],
                                  dtype=torch.bool, device="cuda")
        both = []
        for pool, new in ((st["k"], st["k_new"]), (st["v"], st["v_new"])):
            cached = pool[b] if st["table"] is None else pool[st["table"][b, :-(-n // page)].long()].flatten(0, 1)
            both.append(torch.cat([cached[:n], new[b]]).double())
        q = st["q"][b].double().view(T, H, G, D).permute(1, 2, 0, 3).reshape(H, G * T, D)
        z = (q @ both[0].permute(1, 2, 0) * st["scale"]).view(H, G, T, n + T)
        z[..., n:].masked_fill_(hidden, -math.inf)
        lse[b] = torch.logsumexp(z, -1).permute(2, 0, 1).reshape(T, -1)
        o = torch.softmax(z, -1).view(H, G * T, n + T) @ both[1].permute(1, 0, 2)
        out[b] = o.view(H, G, T, D).permute(2, 0, 1, 3).reshape(T, -1, D)
    return {"out": out, "lse": lse}


def _angle_rate(case, i):
    """Radians per position of pair i."""
    rd, theta, kind, factor = case["rotary"], case["theta"], case["kind"], case["factor"]
    if kind == "ntk":
        return (theta * factor ** (rd / (rd - 2.0))) ** (-2.0 * i / rd)
    rate = theta ** (-2.0 * i / rd)
    if kind == "linear":
        return rate / factor
    if kind == "yarn":
        def index(turns):          # of the pair that turns so often over the original context
            return rd * math.log(4096 / (2.0 * math.pi * turns)) / (2.0 * math.log(theta))
        first, last = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), rd - 1)
        part = min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
        return rate * (part / factor + 1.0 - part)
    if kind == "wavelength":
        wave = 2.0 * math.pi / rate
        if wave > 8192 / 1.0:
            return rate / factor
        if wave < 8192 / 4.0:
            return rate
        part = (8192 / wave - 1.0) / (4.0 - 1.0)
        return (1.0 - part) * rate / factor + part * rate
    return rate


def _exact_rotation(case, x, position):
    """Each pair as a complex number times e^(i angle)."""
    rd = case["rotary"]
    rates = torch.tensor([_angle_rate(case, i) for i in range(rd // 2)], dtype=torch.float64, device="cuda")
    size = 0.1 * math.log(case["factor"]) + 1.0 if case["kind"] == "yarn" else 1.0
    turn = torch.polar(torch.full((), size, dtype=torch.float64, device="cuda").expand(*position.shape, rd // 2).contiguous(),
                       position.double()[..., None] * rates)[:, :, None]
    y = x.double()
    if case["interleaved"]:
        y[..., :rd] = torch.view_as_real(torch.complex(y[..., 0:rd:2], y[..., 1:rd:2]) * turn).flatten(-2)
    else:
        z = torch.complex(y[..., :rd // 2], y[..., rd // 2:rd]) * turn
        y[..., :rd] = torch.cat([z.real, z.imag], -1)
    return y


def exact(case, seed):
    op = case["op"]
    if op == "counts":
        return None                # whole numbers
    st = prepare(case, seed)
    if op == "prefix":
        return _exact_prefix(case, st)
    if op == "rope":
        return {"out": torch.cat([_exact_rotation(case, x, p) for x, p in
                                  zip(st["x"].split(1), _rope_positions(st).split(1))])}
    B, T = case["B"], case["T"]
    if op == "append":
        k, q = st["k"].double(), None if st["q_out"] is None else st["q_out"].double()
        size = st["k"].shape[1]
        for b in range(B):
            n, m = int(st["len"][b]), int(st["count"][b])
            p = (n if st["position"] is None else int(st["position"][b])) + torch.arange(m, device="cuda")
            at = n + torch.arange(m, device="cuda")
            page = torch.full_like(at, b) if st["table"] is None else st["table"][b, at // size].long()
            k[page, at % size if st["table"] is not None else at] = _exact_rotation(case, st["k_new"][b:b + 1, :m], p[None])[0]
            if q is not None:
                q[b, :m] = _exact_rotation(case, st["q"][b:b + 1, :m], p[None])[0]
        got = {"k": k, "v": None, "new_len": None}
        if q is not None:
            got["q"] = q
        return got
    words = None if st["mask"] is None else st["mask"].cpu().numpy().view(np.uint64)
    want = torch.empty((B, T, case["V"]), dtype=torch.float64, device="cuda")
    node = np.arange(T)
    for b in range(B):
        x = st["logits"][b].double()
        if st["counts"] is not None:
            emitted = (st["counts"][b].long() & 0x7FFFFFFF).double()
            prompt = st["counts"][b] < 0
            tokens = st["tokens"][b].cpu().numpy()
            for t in range(T):
                seen = node <= t if words is None else np.array([int(words[b, t, s // 64]) >> (s % 64) & 1 for s in node], bool)
                n = emitted + torch.from_numpy(np.bincount(tokens[seen], minlength=case["V"])).cuda()
                again = prompt | (n > 0)
                r = float(st["repetition"][b])
                x[t] = torch.where(again, torch.where(x[t] > 0, x[t] / r, x[t] * r), x[t])
                x[t] -= float(st["frequency"][b]) * n + float(st["presence"][b]) * (n > 0)
        if st["bias"] is not None:
            x += st["bias"][b if st["bias"].shape[0] > 1 else 0].double()
        if st["allowed"] is not None:
            bit = (st["allowed"][b][:, :, None] >> torch.arange(32, device="cuda")) & 1
            x[bit.flatten(1)[:, :case["V"]] == 0] = -math.inf
        want[b] = x
    return {"logits": want}
