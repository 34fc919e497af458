"""Runs one stage of the draft-block head on seeded synthetic inputs of the
full-cycle workload's shape (B sequences, L=16, V=151936, d=5120), a few
times, so that a profiler (ncu) can capture that stage's kernels alone.

  python -m draft_selection_dflash2_gb300.profile_stage --stage topk [--B 128] [--reps 3]

Stages: topk, pairs (gate + pair scores), walk0, walk1, conv (one application),
verify0, verify1, lmhead (M=1024 hidden rows against the full vocabulary),
lmhead_gate (the same with the context gate folded in), viterbi (the exact
best-path walk on N(0, 4) scores of B sequences), eval (the Table 1 selector
evaluation of B sequences of 7 positions with uniform candidate ids and the
true token in slot 0 of 80% of the rows), proj (projection-form pair scores
of B sequences: A, B projected from an N(0, 1) [V, d] embedding) and gemm_conv
(the conv fused into an output projection with K = d).  The cache operators have
shapes of their own (64 query heads over 8 kv heads of 128, N(0, 1) inputs, pages
of 64): attention (2 sequences of 131072 positions, one token each),
attention_block (64 blocks of 17 over lengths of 1500 to 12000), attention_tree (8
trees of 64 nodes over 16384 positions), commit (256 paths of 1 to 64 nodes),
scores (16 blocks of 17, 1 to 17 accepted, over lengths of 4096 to 32768) and
evict (16 sequences of 4096 to 32768 positions to 8001).  So have the operators around
them: prefix (64 sequences of one token behind 8192 shared positions and 125 to 1000 of their
own), prefix_block (32 blocks of 17 in four groups behind 16384 shared and 250 to 2000 own
ones), rope (72 heads of 16 x 4096 tokens, 64 of 128 elements rotated in neighbouring pairs),
append (8 prompts of 2048 to 4096 tokens, queries rotated along), logits (128 blocks of 17 over
V = 151936 with penalties, 300 biases and, for every second sequence, about 200 allowed tokens a
node) and counts (32 prompts of 16384 to 32768 tokens).
"""
import argparse
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from draft_selection_dflash2_gb300 import api, synth  # noqa: E402

L, V, D, R, K = 16, 151936, 5120, 256, 16


def bf(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.bfloat16)


def cache_stage(torch, h, rng, stage):
    """One cache operator's call (see the module's text for its shape)."""
    B, T, n = {"attention": (2, 1, 131072), "attention_block": (64, 17, 12000), "attention_tree": (8, 64, 16384),
               "commit": (256, 64, 1000), "scores": (16, 17, 32768), "evict": (16, 0, 32768)}[stage]
    heads, H, dim, page, keep = 64, 8, 128, 64, 8001
    g = torch.Generator(device="cuda")
    g.manual_seed(8)

    def randn(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)

    def pool(positions):
        pages = -(-positions // page)
        table = torch.from_numpy(rng.permutation(B * pages).reshape(B, pages).astype(np.int32)).cuda()
        return api.KVCache(randn(B * pages, page, H, dim), randn(B * pages, page, H, dim), table)

    cache = pool(n + T)
    ragged = stage in ("attention_block", "scores", "evict")
    lens = torch.from_numpy((rng.integers(n // 8, n + 1, B) if ragged else np.full(B, n)).astype(np.int32)).cuda()
    if stage == "evict":
        dst = pool(keep)
        scores = torch.rand((B, H, n), generator=g, device="cuda")
        return lambda: api.cache_evict(h, scores, cache, lens, dst, keep, 500)
    count = torch.from_numpy(rng.integers(1, T + 1, B).astype(np.int32)).cuda()
    q, k, v = randn(B, T, heads, dim), randn(B, T, H, dim), randn(B, T, H, dim)
    scores = torch.zeros((B, H, n + T), device="cuda")
    if stage == "commit":
        return lambda: api.cache_commit(h, k, v, cache, lens, count, scores=scores)
    if stage == "scores":
        lse = torch.full((B, T, heads), 10.0, device="cuda")
        return lambda: api.cache_scores(h, q, lse, cache, lens, scores, count)
    mask = None
    if stage == "attention_tree":
        # node t's parent is one of the six before it
        sees = np.zeros((B, T, T), bool)
        for t in range(T):
            if t:
                parent = t - 1 - np.minimum(rng.integers(0, 6, B), t - 1)
                sees[:, t] = sees[np.arange(B), parent]
            sees[:, t, t] = True
        mask = torch.from_numpy(np.packbits(sees, axis=-1, bitorder="little").view(np.int64).copy()).cuda()
    ws = torch.empty(api.tree_attention_workspace(h, B, T, heads, H, dim), dtype=torch.uint8, device="cuda")
    return lambda: api.tree_attention(h, q, cache, lens, k, v, tree_mask=mask, workspace=ws)


def serve_stage(torch, h, rng, stage):
    """One call of an operator around the cache (see the module's text for its shape)."""
    heads, H, dim, page = 64, 8, 128, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def randn(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)

    def i32(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def pool(table):
        shape = (int(table.max()) + 1, page, H, dim)
        return api.KVCache(randn(*shape), randn(*shape), i32(table))

    if stage in ("prefix", "prefix_block"):
        B, T, groups, shared, own = {"prefix": (64, 1, 1, 8192, 1000), "prefix_block": (32, 17, 4, 16384, 2000)}[stage]
        first, mine = shared // page, -(-(own + T) // page)
        group = np.arange(B) * groups // B
        table = np.concatenate([group[:, None] * first + np.arange(first),
                                groups * first + np.arange(B * mine).reshape(B, mine)], axis=1)
        cache, starts = pool(table), i32(np.arange(groups + 1) * B // groups)
        lens, prefix = i32(shared + rng.integers(own // 8, own + 1, B)), i32(np.full(groups, shared))
        q, k, v = randn(B, T, heads, dim), randn(B, T, H, dim), randn(B, T, H, dim)
        ws = torch.empty(api.prefix_attention_workspace(h, B, T, heads, H, dim), dtype=torch.uint8, device="cuda")
        return lambda: api.prefix_attention(h, q, cache, lens, prefix, starts, k, v, workspace=ws)
    if stage == "rope":
        x = randn(16, 4096, heads + 16, dim)[:, :, :heads + 8]
        out, r = torch.empty(x.shape, dtype=x.dtype, device="cuda"), api.Rope(64, theta=500000.0, interleaved=True)
        return lambda: api.rope(h, x, r, out=out)
    if stage == "append":
        B, T = 8, 4096
        cache, count = pool(np.arange(B * T // page).reshape(B, -1)), i32(rng.integers(T // 2, T + 1, B))
        q, k, v = randn(B, T, heads + 2 * H, dim).split([heads, H, H], 2)
        out, lens, r = torch.zeros((B, T, heads, dim), dtype=q.dtype, device="cuda"), i32(np.zeros(B)), api.Rope(dim)
        return lambda: api.cache_append(h, k, v, cache, lens, r, count=count, q=q, q_out=out)
    B, N = (128, 17) if stage == "logits" else (32, 32768)
    tokens, counts = i32(rng.integers(0, V, (B, N))), torch.zeros((B, V), dtype=torch.int32, device="cuda")
    if stage == "counts":
        count = i32(rng.integers(N // 2, N + 1, B))
        return lambda: api.token_counts(h, tokens, counts, count, prompt=True)
    api.token_counts(h, i32(rng.integers(0, V, (B, 2000))), counts)
    api.token_counts(h, i32(rng.integers(0, V, (B, 2000))), counts, prompt=True)
    logits, bias = randn(B, N, V), torch.zeros((1, V), device="cuda")
    bias[0, torch.from_numpy(rng.permutation(V)[:300]).cuda()] = 1.5
    allowed = np.full((B, N, -(-V // 32)), -1, np.int32)
    for b in range(0, B, 2):
        bits = np.zeros((N, allowed.shape[2] * 32), np.uint8)
        bits[np.arange(N)[:, None], rng.integers(0, V, (N, 200))] = 1
        allowed[b] = np.packbits(bits, axis=-1, bitorder="little").view(np.int32)
    allowed = i32(allowed)
    factor = [torch.full((B,), x, device="cuda") for x in (1.1, 0.2, 0.2)]
    return lambda: api.logits_adjust(h, logits, counts, tokens, None, *factor, bias, allowed, out=logits)


def main():
    import torch

    ap = argparse.ArgumentParser()
    ap.add_argument("--stage", required=True,
                    choices=["topk", "pairs", "walk0", "walk1", "conv", "verify0", "verify1", "lmhead",
                             "lmhead_gate", "viterbi", "eval", "proj", "gemm_conv", "attention", "attention_block",
                             "attention_tree", "commit", "scores", "evict", "prefix", "prefix_block", "rope", "append",
                             "logits", "counts"])
    ap.add_argument("--B", type=int, default=128)
    ap.add_argument("--reps", type=int, default=3)
    args = ap.parse_args()
    torch.cuda.set_device(0)
    B = args.B
    h = api.Handle(0)
    rng = np.random.default_rng(0)
    if args.stage in ("attention", "attention_block", "attention_tree", "commit", "scores", "evict"):
        run = cache_stage(torch, h, rng, args.stage)
    elif args.stage in ("prefix", "prefix_block", "rope", "append", "logits", "counts"):
        run = serve_stage(torch, h, rng, args.stage)
    elif args.stage == "topk":
        U = bf(torch, synth.logits_planted(rng, B * L, V))
        run = lambda: api.topk(h, U)  # noqa: E731
    elif args.stage in ("pairs", "walk0", "walk1"):
        U = bf(torch, synth.logits_planted(rng, B * L, V))
        vals, idx = api.topk(h, U)
        del U
        hs = bf(torch, synth.normal_bits(1, (B, L, D)))
        W_H = bf(torch, synth.normal_bits(2, (R, D), std=0.02))
        A = bf(torch, synth.normal_bits(3, (V, R), std=0.02))
        Bt = bf(torch, synth.normal_bits(4, (V, R), std=0.02))
        lv = torch.from_numpy(rng.integers(0, V, B).astype(np.int32)).cuda()
        ci, cv = idx.view(B, L, K), vals.view(B, L, K)
        if args.stage == "pairs":
            run = lambda: api.pair_scores(h, ci, cv, lv, hs, W_H, None, A, Bt)  # noqa: E731
        else:
            S, _ = api.pair_scores(h, ci, cv, lv, hs, W_H, None, A, Bt)
            T = 0.0 if args.stage == "walk0" else 1.0
            run = lambda: api.walk(h, S, ci, temperature=T, seed=1)  # noqa: E731
    elif args.stage == "conv":
        x = bf(torch, synth.normal_bits(1, (B, L, D)))
        xp = bf(torch, synth.normal_bits(2, (B, D)))
        k0, k1, W_c = (bf(torch, a) for a in synth.conv_layer_params(3, D))
        y = torch.empty((B, L, D), dtype=torch.bfloat16, device="cuda")
        cws = torch.empty(api.conv2tap_workspace(h, B, L, D), dtype=torch.uint8, device="cuda")
        run = lambda: api.conv2tap(h, x, xp, k0, k1, W_c, y=y, workspace=cws)  # noqa: E731
    elif args.stage in ("verify0", "verify1"):
        T = 0.0 if args.stage == "verify0" else 1.0
        tok = rng.integers(0, V, (B, L)).astype(np.int32)
        ci = np.concatenate([tok[..., None], rng.integers(0, V, (B, L, K - 1))], axis=-1).astype(np.int32)
        slot = np.zeros((B, L), np.int32)
        q = np.full((B, L, K), 1.0 / K, np.float32)
        target = bf(torch, synth.target_planted(5, tok, V, agree=0.85, plant=8.0))
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        tok_d, slot_d, q_d, ci_d = dev(tok), dev(slot), dev(q), dev(ci)
        ws = torch.empty(api.verify_workspace(h, B, L, V), dtype=torch.uint8, device="cuda")
        run = lambda: api.verify(h, target, tok_d, slot_d, q_d, ci_d, temperature=T, seed=1, workspace=ws)  # noqa: E731
    elif args.stage == "viterbi":
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        S = torch.randn((B, L, K, K), generator=g, device="cuda") * 2
        ci = torch.randint(0, V, (B, L, K), generator=g, device="cuda", dtype=torch.int32)
        run = lambda: api.walk_viterbi(h, S, ci)  # noqa: E731
    elif args.stage == "eval":
        g = torch.Generator(device="cuda")
        g.manual_seed(6)
        Le = 7
        gt = torch.randint(0, V, (B, Le), generator=g, device="cuda", dtype=torch.int32)
        cand = torch.randint(0, V, (B, Le, K), generator=g, device="cuda", dtype=torch.int32)
        hit = torch.rand((B, Le), generator=g, device="cuda") < 0.8
        cand[:, :, 0] = torch.where(hit, gt, cand[:, :, 0])
        run = lambda: api.selector_eval(h, gt, cand)  # noqa: E731
    elif args.stage == "gemm_conv":
        A = bf(torch, synth.normal_bits(1, (B, L, D)))
        Wp = bf(torch, synth.normal_bits(2, (D, D), std=D ** -0.5))
        hs = bf(torch, synth.normal_bits(3, (B, L, D)))
        xp = bf(torch, synth.normal_bits(4, (B, D)))
        k0, k1, W_c = (bf(torch, a) for a in synth.conv_layer_params(5, D))
        run = lambda: api.gemm_conv2tap(h, A, Wp, xp, hs, k0, k1, W_c)  # noqa: E731
    elif args.stage == "proj":
        g = torch.Generator(device="cuda")
        g.manual_seed(7)
        ci = torch.randint(0, V, (B, L, K), generator=g, device="cuda", dtype=torch.int32)
        cv = torch.randn((B, L, K), generator=g, device="cuda")
        lv = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
        H = torch.rand((B, L, R), generator=g, device="cuda")
        E = torch.randn((V, D), generator=g, device="cuda").to(torch.bfloat16)
        WA = (torch.randn((R, D), generator=g, device="cuda") / D ** 0.5).to(torch.bfloat16)
        WB = (torch.randn((R, D), generator=g, device="cuda") / D ** 0.5).to(torch.bfloat16)
        run = lambda: api.pair_scores_proj(h, ci, cv, lv, H, E, WA, WB)  # noqa: E731
    else:
        M = 1024
        hidden = bf(torch, synth.normal_bits(1, (M, D)))
        W = bf(torch, synth.normal_bits(2, (V, D), std=0.02))
        ws = torch.empty(max(api.lmhead_topk_workspace(h, M, V, D), 256), dtype=torch.uint8, device="cuda")
        if args.stage == "lmhead_gate":
            W_H = bf(torch, synth.normal_bits(3, (R, D), std=0.02))
            run = lambda: api.lmhead_topk_gate(h, hidden, W, W_H, workspace=ws)  # noqa: E731
        else:
            run = lambda: api.lmhead_topk(h, hidden, W, workspace=ws)  # noqa: E731
    for _ in range(args.reps):
        run()
    torch.cuda.synchronize()
    assert h.device_error() == 0
    print(f"{args.stage}: {args.reps} runs ok")
    h.close()


if __name__ == "__main__":
    main()
