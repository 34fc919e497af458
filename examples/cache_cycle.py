"""Draft-verify cycles over a key/value cache that stays within a budget.

One attention layer stands in for the target model: its queries, keys and values are random
projections of the tokens' embeddings and its logits the products of its output with the same
embeddings, so every quantity has the shapes and the flow of a served model with nothing trained.
Each cycle

  1. drafts a block of L tokens per sequence (here: the target's own greedy choices, spoiled at
     random, so that verification accepts some of them);
  2. runs the target over the block in one pass: tree_attention from the L + 1 nodes (the last
     verified token and the drafts) to the cache and to one another;
  3. verifies the block against the pass's logits: verify gives each sequence's accepted length;
  4. commits the accepted nodes' keys and values: cache_commit;
  5. adds to every cached position the attention weight that the accepted nodes gave it: cache_scores;
  6. when the longest sequence nears the cache's capacity, keeps the recent positions and those
     weighed most in the other half of the page pool: cache_evict, and the two halves change places.

    python examples/cache_cycle.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from draft_selection_dflash2_gb300 import api  # noqa: E402


class Target:
    """One layer of grouped-query attention over random embeddings."""

    def __init__(self, V, heads, kv_heads, dim, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        width = 256

        def randn(*shape, std):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

        self.E = randn(V, width, std=1.0)
        self.W_qkv = randn((heads + 2 * kv_heads) * dim, width, std=width ** -0.5)
        self.W_o = randn(width, heads * dim, std=2.0 * (heads * dim) ** -0.5)

    def qkv(self, tokens):
        """[B, T] ids -> views q [B, T, heads, dim], k and v [B, T, kv_heads, dim] of one fused projection."""
        x = (self.E[tokens.long()] @ self.W_qkv.T).unflatten(-1, (-1, self.dim))
        return x.split([self.heads, self.kv_heads, self.kv_heads], dim=2)

    def logits(self, tokens, out):
        x = self.E[tokens.long()] + out.flatten(2) @ self.W_o.T
        return x @ self.E.T


def run(cycles=24, B=4, L=16, V=4096, heads=16, kv_heads=4, dim=128, page=64, capacity=256, keep=128, recent=32, seed=0):
    """-> per cycle (accepted lengths, cache lengths after it)."""
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = Target(V, heads, kv_heads, dim, seed)
    pages = capacity // page
    # one pool; every sequence owns two sets of pages and uses one of them
    pool = torch.zeros(2, 2 * B * pages, page, kv_heads, dim, dtype=torch.bfloat16, device="cuda")
    tables = torch.randperm(2 * B * pages, generator=gen, device="cuda").to(torch.int32).view(2, B, pages)
    cache, spare = (api.KVCache(pool[0], pool[1], tables[i]) for i in range(2))
    scores = torch.zeros(B, kv_heads, capacity, device="cuda")
    spare_scores = torch.zeros_like(scores)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    last = torch.randint(0, V, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
    log = []
    with api.Handle(0) as h:
        T = L + 1
        workspace = torch.empty(api.tree_attention_workspace(h, B, T, heads, kv_heads, dim), dtype=torch.uint8, device="cuda")
        for _ in range(cycles):
            # 1. a block: the target's greedy continuation, one token at a time, spoiled with probability 1/10
            block = last
            for _ in range(L):
                q, k, v = model.qkv(block)
                out, _ = api.tree_attention(h, q, cache, lens, k, v, workspace=workspace)
                nxt = model.logits(block, out)[:, -1].argmax(-1, keepdim=True).to(torch.int32)
                spoil = torch.rand(B, 1, generator=gen, device="cuda") < 0.1
                block = torch.cat([block, torch.where(spoil, (nxt + 1) % V, nxt)], 1)
            # 2. one pass over the block
            q, k, v = model.qkv(block)
            out, lse = api.tree_attention(h, q, cache, lens, k, v, workspace=workspace)
            # 3. the longest accepted prefix, and the target's next token
            accept, tokens = api.verify(h, model.logits(block, out).contiguous(), block[:, 1:].contiguous())
            last = tokens.gather(1, accept[:, None].long() - 1)
            # 4. and 5.: the accepted nodes are the first accept[b] of the block
            new_lens = api.cache_commit(h, k, v, cache, lens, count=accept, scores=scores)
            api.cache_scores(h, q, lse, cache, lens, scores, count=accept)
            lens = new_lens
            # 6.
            if int(lens.max()) + T > capacity:
                _, lens, _ = api.cache_evict(h, scores, cache, lens, spare, keep, recent, dst_scores=spare_scores)
                cache, spare, scores, spare_scores = spare, cache, spare_scores, scores
            log.append((accept.tolist(), lens.tolist()))
        error = h.device_error()
        if error:
            raise RuntimeError(f"device error word {error:#x}")
    return log


if __name__ == "__main__":
    for i, (accept, lens) in enumerate(run()):
        print(f"cycle {i}: accepted {accept}, cache {lens}")
