"""The cache operators together: draft-verify cycles over a cache within a budget."""
import importlib.util
import os

import pytest
import torch

from draft_selection_dflash2_gb300 import api
from gpu_common import handle  # noqa: F401
from test_gpu_determinism import Guarded

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("cache_cycle", os.path.join(ROOT, "examples", "cache_cycle.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_cycles_stay_within_the_budget(handle):
    log = example().run(cycles=20, capacity=192, keep=64, recent=16)
    before = [0, 0, 0, 0]
    evicted = 0
    for accept, lens in log:
        assert all(1 <= a <= 17 for a in accept)
        grown = [b + a for b, a in zip(before, accept)]
        if lens != grown:
            evicted += 1
            assert lens == [min(g, 64) for g in grown] and max(grown) + 17 > 192
        before = lens
    assert evicted >= 1
    assert sum(sum(a) for a, _ in log) > 20 * 4 * 3     # most drafts are the target's own choices


def test_a_committed_block_reads_as_the_same_attention(handle):
    # the last token of a block attends the same keys before and after the block joins the cache
    gen = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)

    cache = api.KVCache(randn(12, 32, 2, 128), randn(12, 32, 2, 128), torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6))
    lens = torch.tensor([150, 31], dtype=torch.int32, device="cuda")
    q, k, v = randn(2, 9, 8, 128), randn(2, 9, 2, 128), randn(2, 9, 2, 128)
    out, lse = api.tree_attention(handle, q, cache, lens, k, v)
    new = api.cache_commit(handle, k, v, cache, lens)
    again, lse2 = api.tree_attention(handle, q[:, -1:], cache, new)
    assert (lse2[:, 0] - lse[:, -1]).abs().max() <= 1e-5
    # two bf16 roundings of the same value, and the weights' own: at most 2 units in the last place
    a, b = out[:, -1].float(), again[:, 0].float()
    assert ((a - b).abs() <= 2.0 ** -6 * torch.maximum(a.abs(), b.abs()) + 1e-3).all()


def test_outputs_stay_inside_their_buffers(handle):
    gen = torch.Generator(device="cuda").manual_seed(2)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)

    B, T, heads, H, D = 3, 5, 6, 2, 64
    table = torch.randperm(24, generator=gen, device="cuda").to(torch.int32).view(3, 8)
    lens = torch.tensor([100, 0, 77], dtype=torch.int32, device="cuda")
    q, k, v = randn(B, T, heads, D), randn(B, T, H, D), randn(B, T, H, D)
    outs = []
    for _ in range(2):
        g = Guarded()
        pk, pv = g((24, 16, H, D), torch.bfloat16), g((24, 16, H, D), torch.bfloat16)
        gen2 = torch.Generator(device="cuda").manual_seed(3)
        for x in (pk, pv):
            x.copy_(torch.randn(x.shape, generator=gen2, device="cuda"))
        cache = api.KVCache(pk, pv, table)
        out, lse = g((B, T, heads, D), torch.bfloat16), g((B, T, heads), torch.float32)
        ws = g((api.tree_attention_workspace(handle, B, T, heads, H, D),), torch.uint8)
        api.tree_attention(handle, q, cache, lens, k, v, out=out, lse=lse, workspace=ws)
        scores, new = g((B, H, 128), torch.float32), g((B,), torch.int32)
        scores.zero_()
        api.cache_commit(handle, k, v, cache, lens, scores=scores, new_len=new)
        api.cache_scores(handle, q, lse, cache, lens, scores)
        dk, dv = g((3, 40, H, D), torch.bfloat16), g((3, 40, H, D), torch.bfloat16)
        kept, n2, ds = g((B, H, 33), torch.int32), g((B,), torch.int32), g((B, H, 33), torch.float32)
        api.cache_evict(handle, scores, cache, new, api.KVCache(dk, dv), 33, 4, kept=kept, new_len=n2, dst_scores=ds)
        g.check()
        outs.append([t.clone() for t in (out, lse, scores, new, kept, n2, pk, pv)])
    for a, b in zip(*outs):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert handle.device_error() == 0


def test_calls_in_a_graph(handle):
    gen = torch.Generator(device="cuda").manual_seed(4)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)

    cache = api.KVCache(randn(2, 700, 4, 128), randn(2, 700, 4, 128))
    lens = torch.tensor([600, 333], dtype=torch.int32, device="cuda")
    q, k, v = randn(2, 17, 16, 128), randn(2, 17, 4, 128), randn(2, 17, 4, 128)
    ws = torch.empty(api.tree_attention_workspace(handle, 2, 17, 16, 4, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, 17, 16, device="cuda")
    scores = torch.zeros(2, 4, 700, device="cuda")
    want = api.tree_attention(handle, q, cache, lens, k, v)
    api.cache_scores(handle, q, want[1], cache, lens, scores)
    first = scores.clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        api.tree_attention(handle, q, cache, lens, k, v, out=out, lse=lse, workspace=ws)
        scores.zero_()
        api.cache_scores(handle, q, lse, cache, lens, scores)
    for shift in (0, 1):
        lens.copy_(torch.tensor([600 - shift, 333], dtype=torch.int32))   # lengths are read by the replay
        graph.replay()
        torch.cuda.synchronize()
        if shift == 0:
            assert torch.equal(out, want[0]) and torch.equal(scores, first)
        else:
            assert not torch.equal(out[0], want[0][0]) and torch.equal(out[1], want[0][1])
    assert handle.device_error() == 0
