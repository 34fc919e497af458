"""The operators around one verify pass together, as a served model would use them: prompts shared by several sequences,
appended with their keys rotated; blocks of drafts whose queries and keys are rotated to their positions; attention over the
shared prompt and each sequence's own cache; the logits' penalties and allowed tokens; verification; and the accepted tokens
into the cache and the counts.  Everything is compared with plain torch at every step."""
import math

import pytest
import torch

from draft_selection_dflash2_gb300 import api
from gpu_common import handle  # noqa: F401
from test_gpu_cache_limits import check, definition

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rotate(x, pos, inverse_rates):
    """Half layout, whole head, in 64 bits."""
    a = pos.double()[..., None] * inverse_rates
    c, s = a.cos()[:, :, None], a.sin()[:, :, None]
    half = x.shape[-1] // 2
    one, two = x.double()[..., :half], x.double()[..., half:]
    return torch.cat([one * c - two * s, two * c + one * s], -1)


def near(got, want, what):
    # a rounding to bf16, and fp32 before it (see test_gpu_rope.py; |x1| + |x2| is below 16 here)
    assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -17).all(), what


@pytest.mark.parametrize("captured", [False, True])
def test_cycles(handle, captured):
    B, G, L, V, heads, H, D, page, P = 6, 2, 4, 500, 8, 2, 64, 16, 256
    T, width, capacity = L + 1, 128, 30000
    gen = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(BF)  # noqa: E731
    E = randn(V, width)
    W_qkv, W_o = randn((heads + 2 * H) * D, width, std=width ** -0.5), randn(width, heads * D, std=(heads * D) ** -0.5)
    qkv = lambda tok: (E[tok.long()] @ W_qkv.T).unflatten(-1, (-1, D)).split([heads, H, H], 2)  # noqa: E731
    rates = 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    rope = api.Rope(D)
    # two groups of three sequences, each with a prompt of its own in shared pages; the pages behind it are each sequence's own
    prompt = torch.randint(0, V, (G, P), generator=gen, device="cuda", dtype=torch.int32)
    shared, own = P // page, 8
    pool = torch.zeros(2, G * shared + B * own, page, H, D, dtype=BF, device="cuda")
    table = torch.zeros(B, capacity // page, dtype=torch.int32, device="cuda")
    for b in range(B):
        g = b // 3
        table[b, :shared] = torch.arange(g * shared, (g + 1) * shared)
        table[b, shared:shared + own] = G * shared + b * own + torch.arange(own)
    cache = api.KVCache(pool[0], pool[1], table)
    first = api.KVCache(pool[0], pool[1], table[::3].contiguous())
    none = torch.zeros(G, dtype=torch.int32, device="cuda")
    q, k, v = qkv(prompt)
    plen, _ = api.cache_append(handle, k, v, first, none, rope)
    assert plen.tolist() == [P, P]
    keys = rotate(k, torch.arange(P, device="cuda")[None].expand(G, P), rates)
    near(pool[0][:G * shared].view(G, P, H, D), keys, "prompt")
    counts = torch.zeros(B, 504, dtype=torch.int32, device="cuda")[:, :V]
    api.token_counts(handle, prompt.repeat_interleave(3, 0), counts, prompt=True)
    start = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    lens = plen.repeat_interleave(3).contiguous()
    rep, pres = torch.full((B,), 1.3, device="cuda"), torch.full((B,), 0.5, device="cuda")
    allowed = torch.full((1, 1, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    allowed[..., 0] = ~0xFF                                    # the first 8 tokens are never allowed
    block = torch.randint(0, V, (B, T), generator=gen, device="cuda", dtype=torch.int32)
    ws = torch.empty(api.prefix_attention_workspace(handle, B, T, heads, H, D), dtype=torch.uint8, device="cuda")
    workspaces = dict(out=torch.empty(B, T, heads, D, dtype=BF, device="cuda"), lse=torch.empty(B, T, heads, device="cuda"),
                      workspace=ws)

    def cycle():
        q, k, v = qkv(block)
        q0, k0 = q.clone(), k.clone()
        api.rope(handle, q, rope, lens, out=q)                 # in place: k and v keep their common strides
        api.rope(handle, k, rope, lens, out=k)
        out, lse = api.prefix_attention(handle, q, cache, lens, plen, start, k, v, **workspaces)
        raw = torch.zeros(B, T, 504, dtype=BF, device="cuda")[..., :V]
        raw.copy_((E[block.long()] + out.flatten(2) @ W_o.T) @ E.T)
        logits = api.logits_adjust(handle, raw, counts, block, repetition=rep, presence=pres, allowed=allowed)
        accept, tokens = api.verify(handle, logits, block[:, 1:].contiguous(), V=V)
        new_lens = api.cache_commit(handle, k, v, cache, lens, count=accept)
        before = counts.clone()
        api.token_counts(handle, block, counts, count=accept)
        return dict(q=q0, k=k0, v=v, qr=q, kr=k, out=out, raw=raw, logits=logits, accept=accept, tokens=tokens,
                    new_lens=new_lens, before=before)

    if captured:
        for _ in range(2):                                     # libraries' first calls stay out of the graph
            (E[block.long()] + torch.zeros(B, T, heads * D, dtype=BF, device="cuda") @ W_o.T) @ E.T
            qkv(block)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = cycle()
    accepted = 0
    for step in range(6):
        hist = counts.clone()
        n = lens.tolist()
        rows = [(pool[0][table[b, :-(-m // page)].long()].flatten(0, 1)[:m].clone(),
                 pool[1][table[b, :-(-m // page)].long()].flatten(0, 1)[:m].clone()) for b, m in enumerate(n)]
        if captured:
            graph.replay()
        else:
            got = cycle()
        pos = lens[:, None] + torch.arange(T, device="cuda")
        near(got["qr"], rotate(got["q"], pos, rates), "queries")
        near(got["kr"], rotate(got["k"], pos, rates), "keys")
        check(got["out"], definition(got["qr"], rows, got["kr"], got["v"], None, D ** -0.5))
        for b in range(B):
            for t in range(T):
                x = got["raw"][b, t].double()
                seen = (hist[b] & 0x7FFFFFFF) + torch.bincount(block[b, :t + 1].long(), minlength=V)
                known = (seen > 0) | (hist[b] < 0)
                want = torch.where(known, torch.where(x > 0, x / 1.3, x * 1.3), x) - 0.5 * (seen > 0)
                want[:8] = -math.inf
                y = got["logits"][b, t].double()
                assert torch.equal(torch.isinf(y), torch.isinf(want))
                assert ((y - want).abs()[8:] <= (2.0 ** -8 * want.abs() + 2.0 ** -20 * (x.abs() * 1.3 + 1))[8:]).all()
            # verification of the adjusted logits: the longest prefix that is the target's choice (ties: lowest id)
            top = got["logits"][b].float().argmax(-1).tolist()
            m = 1
            while m < T and top[m - 1] == int(block[b, m]):
                m += 1
            assert int(got["accept"][b]) == m and got["tokens"][b, :m].tolist() == top[:m]
            assert int(got["new_lens"][b]) == n[b] + m
            at = n[b] + torch.arange(m, device="cuda")
            assert torch.equal(pool[0][table[b].long()[at // page], at % page], got["kr"][b, :m])
            assert torch.equal(counts[b], hist[b] + torch.bincount(block[b, :m].long(), minlength=V).int())
            accepted += m
        # the next block: the target's next token, then its own choices for the rest, spoiled here and there
        last = got["tokens"].gather(1, got["accept"][:, None].long() - 1)
        spoil = torch.randint(0, V, (B, L), generator=gen, device="cuda", dtype=torch.int32)
        keep = torch.rand(B, L, generator=gen, device="cuda") < 0.5
        guess = got["logits"][:, :L].float().argmax(-1).int()
        block.copy_(torch.cat([last, torch.where(keep, guess, spoil)], 1))
        lens.copy_(got["new_lens"])
    assert accepted >= 6 * B and handle.device_error() == 0


def test_append_allocates_what_it_is_not_given(handle):
    cache = api.KVCache(*(torch.zeros(2, 32, 2, 64, dtype=BF, device="cuda") for _ in range(2)))
    kn, vn, q = (torch.randn(2, 5, n, 64, device="cuda").to(BF) for n in (2, 2, 4))
    lens = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    count = torch.tensor([2, 5], dtype=torch.int32, device="cuda")
    rope = api.Rope(64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        new_len, q_out = api.cache_append(handle, kn, vn, cache, lens, rope, count, q=q, stream=stream)
        torch.cuda.synchronize()
        assert new_len.tolist() == [5, 5] and (q_out[0, 2:] == 0).all()
        assert torch.equal(q_out[1], api.rope(handle, q, rope, lens)[1])
    assert handle.device_error() == 0
