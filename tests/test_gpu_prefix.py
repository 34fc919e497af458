"""Attention over shared prefixes against the definition in 64 bits.

The definition, its bounds on `out` and the reference are those of tree_attention (test_gpu_cache_limits.py); lse is
bound by dz + 1e-6 (1 + |lse|) as in test_gpu_cache.py.  What no sequence owns holds NaN."""
import math

import numpy as np
import pytest
import torch

from draft_selection_dflash2_gb300 import api
from gpu_common import handle  # noqa: F401
from test_gpu_cache import randn, random_tree, words
from test_gpu_cache_limits import check, definition

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def roomy(groups, H, capacity):
    """A capacity for which sharing is expected to pay, whatever the lengths."""
    B = sum(len(own) for _, own in groups)
    return max(capacity, 128 * (6000 // max(1, (B - len(groups)) * H) + 1))


def shared_cache(gen, groups, H, D, page, capacity, layout="nhd", spoil=None, room=None):
    """groups: [(shared positions, [own positions of each sequence])] -> (cache, rows, cache_len, prefix_len, prefix_start).

    Whole pages of the shared positions are the same pages; the positions behind them, and everything without a block
    table, are copies.  spoil(kk, vv): changes a group's shared rows before they are written.  room: the capacity that the
    block table (or, without one, the memory) has, of which only the first `capacity` positions are ever used."""
    B = sum(len(own) for _, own in groups)
    rows, lens, prefix, start = [], [], [], [0]
    for P, own in groups:
        kk, vv = randn(gen, P, H, D, std=1.5), randn(gen, P, H, D)
        if spoil is not None:
            spoil(kk, vv)
        for n in own:
            rows.append((torch.cat([kk, randn(gen, n, H, D, std=1.5)]), torch.cat([vv, randn(gen, n, H, D)])))
            lens.append(P + n)
        prefix.append(P)
        start.append(len(rows))
    if page == 0:
        pages, size, table = B, room or capacity, None
    else:
        per, size = -(-capacity // page), page
        pages = B * per + 2
        perm = torch.randperm(pages, generator=torch.Generator().manual_seed(gen.initial_seed()))
        table = perm[:B * per].reshape(B, per).to(torch.int32).cuda()
        for g, (P, own) in enumerate(groups):
            table[start[g]:start[g + 1], :P // page] = table[start[g]:start[g] + 1, :P // page].clone()
        if room:
            table = torch.cat([table, table.new_full((B, max(0, -(-room // page) - per)), pages - 1)], 1)
    shape = (pages, size, H, D) if layout == "nhd" else (pages, H, size, D)
    k = torch.full(shape, NAN, dtype=torch.bfloat16, device="cuda")
    v = torch.full(shape, NAN, dtype=torch.bfloat16, device="cuda")
    if layout == "hnd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    for b, (kk, vv) in enumerate(rows):
        j = torch.arange(kk.shape[0], device="cuda")
        at = (torch.full_like(j, b), j) if table is None else (table[b].long()[j // size], j % size)
        k[at], v[at] = kk, vv
    return api.KVCache(k, v, table), rows, i32(lens), i32(prefix), i32(start)


def logsumexp(q, rows, k_new, sees, scale):
    """fp64 lse and dz of the definition."""
    B, T, heads, D = q.shape
    H = rows[0][0].shape[1]
    G = heads // H
    lse = torch.full((B, T, heads), -INF, dtype=torch.float64, device="cuda")
    dz = torch.zeros_like(lse)
    for b in range(B):
        for hq in range(heads):
            kk = rows[b][0][:, hq // G].double()
            vis = torch.ones(T, kk.shape[0], dtype=torch.bool, device="cuda")
            if k_new is not None:
                kk = torch.cat([kk, k_new[b, :, hq // G].double()])
                s = torch.ones(T, T, dtype=torch.bool, device="cuda").tril() if sees is None else sees[b]
                vis = torch.cat([vis, s], 1)
            if kk.shape[0] == 0:
                continue
            qq = q[b, :, hq].double()
            lse[b, :, hq] = torch.logsumexp(torch.where(vis, qq @ kk.T * scale, -INF), 1)
            dz[b, :, hq] = D * 2.0 ** -23 * torch.where(vis, qq.abs() @ kk.abs().T * scale, 0.0).amax(1)
    return lse, dz


def check_lse(lse, want, dz):
    dead = torch.isinf(want)
    assert torch.equal(torch.isinf(lse) & (lse < 0), dead)
    assert ((lse.double() - want).abs() <= dz + 1e-6 * (1 + want.abs()))[~dead].all()


CASES = [
    # groups, T, heads, H, D, page, layout, tree
    ([(300, [5])], 1, 4, 1, 128, 16, "nhd", False),                        # a sequence by itself
    ([(128, [0, 0])], 1, 1, 1, 64, 16, "nhd", False),                      # one tile, nothing of their own
    ([(127, [1, 129, 0])], 1, 8, 2, 128, 16, "nhd", False),                # less than a tile
    ([(0, [0, 3]), (0, [])], 2, 4, 2, 64, 32, "nhd", False),               # no prefix, a group without sequences
    ([(1008, [200, 30, 177, 1])], 1, 32, 8, 128, 16, "nhd", False),
    ([(640, [100] * 17)], 1, 16, 2, 128, 64, "nhd", False),                # 136 rows: a tile and 8 rows
    ([(384, [9, 0, 300]), (1, [40]), (515, [1, 2, 3, 4, 5]), (256, [7, 8])], 9, 12, 2, 64, 0, "nhd", True),
    ([(1300, [64, 250]), (129, [500, 0, 0])], 17, 16, 2, 128, 128, "hnd", False),      # blocks across sequences' ends
    ([(700, [10, 20, 30])], 33, 10, 2, 128, 32, "hnd", True),              # groups of 5: 25 nodes a tile
    ([(513, [1, 90])], 65, 4, 4, 64, 16, "nhd", True),                     # two mask words
    ([(260, [77, 5])], 128, 6, 2, 128, 256, "nhd", False),                 # the longest block, pages beyond a tile
    ([(400, [3, 2, 1])], 3, 128, 1, 64, 64, "nhd", True),                  # 128 query heads on one kv head
    ([(20000, [4, 300])], 2, 8, 1, 128, 64, "nhd", False),                 # one head: the prefix is split many ways
    ([(256, [20] * 40), (128, [1] * 30)], 1, 4, 4, 128, 16, "nhd", False), # many sequences of one tile each
]


@pytest.mark.parametrize("groups,T,heads,H,D,page,layout,tree", CASES)
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("shared", [True, False])
def test_prefix_attention(handle, groups, T, heads, H, D, page, layout, tree, drafted, shared):
    """shared: with a capacity for which sharing pays; otherwise the call is taken as tree attention."""
    gen = torch.Generator(device="cuda").manual_seed(T * 100 + heads)
    cap = max(P + max(own, default=0) for P, own in groups) + 3
    cache, rows, cl, pl, ps = shared_cache(gen, groups, H, D, page, cap, layout, room=roomy(groups, H, cap) if shared else None)
    B = len(rows)
    q, kn, vn = randn(gen, B, T, heads + 2 * H, D).split([heads, H, H], 2)
    sees = mask = None
    if not drafted:
        kn = vn = None
    elif tree:
        s = random_tree(np.random.default_rng(T), B, T)
        sees, mask = torch.from_numpy(s).cuda(), words(s)
    out, lse = api.prefix_attention(handle, q, cache, cl, pl, ps, kn, vn, tree_mask=mask)
    check(out, definition(q, rows, kn, vn, sees, D ** -0.5))
    check_lse(lse, *logsumexp(q, rows, kn, sees, D ** -0.5))
    again = api.prefix_attention(handle, q, cache, cl, pl, ps, kn, vn, tree_mask=mask)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    # nothing declared shared: the same sums
    alone, _ = api.prefix_attention(handle, q, cache, cl, pl[:0], k_new=kn, v_new=vn, tree_mask=mask)
    check(alone, definition(q, rows, kn, vn, sees, D ** -0.5))
    assert handle.device_error() == 0


def test_the_whole_batch_as_one_group_and_a_scale(handle):
    gen = torch.Generator(device="cuda").manual_seed(1)
    cache, rows, cl, pl, _ = shared_cache(gen, [(400, [1, 60, 200])], 2, 128, 32, 610, room=60000)
    q = randn(gen, 3, 4, 6, 128)
    out, lse = api.prefix_attention(handle, q, cache, cl, pl, scale=0.25)
    check(out, definition(q, rows, None, None, None, 0.25))
    check_lse(lse, *logsumexp(q, rows, None, None, 0.25))
    # a prefix that is declared shorter than it is
    out, _ = api.prefix_attention(handle, q, cache, cl, i32([130]), scale=0.25)
    check(out, definition(q, rows, None, None, None, 0.25))
    assert handle.device_error() == 0


def test_more_sequences_than_the_list_takes_at_once(handle):
    """1500 sequences in 500 groups: stretches past the first 1024."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    rng = np.random.default_rng(0)
    groups = [(int(rng.integers(0, 300)), [int(n) for n in rng.integers(0, 40, 3)]) for _ in range(500)]
    cache, rows, cl, pl, ps = shared_cache(gen, groups, 1, 64, 16, 345, room=1000)
    q, kn, vn = randn(gen, 1500, 1, 4, 64).split([2, 1, 1], 2)
    out, lse = api.prefix_attention(handle, q, cache, cl, pl, ps, kn, vn)
    want, _ = api.tree_attention(handle, q, cache, cl, kn, vn)
    pick = list(range(0, 1500, 97)) + [1023, 1024, 1025, 1499]
    d = definition(q[pick], [rows[b] for b in pick], kn[pick], vn[pick], None, 64 ** -0.5)
    check(out[pick], d)
    assert ((out - want).float().abs() <= 2.0 ** -6 * (1 + want.float().abs())).all()
    assert handle.device_error() == 0


@pytest.mark.parametrize("bad", [[1, 2, 4], [0, 3, 2], [0, 2, 3], [0, -1, 4], [0, 2, 1 << 30], [0, 1 << 31 - 1, 4]])
def test_starts_that_do_not_ascend_are_flagged(handle, bad):
    gen = torch.Generator(device="cuda").manual_seed(3)
    cache, rows, cl, pl, ps = shared_cache(gen, [(300, [5, 6]), (256, [7, 0])], 2, 64, 16, 330, room=60000)
    q = randn(gen, 4, 3, 4, 64)
    out, _ = api.prefix_attention(handle, q, cache, cl, pl, torch.tensor(bad, dtype=torch.int64, device="cuda").to(torch.int32))
    assert handle.device_error() == 0x10
    check(out, definition(q, rows, None, None, None, 64 ** -0.5))


def test_lengths_out_of_range_are_clamped_and_flagged(handle):
    gen = torch.Generator(device="cuda").manual_seed(4)
    cache, rows, cl, pl, ps = shared_cache(gen, [(300, [5, 0]), (256, [7, 0])], 2, 64, 16, 336, room=60000)
    q = randn(gen, 4, 3, 4, 64)
    want = definition(q, rows, None, None, None, 64 ** -0.5)
    for lens in ([1 << 30, 256], [301, 256], [-1, 256]):        # above the capacity, above a length, negative
        out, _ = api.prefix_attention(handle, q, cache, cl, i32(lens), ps)
        assert handle.device_error() == 0x10
        check(out, want)
    # a sequence that is shorter than its group's prefix: the prefix stops there
    short = cl.clone()
    short[1] = 200
    out, _ = api.prefix_attention(handle, q, cache, short, pl, ps)
    assert handle.device_error() == 0x10
    cut = [rows[0], tuple(x[:200] for x in rows[1]), rows[2], rows[3]]
    check(out, definition(q, cut, None, None, None, 64 ** -0.5))
    # cache lengths out of range: the capacity and 0
    full = api.KVCache(torch.ones_like(cache.k), torch.ones_like(cache.v), cache.block_table)
    out, lse = api.prefix_attention(handle, q, full, i32([-3, 1 << 30, 0, 0]), i32([0, 0]), ps)
    assert handle.device_error() == 0x10
    assert (out[1] == 1).all() and (out[[0, 2, 3]] == 0).all() and torch.isneginf(lse[[0, 2, 3]]).all()


def test_bad_pages_are_flagged(handle):
    gen = torch.Generator(device="cuda").manual_seed(5)
    cache, rows, cl, pl, ps = shared_cache(gen, [(256, [20, 20])], 2, 64, 16, 300, room=120000)
    q = randn(gen, 2, 1, 4, 64)
    table = cache.block_table.clone()
    table[0, 2], table[1, 17] = -1, 1 << 30
    full = api.KVCache(torch.ones_like(cache.k), torch.ones_like(cache.v), table)
    out, _ = api.prefix_attention(handle, q, full, cl, pl, ps)
    assert handle.device_error() == 0x8 and (out == 1).all()


@pytest.mark.parametrize("groups,T,heads,H,D,page", [
    ([(300, [5, 40])], 1, 8, 2, 128, 16), ([(900, [140, 0, 3])], 40, 16, 2, 64, 32),
    ([(3000, [2500, 700, 1]), (500, [9, 9])], 17, 16, 2, 128, 64), ([(20000, [64, 9])], 2, 8, 1, 64, 64)])
def test_infinite_and_nan_values(handle, groups, T, heads, H, D, page):
    """In the prefix they reach every row of the group; in what one sequence owns, that sequence alone."""
    gen = torch.Generator(device="cuda").manual_seed(T)

    def spoil(kk, vv):
        n = vv.shape[0]
        vv[n // 2, :, 3] = INF
        vv[5, :, 3] = INF
        vv[7, 0, 20], vv[n - 130, 0, 20] = INF, -INF       # both: NaN
        vv[9, H - 1, 33] = NAN

    cap = max(P + max(own) for P, own in groups)
    for full in (False, True):
        def rows_of_prefix(kk, vv):
            spoil(kk, vv)
            if full:
                kk[11] = -INF
        cache, rows, cl, pl, ps = shared_cache(gen, groups, H, D, page, cap, spoil=rows_of_prefix, room=roomy(groups, H, cap))
        B = len(rows)
        q, kn, vn = (randn(gen, B, T, n, D) for n in (heads, H, H))
        if full:
            q = q.abs()             # every score of that key is -inf: its value does not reach a row
        rows[0][1][-1, :, D - 1] = -INF
        at = rows[0][0].shape[0] - 1
        page_of = cache.block_table[0].long()[at // page]
        cache.v[page_of, at % page] = rows[0][1][-1]
        out, _ = api.prefix_attention(handle, q, cache, cl, pl, ps, kn, vn)
        again, _ = api.prefix_attention(handle, q, cache, cl, pl, ps, kn, vn)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
        want = definition(q, rows, kn, vn, None, D ** -0.5)
        check(out, want)
        assert torch.isposinf(out[..., 3]).all() and torch.isneginf(out[0, ..., D - 1]).all()
        assert torch.isfinite(out[1:, ..., D - 1]).all() and handle.device_error() == 0


@pytest.mark.parametrize("T,heads,H,D", [(3, 8, 2, 128), (9, 12, 2, 64), (17, 16, 2, 128), (5, 4, 2, 64)])
@pytest.mark.parametrize("tree", [True, False])
def test_infinite_and_nan_drafted_values(handle, T, heads, H, D, tree):
    """They reach the rows that see their nodes, of their sequences alone; many short items follow one another on a CTA."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    rng = np.random.default_rng(T)
    groups = [(256, [int(n) for n in rng.integers(0, 50, 100)]), (130, [int(n) for n in rng.integers(0, 200, 60)])]
    cache, rows, cl, pl, ps = shared_cache(gen, groups, H, D, 16, 340, room=4000)
    B = len(rows)
    q, kn, vn = (randn(gen, B, T, n, D) for n in (heads, H, H))
    sees = mask = None
    if tree:
        s = random_tree(rng, B, T)
        sees, mask = torch.from_numpy(s).cuda(), words(s)
    for b in range(0, B, 3):
        vn[b, b % T, b % H, b % D] = (INF, -INF, NAN)[b // 3 % 3]
    kn[7, T - 1, 0] = NAN
    out, _ = api.prefix_attention(handle, q, cache, cl, pl, ps, kn, vn, tree_mask=mask)
    want = definition(q, rows, kn, vn, sees, D ** -0.5)
    want[0][7, T - 1, :heads // H] = NAN       # a NaN score makes its row's softmax NaN (the definition's helper takes that for an empty row)
    check(out, want)
    again, _ = api.prefix_attention(handle, q, cache, cl, pl, ps, kn, vn, tree_mask=mask)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and handle.device_error() == 0


@pytest.mark.parametrize("first,second", [(30, 0), (31, 0), (29, 3), (61, 1), (62, 0), (63, 0), (64, 0), (40, 24), (1, 64)])
def test_any_number_of_stretches(handle, first, second):
    """Around the numbers of groups and sequences at which the list of stretches is made in another way."""
    gen = torch.Generator(device="cuda").manual_seed(first)
    rng = np.random.default_rng(first)
    groups = [(384, [int(n) for n in rng.integers(0, 90, first)])]
    groups += [(130, [int(n) for n in rng.integers(0, 90, second)])] if second else []
    cache, rows, cl, pl, ps = shared_cache(gen, groups, 1, 64, 16, 480, room=40000)
    B = len(rows)
    q, kn, vn = (randn(gen, B, 2, n, 64) for n in (4, 1, 1))
    out, lse = api.prefix_attention(handle, q, cache, cl, pl, ps, kn, vn)
    check(out, definition(q, rows, kn, vn, None, 64 ** -0.5))
    check_lse(lse, *logsumexp(q, rows, kn, None, 64 ** -0.5))
    assert handle.device_error() == 0
    # one sequence shorter than its group's prefix, and starts that are none
    short = cl.clone()
    short[B - 1] = 120
    out, _ = api.prefix_attention(handle, q, cache, short, pl, ps, kn, vn)
    assert handle.device_error() == 0x10
    cut = rows[:-1] + [tuple(x[:120] for x in rows[-1])]
    check(out, definition(q, cut, kn, vn, None, 64 ** -0.5))
    out, _ = api.prefix_attention(handle, q, cache, cl, pl, ps + 1, kn, vn)
    assert handle.device_error() == 0x10
    check(out, definition(q, rows, kn, vn, None, 64 ** -0.5))


def test_a_graph_replays_on_new_lengths_and_groups(handle):
    gen = torch.Generator(device="cuda").manual_seed(7)
    B, T, heads, H, D = 6, 3, 8, 2, 128
    plans = [[(256, [1, 2, 3]), (300, [9, 0, 77])], [(700, [0, 5, 6, 7, 8, 9]), (0, [])], [(0, [40]), (200, [1, 1, 1, 1, 1])]]
    sets = [shared_cache(gen, plan, H, D, 16, 720, room=60000) for plan in plans]
    k, v, table = (x.clone() for x in (sets[0][0].k, sets[0][0].v, sets[0][0].block_table))
    cache, cl, pl, ps = api.KVCache(k, v, table), i32([0] * B), i32([0, 0]), i32([0, 3, 6])
    q, kn, vn = randn(gen, B, T, heads + 2 * H, D).split([heads, H, H], 2)
    out, lse = torch.zeros(B, T, heads, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, T, heads, device="cuda")
    ws = torch.empty(api.prefix_attention_workspace(handle, B, T, heads, H, D), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.prefix_attention(handle, q, cache, cl, pl, ps, kn, vn, out=out, lse=lse, workspace=ws)
    for c, rows, cl1, pl1, ps1 in sets:
        for to, x in ((k, c.k), (v, c.v), (table, c.block_table), (cl, cl1), (pl, pl1), (ps, ps1)):
            to.copy_(x)
        ws.fill_(255)                                       # nothing of the last call is needed
        graph.replay()
        check(out, definition(q, rows, kn, vn, None, D ** -0.5))
    assert handle.device_error() == 0


def test_two_streams_at_once(handle):
    gen = torch.Generator(device="cuda").manual_seed(8)
    cache, rows, cl, pl, ps = shared_cache(gen, [(900, [30, 40, 50, 60])], 4, 128, 64, 970, room=60000)
    qs = [randn(gen, 4, 5, 16, 128) for _ in range(2)]
    want = [api.prefix_attention(handle, q, cache, cl, pl, ps)[0] for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [api.prefix_attention(handle, q, cache, cl, pl, ps, stream=s)[0] for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_empty_calls_and_refusals(handle):
    gen = torch.Generator(device="cuda").manual_seed(9)
    cache, rows, cl, pl, ps = shared_cache(gen, [(128, [3, 4])], 2, 64, 16, 140)
    q = randn(gen, 2, 3, 4, 64)
    for shape in ((0, 3, 4, 64), (2, 0, 4, 64)):
        x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        assert api.prefix_attention(handle, x, cache, cl[:shape[0]], pl[:0])[0].shape == shape
    ws = torch.empty(api.prefix_attention_workspace(handle, 2, 3, 4, 2, 64), dtype=torch.uint8, device="cuda")
    for kw, error in ((dict(prefix_start=ps[:1]), ValueError), (dict(prefix_start=ps.long()), ValueError),
                      (dict(prefix_len=pl.float()), ValueError), (dict(prefix_len=i32([1, 1]), prefix_start=None), api.Dflash2Error),
                      (dict(prefix_len=i32([1, 1, 1]), prefix_start=i32([0, 1, 2, 2])), api.Dflash2Error),
                      (dict(workspace=ws[:-256]), api.Dflash2Error), (dict(k_new=q[:, :, :2]), ValueError),
                      (dict(scale=0.0), api.Dflash2Error), (dict(out=q[:, :2]), ValueError),
                      (dict(tree_mask=torch.zeros(2, 3, 1, dtype=torch.int64, device="cuda")), api.Dflash2Error),
                      (dict(cache_len=cl.cpu()), ValueError)):
        with pytest.raises(error):
            api.prefix_attention(handle, **{**dict(q=q, cache=cache, cache_len=cl, prefix_len=pl, prefix_start=ps), **kw})
    wide, rows, cl, _, _ = shared_cache(gen, [(128, [3, 4])], 2, 64, 16, 140, room=100000)
    for shape in ((2, 1), (1, 3), (2, 3)):                  # any strides will do
        x = randn(gen, 5, 5, 4, 64)[:shape[0], 1:1 + shape[1]]
        out, _ = api.prefix_attention(handle, x, wide, cl[:shape[0]], i32([128 if shape[0] > 1 else 0]))
        check(out, definition(x, rows[:shape[0]], None, None, None, 64 ** -0.5))
    assert handle.device_error() == 0
