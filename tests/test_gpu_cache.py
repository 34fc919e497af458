"""The cache operators against plain 64-bit forms: attention from a drafted
block or tree over a paged cache, the commit of an accepted path, accumulated
attention weights, and eviction.

Whatever no sequence owns (positions past a length, unused pages) holds NaN, so
a value that leaks from there shows.  Bounds, per element:
  z     a fp32 dot product of D terms: dz = D 2^-23 max(scale <|q|, |k|>)
  lse   dz + 1e-6 (1 + |lse|)             (exp2, log2 and sums in fp32)
  out   2^-9 |out| (its own rounding) + 2^-9 A (the weights' rounding to bf16) +
        2 dz A, A = sum p |v|, and 5% of all that for second-order terms
  score (dz + 2^-20) w + 2^-22 (w + what was there)
"""
import math

import numpy as np
import pytest
import torch

from draft_selection_dflash2_gb300 import api
from gpu_common import handle  # noqa: F401

pytestmark = pytest.mark.gpu
NAN = float("nan")


def randn(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def make_cache(gen, lens, H, D, page, capacity, layout="nhd", extra=2):
    """A cache whose owned positions are normal and everything else NaN; the dense rows [B][n, H, D] beside it."""
    B = len(lens)
    if page == 0:
        pages, size, table = B, capacity, None
    else:
        per = -(-capacity // page)
        pages, size = B * per + extra, page
        perm = torch.randperm(pages, generator=torch.Generator().manual_seed(gen.initial_seed()))
        table = perm[:B * per].reshape(B, per).to(torch.int32).cuda()
    shape = (pages, size, H, D) if layout == "nhd" else (pages, H, size, D)
    k = torch.full(shape, NAN, dtype=torch.bfloat16, device="cuda")
    v = torch.full(shape, NAN, dtype=torch.bfloat16, device="cuda")
    if layout == "hnd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    cache = api.KVCache(k, v, table)
    rows = []
    for b, n in enumerate(lens):
        kk, vv = randn(gen, n, H, D, std=1.5), randn(gen, n, H, D)
        rows.append((kk, vv))
        write_rows(cache, b, 0, kk, vv)
    return cache, rows


def place(cache, b, j):
    """(page, row) index tensors of positions j of sequence b."""
    size = cache.k.shape[1]
    if cache.block_table is None:
        return torch.full_like(j, b), j
    return cache.block_table[b].long()[j // size], j % size


def write_rows(cache, b, j0, kk, vv):
    j = torch.arange(j0, j0 + kk.shape[0], device="cuda")
    cache.k[place(cache, b, j)], cache.v[place(cache, b, j)] = kk, vv


def read_rows(cache, b, n):
    j = torch.arange(n, device="cuda")
    return cache.k[place(cache, b, j)], cache.v[place(cache, b, j)]


def random_tree(rng, B, T):
    sees = np.zeros((B, T, T), bool)
    for b in range(B):
        for t in range(T):
            if t:
                p = int(rng.integers(max(0, t - 5), t))
                sees[b, t] = sees[b, p]
            sees[b, t, t] = True
    return sees


def words(sees):
    B, T, _ = sees.shape
    bits = np.zeros((B, T, (T + 63) // 64 * 64), np.uint8)
    bits[:, :, :T] = sees
    return torch.from_numpy(np.packbits(bits, axis=-1, bitorder="little").view(np.int64).copy()).cuda()


def reference(q, rows, k_new, v_new, sees, scale):
    """fp64 (out, lse, A, dz) by sequence and kv head."""
    B, T, heads, D = q.shape
    H = rows[0][0].shape[1]
    G = heads // H
    out = torch.zeros(B, T, heads, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, heads), -math.inf, dtype=torch.float64, device="cuda")
    A, dz = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        n = rows[b][0].shape[0]
        for h in range(H):
            qq = q[b, :, h * G:(h + 1) * G].double().reshape(T * G, D)
            kk, vv = rows[b][0][:, h].double(), rows[b][1][:, h].double()
            vis = torch.ones(T * G, n, dtype=torch.bool, device="cuda")
            if k_new is not None:
                kk = torch.cat([kk, k_new[b, :, h].double()])
                vv = torch.cat([vv, v_new[b, :, h].double()])
                s = torch.from_numpy(sees[b]).cuda()
                vis = torch.cat([vis, s.repeat_interleave(G, 0)], 1)
            z = qq @ kk.T * scale
            zabs = torch.where(vis, qq.abs() @ kk.abs().T * scale, 0.0)
            z = torch.where(vis, z, -math.inf)
            if z.shape[1] == 0:
                continue
            m = z.amax(1, keepdim=True)
            p = torch.where(vis, torch.exp(z - torch.where(torch.isinf(m), 0.0, m)), 0.0)
            l = p.sum(1, keepdim=True)
            p = p / torch.where(l == 0, 1.0, l)
            # a masked weight times a masked NaN is not part of the sum
            o = torch.stack([(torch.where(vis[r][:, None], p[r][:, None] * vv, 0.0)).sum(0) for r in range(T * G)])
            a = torch.stack([(torch.where(vis[r][:, None], p[r][:, None] * vv.abs(), 0.0)).sum(0)
                             for r in range(T * G)])
            out[b, :, h * G:(h + 1) * G] = o.reshape(T, G, D)
            A[b, :, h * G:(h + 1) * G] = a.reshape(T, G, D)
            lse[b, :, h * G:(h + 1) * G] = (m + l.log()).reshape(T, G)
            dz[b, :, h * G:(h + 1) * G] = (D * 2.0 ** -23 * zabs.nan_to_num(0.0).amax(1)).reshape(T, G)
    return out, lse, A, dz


def check_attention(got, want):
    out, lse = got
    ro, rl, A, dz = want
    assert out.dtype == torch.bfloat16 and lse.dtype == torch.float32
    dead = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), dead)
    assert (out[dead] == 0).all()
    live = ~dead
    el = (lse.double() - rl)[live].abs()
    assert (el <= (dz + 1e-6 * (1 + rl.abs()))[live]).all(), el.max()
    tol = 1.05 * (2.0 ** -9 * (ro.abs() + A) + 2 * dz[..., None] * A)
    err = (out.double() - ro).abs()
    assert (err <= tol)[live].all(), (err - tol)[live].max()


CASES = [
    # lens, T, heads, kv_heads, D, page, layout, tree
    ([0], 1, 4, 1, 128, 16, "nhd", False),                  # nothing cached: a node sees itself
    ([1], 1, 1, 1, 64, 16, "nhd", False),
    ([127, 128, 129], 1, 8, 2, 128, 16, "nhd", False),      # around a tile's end
    ([500], 17, 32, 8, 128, 64, "nhd", False),
    ([1000, 3, 0, 255, 256, 257], 5, 6, 2, 64, 32, "nhd", True),   # ragged, one empty, groups of 3
    ([700, 65], 33, 10, 2, 128, 128, "hnd", True),          # head-major pages, groups of 5
    ([300, 1025], 64, 16, 2, 128, 256, "nhd", True),        # 512 rows per kv head, pages larger than a tile
    ([513], 65, 4, 4, 64, 16, "nhd", True),                 # two mask words
    ([200, 77], 128, 6, 2, 128, 16, "nhd", False),          # the longest block
    ([90, 40], 3, 128, 1, 64, 64, "nhd", True),             # 128 query heads on one kv head
    ([301, 77, 5], 7, 16, 1, 128, 0, "nhd", False),         # one contiguous buffer each, odd capacity
    ([3000], 2, 8, 8, 64, 0, "hnd", True),
    ([4000, 2500, 1], 17, 12, 4, 128, 64, "hnd", False),
    ([20000], 4, 8, 1, 128, 64, "nhd", False),              # one head: the axis is split many ways
]


@pytest.mark.parametrize("lens,T,heads,H,D,page,layout,tree", CASES)
def test_attention(handle, lens, T, heads, H, D, page, layout, tree):
    gen = torch.Generator(device="cuda").manual_seed(len(lens) * 1000 + T)
    rng = np.random.default_rng(T)
    B = len(lens)
    cache, rows = make_cache(gen, lens, H, D, page, max(lens) + 3, layout)
    # q and the new rows are views of one fused tensor, so that no stride is a dense one
    qkv = randn(gen, B, T, heads + 2 * H, D)
    q, kn, vn = qkv[:, :, :heads], qkv[:, :, heads:heads + H], qkv[:, :, heads + H:]
    sees = random_tree(rng, B, T) if tree else np.tril(np.ones((T, T), bool))[None].repeat(B, 0)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    mask = words(sees) if tree else None
    got = api.tree_attention(handle, q, cache, cl, kn, vn, tree_mask=mask)
    want = reference(q, rows, kn, vn, sees, D ** -0.5)
    check_attention(got, want)
    again = api.tree_attention(handle, q, cache, cl, kn, vn, tree_mask=mask)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert handle.device_error() == 0


@pytest.mark.parametrize("lens,T,page", [([0, 130, 0], 3, 16), ([257, 1], 40, 0), ([64], 1, 64)])
def test_attention_to_the_cache_alone(handle, lens, T, page):
    gen = torch.Generator(device="cuda").manual_seed(5)
    cache, rows = make_cache(gen, lens, 2, 128, page, max(lens) + 1)
    q = randn(gen, len(lens), T, 8, 128)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = api.tree_attention(handle, q, cache, cl, scale=0.25)
    check_attention(got, reference(q, rows, None, None, None, 0.25))
    assert handle.device_error() == 0


def test_masks_that_leave_rows_empty_and_hide_non_finite_nodes(handle):
    # nodes 2 and 5 hold NaN and infinities and are seen by nobody but themselves; node 3 sees nothing
    gen = torch.Generator(device="cuda").manual_seed(6)
    for T, lens in ((8, [0, 200]), (70, [0, 131])):
        cache, rows = make_cache(gen, lens, 2, 128, 16, 210)
        q, kn, vn = randn(gen, 2, T, 8, 128), randn(gen, 2, T, 2, 128), randn(gen, 2, T, 2, 128)
        kn[:, 2] = NAN
        vn[:, 2, :, 5] = NAN
        vn[:, 2, :, 9] = math.inf
        vn[:, 5] = -math.inf
        sees = np.tril(np.ones((T, T), bool))[None].repeat(2, 0)
        sees[:, :, [2, 5]] = False
        sees[:, 3] = False
        cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        got = api.tree_attention(handle, q, cache, cl, kn, vn, tree_mask=words(sees))
        check_attention(got, reference(q, rows, kn, vn, sees, 128 ** -0.5))
        assert (got[0][0, 3] == 0).all() and torch.isneginf(got[1][0, 3]).all()
        # where node 5 is visible its infinities arrive, and only there
        sees[:, 7, 5] = True
        out, _ = api.tree_attention(handle, q, cache, cl, kn, vn, tree_mask=words(sees))
        assert torch.isneginf(out[:, 7]).all()
        rest = [t for t in range(T) if t != 7]
        assert torch.equal(out[:, rest], got[0][:, rest])
    assert handle.device_error() == 0


def test_scores_at_the_lowest_value_and_large_scores(handle):
    # keys that put every z at -inf leave a row empty; one key far above the rest takes all the weight
    gen = torch.Generator(device="cuda").manual_seed(7)
    cache, rows = make_cache(gen, [150], 1, 64, 16, 150)
    q = torch.ones(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    cl = torch.tensor([150], dtype=torch.int32, device="cuda")
    rows[0][0][:] = -math.inf
    write_rows(cache, 0, 0, *rows[0])
    out, lse = api.tree_attention(handle, q, cache, cl)
    assert (out == 0).all() and torch.isneginf(lse).all()
    rows[0][0][:] = -3.0e38
    rows[0][0][77] = 100.0
    write_rows(cache, 0, 0, *rows[0])
    out, lse = api.tree_attention(handle, q, cache, cl, scale=1.0)
    v = rows[0][1][77, 0].float()
    assert ((out[0, 0] - v).abs() <= 2.0 ** -8 * v.abs()).all() and ((lse - 6400.0).abs() <= 6401e-6).all()
    # a maximum that keeps rising along the axis rescales the sums again and again
    rows[0][0][:] = (torch.arange(150, device="cuda") * 0.5)[:, None, None].to(torch.bfloat16)
    write_rows(cache, 0, 0, *rows[0])
    check_attention(api.tree_attention(handle, q, cache, cl), reference(q, rows, None, None, None, 0.125))


def test_a_rising_maximum_over_many_tiles(handle):
    gen = torch.Generator(device="cuda").manual_seed(8)
    n = 5000
    cache, rows = make_cache(gen, [n], 2, 128, 64, n)
    ramp = torch.linspace(0.0, 3.0, n, device="cuda")[:, None, None]
    rows[0][0].copy_((rows[0][0].float() * 0.2 + ramp).to(torch.bfloat16))
    write_rows(cache, 0, 0, *rows[0])
    q = randn(gen, 1, 17, 8, 128).abs()
    kn, vn = randn(gen, 1, 17, 2, 128), randn(gen, 1, 17, 2, 128)
    sees = np.tril(np.ones((17, 17), bool))[None]
    cl = torch.tensor([n], dtype=torch.int32, device="cuda")
    check_attention(api.tree_attention(handle, q, cache, cl, kn, vn),
                    reference(q, rows, kn, vn, sees, 128 ** -0.5))


def test_lengths_and_pages_outside_their_range_are_clamped_and_flagged(handle):
    gen = torch.Generator(device="cuda").manual_seed(9)
    cache, rows = make_cache(gen, [48, 48], 1, 64, 16, 48)
    q, kn, vn = randn(gen, 2, 2, 2, 64), randn(gen, 2, 2, 1, 64), randn(gen, 2, 2, 1, 64)
    sees = np.tril(np.ones((2, 2), bool))[None].repeat(2, 0)
    cl = torch.tensor([1000, -4], dtype=torch.int32, device="cuda")
    got = api.tree_attention(handle, q, cache, cl, kn, vn)
    assert handle.device_error() == api.DEVERR_BAD_LENGTH
    rows[1] = (rows[1][0][:0], rows[1][1][:0])
    check_attention(got, reference(q, rows, kn, vn, sees, 0.125))
    good = cache.block_table.clone()
    cache.block_table[0, 1] = 10 ** 6
    cache.block_table[1, 2] = -7
    cl = torch.tensor([48, 20], dtype=torch.int32, device="cuda")
    api.tree_attention(handle, q, cache, cl, kn, vn)
    assert handle.device_error() == api.DEVERR_BAD_PAGE
    # an entry past the length is not looked at
    cache.block_table.copy_(good)
    cache.block_table[1, 2] = -7
    api.tree_attention(handle, q, cache, cl, kn, vn)
    assert handle.device_error() == 0


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("lens,T,H,D,page,layout,tree", [
    ([0], 1, 1, 64, 16, "nhd", False), ([15, 16, 17], 17, 8, 128, 16, "nhd", False),
    ([100, 0, 63], 65, 2, 64, 32, "hnd", True), ([7, 300], 128, 3, 128, 0, "nhd", True)])
def test_commit(handle, lens, T, H, D, page, layout, tree):
    gen = torch.Generator(device="cuda").manual_seed(T)
    rng = np.random.default_rng(T)
    B = len(lens)
    cap = max(lens) + T
    cache, rows = make_cache(gen, lens, H, D, page, cap, layout)
    kv = randn(gen, B, T, 2 * H, D)
    kn, vn = kv[:, :, :H], kv[:, :, H:]
    count = rng.integers(0, T + 1, B).astype(np.int32)
    path = None
    if tree:
        path = np.full((B, T), -1, np.int32)
        for b in range(B):
            path[b, :count[b]] = np.sort(rng.permutation(T)[:count[b]])
    before = cache.k.clone(), cache.v.clone()
    scores = torch.full((B, H, cap), 5.0, device="cuda")
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new_len = api.cache_commit(handle, kn, vn, cache, cl, torch.from_numpy(count).cuda(),
                               None if path is None else torch.from_numpy(path).cuda(), scores)
    want = [n + int(c) for n, c in zip(lens, count)]
    assert new_len.tolist() == want and cl.tolist() == lens
    expect = api.KVCache(before[0].contiguous(), before[1].contiguous(), cache.block_table)
    for b in range(B):
        nodes = list(range(count[b])) if path is None else path[b, :count[b]].tolist()
        write_rows(expect, b, lens[b], kn[b, nodes], vn[b, nodes])
        s = torch.full((H, cap), 5.0, device="cuda")
        s[:, lens[b]:want[b]] = 0.0
        assert torch.equal(scores[b], s)
    for x, y in ((cache.k, expect.k), (cache.v, expect.v)):
        assert torch.equal(x.contiguous().view(torch.int16), y.view(torch.int16))
    assert handle.device_error() == 0


def test_commit_defaults_and_what_does_not_fit(handle):
    gen = torch.Generator(device="cuda").manual_seed(3)
    cache, rows = make_cache(gen, [30, 4], 2, 64, 16, 32)
    kn, vn = randn(gen, 2, 5, 2, 64), randn(gen, 2, 5, 2, 64)
    cl = torch.tensor([30, 4], dtype=torch.int32, device="cuda")
    assert api.cache_commit(handle, kn, vn, cache, cl).tolist() == [32, 9]      # 3 of the 5 do not fit
    assert handle.device_error() == api.DEVERR_BAD_LENGTH
    assert torch.equal(read_rows(cache, 0, 32)[0][30:], kn[0, :2])
    assert torch.equal(read_rows(cache, 1, 9)[1][4:], vn[1])
    # a page outside the cache is not written, a node outside the block is clamped
    cl = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    cache.block_table[0, 0] = 99
    path = torch.tensor([[0, 1, 2, 3, 4], [7, -1, 0, 0, 0]], dtype=torch.int32, device="cuda")
    count = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    before = cache.k.clone()
    assert api.cache_commit(handle, kn, vn, cache, cl, count, path).tolist() == [1, 11]
    assert handle.device_error() == api.DEVERR_BAD_PAGE | api.DEVERR_BAD_NODE
    assert torch.equal(read_rows(cache, 1, 11)[0][9:], kn[1, [4, 0]])
    changed = (cache.k.view(torch.int16) != before.view(torch.int16)).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [int(cache.block_table[1, 0])]
    # counts outside [0, T] are clamped
    cache.block_table[0, 0] = cache.block_table[0, 1]
    count = torch.tensor([-2, 9], dtype=torch.int32, device="cuda")
    cl = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    assert api.cache_commit(handle, kn, vn, cache, cl, count).tolist() == [0, 5]
    assert handle.device_error() == api.DEVERR_BAD_LENGTH


# ---------------------------------------------------------------------------
# scores
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("lens,T,heads,H,D,page,tree", [
    ([1], 1, 1, 1, 64, 16, False), ([127, 128, 129, 0], 1, 8, 2, 128, 16, False),
    ([500, 777], 17, 32, 8, 128, 64, False), ([300, 1000], 64, 16, 2, 128, 32, True),
    ([260], 128, 10, 2, 64, 0, True), ([130, 5], 128, 16, 2, 128, 16, False),
    ([900], 3, 128, 1, 128, 256, True), ([2000, 33], 9, 18, 6, 64, 128, True)])
def test_scores(handle, lens, T, heads, H, D, page, tree):
    gen = torch.Generator(device="cuda").manual_seed(T + 1)
    rng = np.random.default_rng(T)
    B, G = len(lens), heads // H
    cap = max(lens) + 2
    cache, rows = make_cache(gen, lens, H, D, page, cap)
    qkv = randn(gen, B, T, heads + 2 * H, D)
    q = qkv[:, :, :heads]
    count = rng.integers(1, T + 1, B).astype(np.int32)
    count[-1] = T
    path = None
    if tree:
        path = np.full((B, T), -1, np.int32)
        for b in range(B):
            path[b, :count[b]] = np.sort(rng.permutation(T)[:count[b]])
    _, lse, _, _ = reference(q, rows, None, None, None, D ** -0.5)
    lse = lse.float()
    start = torch.rand(B, H, cap, generator=gen, device="cuda")
    scores = start.clone()
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    api.cache_scores(handle, q, lse, cache, cl, scores, torch.from_numpy(count).cuda(),
                     None if path is None else torch.from_numpy(path).cuda())
    for b in range(B):
        nodes = list(range(count[b])) if path is None else path[b, :count[b]].tolist()
        n = lens[b]
        for h in range(H):
            qq = q[b, nodes, h * G:(h + 1) * G].double().reshape(-1, D)
            kk = rows[b][0][:, h].double()
            ll = lse[b, nodes, h * G:(h + 1) * G].double().reshape(-1, 1)
            z = qq @ kk.T * D ** -0.5
            w = torch.where(torch.isinf(ll), 0.0, torch.exp(z - ll)).sum(0)
            dz = D * 2.0 ** -23 * (qq.abs() @ kk.abs().T * D ** -0.5).amax() if n else 0.0
            was = start[b, h, :n].double()
            err = (scores[b, h, :n].double() - was - w).abs()
            assert (err <= (dz + 2.0 ** -20) * w + 2.0 ** -22 * (w + was)).all(), err.max()
        assert torch.equal(scores[b, :, n:], start[b, :, n:])
    twice = start.clone()
    api.cache_scores(handle, q, lse, cache, cl, twice, torch.from_numpy(count).cuda(),
                     None if path is None else torch.from_numpy(path).cuda())
    assert torch.equal(twice, scores)
    assert handle.device_error() == 0


def test_scores_of_empty_rows_and_no_rows(handle):
    gen = torch.Generator(device="cuda").manual_seed(4)
    cache, rows = make_cache(gen, [40, 40], 2, 64, 16, 48)
    q = randn(gen, 2, 3, 4, 64)
    lse = torch.zeros(2, 3, 4, device="cuda")
    lse[0] = -math.inf                     # queries that saw nothing add nothing
    q[1, 2] = NAN                          # a rejected node's query is not looked at
    scores = torch.ones(2, 2, 48, device="cuda")
    cl = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    api.cache_scores(handle, q, lse, cache, cl, scores, torch.tensor([3, 0], dtype=torch.int32, device="cuda"))
    assert (scores == 1.0).all()
    api.cache_scores(handle, q, lse, cache, cl, scores, torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    assert (scores[0] == 1.0).all() and (scores[1, :, :40] > 1.0).all() and (scores[1, :, 40:] == 1.0).all()
    assert handle.device_error() == 0
    # path entries outside the block are clamped and flagged, lengths past the scores' rows too
    path = torch.tensor([[5, 0, 0], [-3, 0, 0]], dtype=torch.int32, device="cuda")
    api.cache_scores(handle, q, lse, cache, cl, scores, torch.ones(2, dtype=torch.int32, device="cuda"), path)
    assert handle.device_error() == api.DEVERR_BAD_NODE
    short = torch.ones(2, 2, 30, device="cuda")
    api.cache_scores(handle, q, lse, cache, cl, short, torch.ones(2, dtype=torch.int32, device="cuda"))
    assert handle.device_error() == api.DEVERR_BAD_LENGTH


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def kept_reference(scores, n, keep, recent):
    """Positions kept of one head: value descending, NaN last, ties by lowest position."""
    if n <= keep:
        return list(range(n))
    s = scores.astype(np.float64)
    key = [(-math.inf if math.isnan(x) else x, not math.isnan(x)) for x in s[:n - recent]]
    order = sorted(range(n - recent), key=lambda j: (not key[j][1], -key[j][0], j))
    return sorted(order[:keep - recent]) + list(range(n - recent, n))


@pytest.mark.parametrize("lens,H,D,page,keep,recent,kind", [
    ([1], 1, 64, 16, 1, 0, "normal"), ([2, 1, 0], 2, 128, 16, 1, 1, "normal"),
    ([100, 50, 99, 51], 2, 64, 16, 50, 7, "ties"), ([5000, 4097], 3, 128, 64, 1001, 100, "normal"),
    ([3000], 8, 128, 0, 2999, 0, "equal"), ([2500, 100], 1, 64, 32, 128, 128, "ties"),
    ([40000, 20000], 2, 64, 64, 7000, 64, "heavy"), ([1500], 2, 128, 128, 400, 3, "odd")])
def test_evict(handle, lens, H, D, page, keep, recent, kind):
    gen = torch.Generator(device="cuda").manual_seed(keep)
    rng = np.random.default_rng(keep)
    B = len(lens)
    cap = max(lens) + 5
    cache, rows = make_cache(gen, lens, H, D, page, cap)
    s = {"normal": lambda: rng.standard_normal((B, H, cap)), "equal": lambda: np.zeros((B, H, cap)),
         "ties": lambda: rng.integers(-2, 3, (B, H, cap)) * 0.5,
         "heavy": lambda: rng.exponential(1.0, (B, H, cap)) ** 8,
         "odd": lambda: rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3.0], (B, H, cap))
         }[kind]().astype(np.float32)
    dst, _ = make_cache(gen, [0] * B, H, D, page, keep)
    scores = torch.from_numpy(s).cuda()
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    before = cache.k.clone()
    out_scores = torch.full((B, H, keep + 3), -9.0, device="cuda")
    kept, new_len, ds = api.cache_evict(handle, scores, cache, cl, dst, keep, recent, dst_scores=out_scores)
    assert new_len.tolist() == [min(n, keep) for n in lens]
    for b in range(B):
        m = min(lens[b], keep)
        dk, dv = read_rows(dst, b, m)
        for h in range(H):
            want = kept_reference(s[b, h], lens[b], keep, recent)
            assert kept[b, h].tolist() == want + [-1] * (keep - m)
            w = torch.tensor(want, dtype=torch.long, device="cuda")
            assert torch.equal(dk[:, h], rows[b][0][w, h]) and torch.equal(dv[:, h], rows[b][1][w, h])
            assert torch.equal(ds[b, h, :m].view(torch.int32), scores[b, h, w].view(torch.int32))
            assert (ds[b, h, m:] == -9.0).all()
        # nothing past the new length was written
        if m < dst.capacity:
            rest = read_rows(dst, b, dst.capacity)[0][m:]
            assert torch.isnan(rest).all()
    assert torch.equal(cache.k.view(torch.int16), before.view(torch.int16))
    assert handle.device_error() == 0


def test_evict_flags_bad_lengths_and_pages(handle):
    gen = torch.Generator(device="cuda").manual_seed(2)
    cache, rows = make_cache(gen, [64], 1, 64, 16, 64)
    dst, _ = make_cache(gen, [0], 1, 64, 16, 16)
    scores = torch.rand(1, 1, 64, device="cuda", generator=gen)
    _, n, _ = api.cache_evict(handle, scores, cache, torch.tensor([65], dtype=torch.int32, device="cuda"), dst, 16, 4)
    assert n.tolist() == [16] and handle.device_error() == api.DEVERR_BAD_LENGTH
    cl = torch.tensor([64], dtype=torch.int32, device="cuda")
    dst.block_table[0, 0] = 12345
    before = dst.k.clone()
    api.cache_evict(handle, scores, cache, cl, dst, 16, 4)
    assert handle.device_error() == api.DEVERR_BAD_PAGE
    assert torch.equal(dst.k.view(torch.int16), before.view(torch.int16))


# ---------------------------------------------------------------------------
# refusals, streams, layout
# ---------------------------------------------------------------------------
def test_refusals_launch_nothing(handle):
    gen = torch.Generator(device="cuda").manual_seed(1)
    cache, _ = make_cache(gen, [20], 2, 64, 16, 32)
    q, kn, vn = randn(gen, 1, 2, 4, 64), randn(gen, 1, 2, 2, 64), randn(gen, 1, 2, 2, 64)
    cl = torch.tensor([20], dtype=torch.int32, device="cuda")
    out = torch.full((1, 2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")

    def status(fn):
        with pytest.raises(api.Dflash2Error) as e:
            fn()
        return e.value.status

    att = lambda q=q, cache=cache, **kw: api.tree_attention(handle, q, cache, cl, kn, vn, out=out, **kw)  # noqa: E731
    for bad in (0.0, -1.0, NAN, math.inf):
        assert status(lambda: att(scale=bad)) == -1
    assert status(lambda: att(workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))) == -7
    odd = api.KVCache(cache.k.flatten()[:10 * 12 * 2 * 64 // 10].view(1, 12, 2, 64),
                      cache.v.flatten()[:12 * 2 * 64].view(1, 12, 2, 64), torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    assert status(lambda: att(cache=odd)) == -2                       # pages of 12
    wide = randn(gen, 1, 2, 4, 65)
    shifted = wide.flatten()[1:1 + 512].view(1, 2, 4, 64)
    assert status(lambda: att(q=shifted)) == -3                       # 2 bytes off
    skew = torch.empty(2 * 4 * 68, dtype=torch.bfloat16, device="cuda").as_strided((1, 2, 4, 64), (544, 272, 68, 1))
    assert status(lambda: att(q=skew)) == -3                          # a stride that is no multiple of 8
    for name in ("q", "lse", "tree_mask"):
        with pytest.raises(ValueError):
            att(**{name: torch.zeros(3, device="cuda")})
    with pytest.raises(ValueError):
        api.tree_attention(handle, q, cache, cl, kn, None)
    with pytest.raises(ValueError):
        api.tree_attention(handle, q, cache, cl.long(), kn, vn)
    big = randn(gen, 1, 129, 4, 64)
    assert status(lambda: api.tree_attention(handle, big, cache, cl)) == -2
    assert status(lambda: api.tree_attention(handle, randn(gen, 1, 1, 3, 64), cache, cl)) == -1
    assert status(lambda: api.cache_commit(handle, kn, vn, cache, cl, new_len=cl)) == -1
    scores = torch.zeros(1, 2, 32, device="cuda")
    dst, _ = make_cache(gen, [0], 2, 64, 16, 16)
    for keep, recent in ((17, 0), (4, 5), (4, -1), (0, 0)):
        assert status(lambda: api.cache_evict(handle, scores, cache, cl, dst, keep, recent)) == -1
    other, _ = make_cache(gen, [0], 1, 64, 16, 16)
    assert status(lambda: api.cache_evict(handle, scores, cache, cl, other, 4, 1)) == -1
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    assert handle.device_error() == 0


def test_another_stream_and_empty_batches(handle):
    gen = torch.Generator(device="cuda").manual_seed(12)
    cache, rows = make_cache(gen, [300], 2, 128, 16, 310)
    q, kn, vn = randn(gen, 1, 17, 8, 128), randn(gen, 1, 17, 2, 128), randn(gen, 1, 17, 2, 128)
    cl = torch.tensor([300], dtype=torch.int32, device="cuda")
    want = api.tree_attention(handle, q, cache, cl, kn, vn)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [api.tree_attention(handle, q, cache, cl, kn, vn, stream=side) for _ in range(3)]
    side.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    none = api.tree_attention(handle, q[:0], cache, cl[:0], kn[:0], vn[:0])
    assert none[0].shape == (0, 17, 8, 128)
    assert api.cache_commit(handle, kn[:, :0], vn[:, :0], cache, cl).tolist() == [300]
    assert handle.device_error() == 0


def test_a_pool_past_32_bits(handle):
    # the last pages of a pool of more than 2^32 elements per tensor (and of 2^33 bytes)
    gen = torch.Generator(device="cuda").manual_seed(13)
    pages = (1 << 32) // (64 * 8 * 128) + 8
    k = torch.empty(pages, 64, 8, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[pages - 1, 3, pages - 3]], dtype=torch.int32, device="cuda")
    cache = api.KVCache(k, v, table)
    rows = [(randn(gen, 150, 8, 128), randn(gen, 150, 8, 128))]
    write_rows(cache, 0, 0, *rows[0])
    cl = torch.tensor([150], dtype=torch.int32, device="cuda")
    kn, vn = randn(gen, 1, 4, 8, 128), randn(gen, 1, 4, 8, 128)
    q = randn(gen, 1, 4, 16, 128)
    n = api.cache_commit(handle, kn, vn, cache, cl)
    rows = [(torch.cat([rows[0][0], kn[0]]), torch.cat([rows[0][1], vn[0]]))]
    got = api.tree_attention(handle, q, cache, n)
    check_attention(got, reference(q, rows, None, None, None, 128 ** -0.5))
    scores = torch.zeros(1, 8, 192, device="cuda")
    api.cache_scores(handle, q, got[1], cache, n, scores)
    assert torch.allclose(scores.sum(-1), torch.full((1, 8), 8.0, device="cuda"), rtol=1e-5)   # 4 nodes x 2 heads
    dst = api.KVCache(k, v, torch.tensor([[pages - 2]], dtype=torch.int32, device="cuda"))
    kept, m, _ = api.cache_evict(handle, scores, cache, n, dst, 64, 10)
    dk, dv = read_rows(dst, 0, 64)
    for h in range(8):
        w = kept[0, h].long()
        assert torch.equal(dk[:, h], rows[0][0][w, h]) and torch.equal(dv[:, h], rows[0][1][w, h])
    assert m.tolist() == [64] and handle.device_error() == 0


@pytest.mark.parametrize("lens,T,heads,H,D", [([100000, 70001], 1, 16, 8, 64), ([60000, 90000], 3, 8, 8, 128),
                                              ([30000], 40, 32, 8, 128)])
def test_long_runs(handle, lens, T, heads, H, D):
    # tens of tiles per CTA: the two pipelines drift apart within the ring
    gen = torch.Generator(device="cuda").manual_seed(14)
    B = len(lens)
    cache, rows = make_cache(gen, lens, H, D, 0, max(lens))
    q, kn, vn = randn(gen, B, T, heads, D), randn(gen, B, T, H, D), randn(gen, B, T, H, D)
    sees = np.tril(np.ones((T, T), bool))[None].repeat(B, 0)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = api.tree_attention(handle, q, cache, cl, kn, vn)
    for _ in range(3):
        again = api.tree_attention(handle, q, cache, cl, kn, vn)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    check_attention(got, reference(q, rows, kn, vn, sees, D ** -0.5))
    assert handle.device_error() == 0


@pytest.mark.parametrize("n,keep,recent", [(3000, 1500, 0), (60000, 30000, 10), (300000, 123457, 4000)])
def test_evict_where_most_scores_are_equal(handle, n, keep, recent):
    # thousands of equal scores around the threshold: ties go to the lowest positions
    gen = torch.Generator(device="cuda").manual_seed(n)
    rng = np.random.default_rng(n)
    s = np.where(rng.random((1, 2, n)) < 0.2, rng.standard_normal((1, 2, n)), 0.25).astype(np.float32)
    cache, rows = make_cache(gen, [n], 2, 64, 0, n)
    dst, _ = make_cache(gen, [0], 2, 64, 0, keep)
    cl = torch.tensor([n], dtype=torch.int32, device="cuda")
    kept, _, _ = api.cache_evict(handle, torch.from_numpy(s).cuda(), cache, cl, dst, keep, recent)
    for h in range(2):
        x = s[0, h, :n - recent]
        order = np.lexsort((np.arange(n - recent), -x.astype(np.float64)))[:keep - recent]
        want = np.concatenate([np.sort(order), np.arange(n - recent, n)])
        assert np.array_equal(kept[0, h].cpu().numpy(), want)
        w = torch.from_numpy(want).cuda()
        assert torch.equal(dst.k[0, :keep, h], rows[0][0][w, h])
    assert handle.device_error() == 0


@pytest.mark.parametrize("lens,cap,T,heads,H,D", [([100, 0, 17], 100, 1, 8, 4, 128), ([128] * 40, 128, 17, 16, 2, 64),
                                                  ([128, 120], 128, 40, 32, 4, 128)])
def test_short_caches_are_taken_whole(handle, lens, cap, T, heads, H, D):
    gen = torch.Generator(device="cuda").manual_seed(T)
    B = len(lens)
    cache, rows = make_cache(gen, lens, H, D, 0, cap)
    q, kn, vn = randn(gen, B, T, heads, D), randn(gen, B, T, H, D), randn(gen, B, T, H, D)
    sees = np.tril(np.ones((T, T), bool))[None].repeat(B, 0)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    check_attention(api.tree_attention(handle, q, cache, cl, kn, vn), reference(q, rows, kn, vn, sees, D ** -0.5))
    assert handle.device_error() == 0


def test_refusals_of_what_passes_the_counters(handle):
    # 2^24 tiles of 128 keys a sequence, 4 kv heads, 64 sequences: 2^32 units
    k = torch.zeros(4, 128, 4, 64, dtype=torch.bfloat16, device="cuda")
    cache = api.KVCache(k, k.clone(), torch.zeros(64, 4, dtype=torch.int32, device="cuda"))
    cache.struct.max_pages = cache.struct.table_ld = (1 << 24) - 2
    q = torch.zeros(64, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    cl = torch.zeros(64, dtype=torch.int32, device="cuda")
    with pytest.raises(api.Dflash2Error) as e:
        api.tree_attention(handle, q, cache, cl)
    assert e.value.status == -2
    with pytest.raises(api.Dflash2Error) as e:
        api.cache_scores(handle, q, torch.zeros(64, 1, 4, device="cuda"), cache, cl, torch.zeros(64, 4, 8, device="cuda"))
    assert e.value.status == -2
    cache.struct.max_pages = 1 << 24                     # a capacity of 2^31
    with pytest.raises(api.Dflash2Error) as e:
        api.tree_attention(handle, q[:1], cache, cl[:1])
    assert e.value.status == -2
    assert handle.device_error() == 0


@pytest.mark.parametrize("T,heads,H", [(48, 16, 2), (65, 8, 1), (112, 16, 2), (128, 8, 1), (9, 128, 1), (128, 64, 1)])
def test_row_tiles_with_runs_of_their_own(handle, T, heads, H):
    # 3, 5, 7, 8, 9 and 64 row tiles: pairs beside one another, a single tile left over, too many pairs to deal out
    gen = torch.Generator(device="cuda").manual_seed(T)
    lens = [6000, 0, 1, 2511]
    B = len(lens)
    cache, rows = make_cache(gen, lens, H, 128, 64, 6000)
    q, kn, vn = randn(gen, B, T, heads, 128), randn(gen, B, T, H, 128), randn(gen, B, T, H, 128)
    sees = np.tril(np.ones((T, T), bool))[None].repeat(B, 0)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = api.tree_attention(handle, q, cache, cl, kn, vn)
    again = api.tree_attention(handle, q, cache, cl, kn, vn)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    check_attention(got, reference(q, rows, kn, vn, sees, 128 ** -0.5))
    assert handle.device_error() == 0


@pytest.mark.parametrize("T,heads,H,D,page,tree", [(17, 32, 4, 128, 64, False), (100, 24, 4, 64, 0, True)])
def test_scores_of_blocks_that_differ_in_accepted_nodes(handle, T, heads, H, D, page, tree):
    # enough units that runs are cut by weight: sequences of many and of few rows, empty ones among them
    lens = [4096, 0, 130, 3000, 4000, 1, 4096, 2500, 0, 129, 3583, 2048]
    test_scores(handle, lens, T, heads, H, D, page, tree)


@pytest.mark.parametrize("lens,T,heads,H,D", [([900], 1, 8, 2, 128), ([1500, 0], 17, 32, 8, 128), ([700, 1, 128, 640, 0, 511], 5, 24, 8, 64),
                                              ([1200, 300], 33, 16, 2, 128), ([129], 128, 16, 1, 64), ([260, 0], 3, 2, 1, 128)])
def test_short_items_shared_by_a_cluster(handle, lens, T, heads, H, D):
    # a few items of a few tiles: CTAs without a tile of their item, one tile each, several
    gen = torch.Generator(device="cuda").manual_seed(T + 40)
    B = len(lens)
    cache, rows = make_cache(gen, lens, H, D, 16, max(lens))
    q, kn, vn = randn(gen, B, T, heads, D), randn(gen, B, T, H, D), randn(gen, B, T, H, D)
    sees = np.tril(np.ones((T, T), bool))[None].repeat(B, 0)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = api.tree_attention(handle, q, cache, cl, kn, vn)
    again = api.tree_attention(handle, q, cache, cl, kn, vn)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    check_attention(got, reference(q, rows, kn, vn, sees, D ** -0.5))
    assert handle.device_error() == 0


@pytest.mark.parametrize("T,heads,H,D", [(5, 24, 4, 128), (33, 32, 4, 64)])
def test_many_items_cut_by_runs(handle, T, heads, H, D):
    # more items than clusters fit: equal runs cut many of them, each into a few parts
    gen = torch.Generator(device="cuda").manual_seed(T + 50)
    lens = [1000 - 37 * i for i in range(26)] + [0, 1]
    B = len(lens)
    cache, rows = make_cache(gen, lens, H, D, 32, max(lens))
    q, kn, vn = randn(gen, B, T, heads, D), randn(gen, B, T, H, D), randn(gen, B, T, H, D)
    sees = np.tril(np.ones((T, T), bool))[None].repeat(B, 0)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = api.tree_attention(handle, q, cache, cl, kn, vn)
    again = api.tree_attention(handle, q, cache, cl, kn, vn)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    check_attention(got, reference(q, rows, kn, vn, sees, D ** -0.5))
    assert handle.device_error() == 0
