"""The cache operators where weights and values are at their limits.

Definition (what a row sees: cached positions below the length, nodes of its mask):
a key with z = -inf adds nothing, whatever its value; any other key adds
exp(z - lse) value, so an infinite or NaN value of it reaches the row.

Bounds, per element, from the number formats alone (no averaging is counted on):
  z      a fp32 dot product of D terms: dz = D 2^-23 max(scale <|q|, |k|>)
  out    2^-8 |out| (one rounding to bf16, 8 significant bits) +
         (2 dz + 2^-15 + n 2^-24) A, A = sum p |v| over n keys: the weights' own error,
         weights in two bf16 terms (2^-16) and fp32 sums
  score  (dz + 2^-20) w + 2^-22 (w + what was there)
"""
import math

import pytest
import torch

from draft_selection_dflash2_gb300 import api
from gpu_common import handle  # noqa: F401
from test_gpu_cache import make_cache, randn, write_rows

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


def lengths(lens):
    return torch.tensor(lens, dtype=torch.int32, device="cuda")


def definition(q, rows, k_new, v_new, sees, scale):
    """fp64 (out, A, dz, n) of the definition above; non-finite values arrive as themselves."""
    B, T, heads, D = q.shape
    H = rows[0][0].shape[1]
    G = heads // H
    out = torch.zeros(B, T, heads, D, dtype=torch.float64, device="cuda")
    A, dz = torch.zeros_like(out), torch.zeros(B, T, heads, dtype=torch.float64, device="cuda")
    most = 0
    for b in range(B):
        for h in range(H):
            qq = q[b, :, h * G:(h + 1) * G].double().reshape(T * G, D)
            kk, vv = rows[b][0][:, h].double(), rows[b][1][:, h].double()
            vis = torch.ones(T * G, kk.shape[0], dtype=torch.bool, device="cuda")
            if k_new is not None:
                kk, vv = torch.cat([kk, k_new[b, :, h].double()]), torch.cat([vv, v_new[b, :, h].double()])
                s = torch.ones(T, T, dtype=torch.bool, device="cuda").tril() if sees is None else sees[b]
                vis = torch.cat([vis, s.repeat_interleave(G, 0)], 1)
            if kk.shape[0] == 0:
                continue
            most = max(most, kk.shape[0])
            z = qq @ kk.T * scale
            adds = vis & (z != -INF)
            z = torch.where(adds, z, -INF)
            p = torch.softmax(z, 1).nan_to_num(0.0)           # a row without a key that adds: 0
            o, a = p @ vv.nan_to_num(0.0, 0.0, 0.0), p @ vv.abs().nan_to_num(0.0, 0.0, 0.0)
            for j in (~torch.isfinite(vv)).any(1).nonzero().flatten().tolist():
                o += torch.where(adds[:, j:j + 1] & ~torch.isfinite(vv[j]), vv[j], 0.0)
            out[b, :, h * G:(h + 1) * G] = o.reshape(T, G, D)
            A[b, :, h * G:(h + 1) * G] = a.reshape(T, G, D)
            zabs = torch.where(adds, qq.abs() @ kk.abs().nan_to_num(0.0, 0.0, 0.0).T * scale, 0.0)
            dz[b, :, h * G:(h + 1) * G] = (D * 2.0 ** -23 * zabs.amax(1)).reshape(T, G)
    return out, A, dz, most


def check(got, want):
    ro, A, dz, n = want
    o = got.double()
    live = torch.isfinite(ro)
    assert torch.equal(torch.isnan(o), torch.isnan(ro))
    assert torch.equal(torch.where(live | torch.isnan(o), 0.0, o), torch.where(live | torch.isnan(ro), 0.0, ro))
    tol = 2.0 ** -8 * ro.abs() + (2 * dz[..., None] + 2.0 ** -15 + n * 2.0 ** -24) * A
    err = torch.where(live, o - ro, 0.0).abs()
    assert (err <= tol)[live].all(), ((err - tol)[live].max(), (err / tol)[live].nan_to_num(0.0).max())


# ---------------------------------------------------------------------------
# weights that gather on few keys
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,T,heads,H,D,keys", [
    (300, 1, 8, 8, 128, 1), (4000, 1, 8, 8, 128, 1), (4000, 1, 8, 8, 128, 2), (20000, 1, 8, 8, 64, 1),
    (20000, 1, 8, 8, 64, 2), (6000, 34, 64, 8, 128, 1), (6000, 34, 64, 8, 128, 2), (6000, 34, 64, 8, 128, 900)])
def test_weights_on_few_keys(handle, n, T, heads, H, D, keys):
    # each (sequence, head) has one key, two, or many equal ones, 3 to 8 powers of two above the first key of every
    # tile, and all others far below: with the maximum of a tile's start P is no power of two, and no error of
    # another key averages it out
    gen = torch.Generator(device="cuda").manual_seed(n + keys)
    B, G = 4, heads // H
    cache, rows = make_cache(gen, [n] * B, H, D, 64, n)
    q = randn(gen, B, 1, H, D).repeat_interleave(G, 2).repeat(1, T, 1, 1)       # a kv head's rows are alike
    above = torch.linspace(3.0, 8.0, B * H, device="cuda").reshape(B, H) * math.log(2.0)
    at = sorted({200 + (n - 250) * i // max(keys, 1) for i in range(keys)})
    for b in range(B):
        kk, vv = rows[b]
        for h in range(H):
            qh = q[b, 0, h * G].float()
            unit = qh / (qh @ qh * D ** -0.5)                  # a key with z = 1
            kk[:, h] = (-12.0 * unit).to(torch.bfloat16)
            kk[::128, h] = 0.0
            kk[at, h] = (above[b, h] * unit).to(torch.bfloat16)
        if keys == 900:
            vv[at] = vv[at[:1]]
        write_rows(cache, b, 0, kk, vv)
    out, _ = api.tree_attention(handle, q.contiguous(), cache, lengths([n] * B))
    check(out, definition(q, rows, None, None, None, D ** -0.5))
    assert handle.device_error() == 0


# ---------------------------------------------------------------------------
# infinities
# ---------------------------------------------------------------------------
SHAPES = [
    # lens, capacity, T, heads, H, D, page
    ([300], 300, 1, 8, 2, 128, 16),                 # a cluster per item, one row tile
    ([900, 140], 900, 40, 16, 2, 64, 32),           # clusters, two row tiles
    ([120] * 24, 128, 3, 16, 4, 64, 0),             # whole items
    ([128, 100], 128, 40, 32, 4, 128, 0),           # whole items of three row tiles
    ([3000, 2500, 700], 30000, 17, 16, 2, 128, 64), # runs, two row tiles
    ([1000 - 30 * i for i in range(20)], 30000, 3, 24, 4, 128, 16),   # many items, cut into a few parts each
    ([40000], 40000, 2, 8, 1, 64, 64),              # one head, many parts
]


@pytest.mark.parametrize("lens,cap,T,heads,H,D,page", SHAPES)
@pytest.mark.parametrize("drafted", [False, True])
def test_infinite_values_of_cached_keys(handle, lens, cap, T, heads, H, D, page, drafted):
    gen = torch.Generator(device="cuda").manual_seed(len(lens) + T)
    B = len(lens)
    cache, rows = make_cache(gen, lens, H, D, page, cap)
    q, kn, vn = randn(gen, B, T, heads, D), randn(gen, B, T, H, D), randn(gen, B, T, H, D)
    if not drafted:
        kn = vn = None
    finite, _ = api.tree_attention(handle, q, cache, lengths(lens), kn, vn)
    for b in range(B):
        n, (kk, vv) = lens[b], rows[b]
        vv[n // 2, :, 3] = INF
        vv[5, :, 3] = INF
        vv[n - 1, :, D - 1] = -INF
        vv[70, 0, 20] = INF                       # +inf and -inf in one column: NaN
        vv[n - 2, 0, 20] = -INF
        vv[9, H - 1, 33] = NAN
        write_rows(cache, b, 0, kk, vv)
    out, _ = api.tree_attention(handle, q, cache, lengths(lens), kn, vn)
    again, _ = api.tree_attention(handle, q, cache, lengths(lens), kn, vn)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    check(out, definition(q, rows, kn, vn, None, D ** -0.5))
    assert torch.isposinf(out[..., 3]).all() and torch.isneginf(out[..., D - 1]).all()
    assert torch.isfinite(finite).all() and handle.device_error() == 0


@pytest.mark.parametrize("lens,cap,T,heads,H,D,page", SHAPES)
def test_values_of_keys_at_minus_infinity_add_nothing(handle, lens, cap, T, heads, H, D, page):
    # cached and drafted keys whose z is -inf hold infinities and NaN
    gen = torch.Generator(device="cuda").manual_seed(len(lens) * 10 + T)
    B = len(lens)
    cache, rows = make_cache(gen, lens, H, D, page, cap)
    q, kn, vn = randn(gen, B, T, heads, D), randn(gen, B, T, H, D), randn(gen, B, T, H, D)
    q[..., 7] = q[..., 7].abs() + 0.5
    for b in range(B):
        n, (kk, vv) = lens[b], rows[b]
        for j, x in ((3, INF), (n // 2, -INF), (n - 1, NAN)):
            kk[j, :, 7] = -INF
            vv[j] = x
        write_rows(cache, b, 0, kk, vv)
    kn[:, T // 2, :, 7] = -INF
    vn[:, T // 2] = INF
    out, _ = api.tree_attention(handle, q, cache, lengths(lens), kn, vn)
    assert torch.isfinite(out).all()
    check(out, definition(q, rows, kn, vn, None, D ** -0.5))
    assert handle.device_error() == 0


@pytest.mark.parametrize("lens,cap,T,heads,H,D,page", SHAPES)
def test_an_infinity_far_below_the_maximum_arrives(handle, lens, cap, T, heads, H, D, page):
    # its weight underflows in fp32 but is not 0; the parts of a cut item meet in both orders
    gen = torch.Generator(device="cuda").manual_seed(len(lens) * 20 + T)
    B = len(lens)
    cache, rows = make_cache(gen, lens, H, D, page, cap)
    q = randn(gen, B, T, heads, D).abs() + 0.25
    for where in (0, -1):
        for b in range(B):
            n, (kk, vv) = lens[b], rows[b]
            kk[0 if where else n - 1] = 16.0      # z of 200 and more
            vv[where % n, :, 11] = -INF
            write_rows(cache, b, 0, kk, vv)
        out, _ = api.tree_attention(handle, q, cache, lengths(lens))
        check(out, definition(q, rows, None, None, None, D ** -0.5))
        assert torch.isneginf(out[..., 11]).all()
        for b in range(B):
            rows[b][0].copy_(randn(gen, *rows[b][0].shape))
            rows[b][1].copy_(randn(gen, *rows[b][1].shape))
    assert handle.device_error() == 0


@pytest.mark.parametrize("lens,cap,T,heads,H,D,page", SHAPES)
def test_values_near_the_largest(handle, lens, cap, T, heads, H, D, page):
    # one key takes nearly all the weight; its value times what P may reach would pass the type's range
    gen = torch.Generator(device="cuda").manual_seed(len(lens) * 30 + T)
    B = len(lens)
    cache, rows = make_cache(gen, lens, H, D, page, cap)
    q = randn(gen, B, T, heads, D).abs() + 0.25
    for b in range(B):
        kk, vv = rows[b]
        kk.mul_(0.01)
        j = min(100, lens[b] - 1)
        kk[j] = 4.6 / D ** 0.5 / q.float().mean().item()      # P of about 2^6.6 where the tile's start set the maximum
        vv[j] = 3.0e38
        vv[j, :, 1] = -3.0e38
        write_rows(cache, b, 0, kk, vv)
    out, _ = api.tree_attention(handle, q, cache, lengths(lens))
    assert torch.isfinite(out).all()
    check(out, definition(q, rows, None, None, None, D ** -0.5))
    assert handle.device_error() == 0


def test_rows_that_see_only_infinite_nodes_at_minus_infinity(handle):
    # nothing is added: out = 0 and lse = -inf, beside rows that see more
    gen = torch.Generator(device="cuda").manual_seed(2)
    for T, lens in ((3, [0, 0]), (40, [0, 200])):
        cache, rows = make_cache(gen, lens, 2, 64, 16, 208)
        q, kn, vn = randn(gen, 2, T, 16, 64), randn(gen, 2, T, 2, 64), randn(gen, 2, T, 2, 64)
        q[..., 7] = q[..., 7].abs() + 0.5
        kn[:, 0, :, 7] = -INF
        vn[:, 0] = INF
        out, lse = api.tree_attention(handle, q, cache, lengths(lens), kn, vn)
        assert (out[0, 0] == 0).all() and torch.isneginf(lse[0, 0]).all() and torch.isfinite(out).all()
        check(out, definition(q, rows, kn, vn, None, 0.125))
    assert handle.device_error() == 0


# ---------------------------------------------------------------------------
# scores
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,heads,H,D", [(1, 8, 1, 128), (2, 16, 1, 64), (5, 6, 2, 64), (17, 16, 2, 128)])
def test_scores_of_infinite_keys(handle, T, heads, H, D):
    # keys with z = -inf for every query, row counts that are and are not multiples of 16, queries that saw nothing
    gen = torch.Generator(device="cuda").manual_seed(T)
    G, n = heads // H, 150
    cache, rows = make_cache(gen, [n], H, D, 16, n)
    q = randn(gen, 1, T, heads, D)
    q[..., 7] = q[..., 7].abs() + 0.5
    kk, vv = rows[0]
    dead = [0, 3, 127, 128, n - 1]
    kk[dead, :, 7] = -INF
    write_rows(cache, 0, 0, kk, vv)
    _, lse = api.tree_attention(handle, q, cache, lengths([n]))
    assert torch.isfinite(lse).all()
    start = torch.rand(1, H, n, generator=gen, device="cuda")
    for empty in (None, 0, T - 1):
        if empty is not None:
            lse[0, empty] = -INF
        scores = start.clone()
        api.cache_scores(handle, q, lse, cache, lengths([n]), scores)
        for h in range(H):
            qq = q[0, :, h * G:(h + 1) * G].double().reshape(-1, D)
            ll = lse[0, :, h * G:(h + 1) * G].double().reshape(-1, 1)
            z = qq @ kk[:, h].double().T * D ** -0.5
            w = torch.where(torch.isinf(ll), 0.0, torch.exp(z - ll)).sum(0)
            assert (w[dead] == 0).all()
            kabs = kk[:, h].double().abs().nan_to_num(0.0, 0.0, 0.0)
            zabs = torch.where(torch.isinf(z), 0.0, qq.abs() @ kabs.T * D ** -0.5)
            dz, was = D * 2.0 ** -23 * zabs.amax(), start[0, h].double()
            err = (scores[0, h].double() - was - w).abs()
            assert (err <= (dz + 2.0 ** -20) * w + 2.0 ** -22 * (w + was)).all(), err.max()
    assert handle.device_error() == 0


@pytest.mark.parametrize("T,heads", [(1, 8), (2, 16)])
def test_scores_of_what_attention_found_empty(handle, T, heads):
    # a cache whose keys put every z at -inf: attention leaves lse = -inf, and nothing is added with it
    cache, rows = make_cache(torch.Generator(device="cuda").manual_seed(1), [140], 1, 64, 16, 140)
    rows[0][0][:] = -INF
    write_rows(cache, 0, 0, *rows[0])
    q = torch.ones(1, T, heads, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = api.tree_attention(handle, q, cache, lengths([140]))
    assert (out == 0).all() and torch.isneginf(lse).all()
    scores = torch.full((1, 1, 140), 2.0, device="cuda")
    api.cache_scores(handle, q, lse, cache, lengths([140]), scores)
    assert (scores == 2.0).all() and handle.device_error() == 0


@pytest.mark.parametrize("B,n,T,heads,H,D", [(40, 128, 1, 32, 16, 128), (60, 100, 17, 32, 16, 64),
                                             (33, 129, 3, 60, 20, 128)])
def test_scores_of_many_short_heads(handle, B, n, T, heads, H, D):
    # runs of several (sequence, head) of one tile each: an issuer of products is idle in every other one
    gen = torch.Generator(device="cuda").manual_seed(B)
    G = heads // H
    lens = [n - 7 * b % 30 for b in range(B)]
    cache, rows = make_cache(gen, lens, H, D, 0, n)
    q = randn(gen, B, T, heads, D)
    _, lse = api.tree_attention(handle, q, cache, lengths(lens))
    first = None
    for _ in range(20):
        scores = torch.zeros(B, H, n, device="cuda")
        api.cache_scores(handle, q, lse, cache, lengths(lens), scores)
        first = scores if first is None else first
        assert torch.equal(scores, first)
    for b in range(B):
        qq = q[b].double().reshape(T, H, G, D)
        z = torch.einsum("thgd,jhd->hjtg", qq, rows[b][0].double()) * D ** -0.5
        w = torch.exp(z - lse[b].double().reshape(T, H, 1, G).permute(1, 2, 0, 3)).sum((2, 3))
        dz = D * 2.0 ** -23 * torch.einsum("thgd,jhd->hjtg", qq.abs(), rows[b][0].double().abs()).max() * D ** -0.5
        assert ((first[b, :, :lens[b]].double() - w).abs() <= (dz + 2.0 ** -20) * w + 2.0 ** -22 * w).all()
        assert (first[b, :, lens[b]:] == 0).all()
    assert handle.device_error() == 0


# ---------------------------------------------------------------------------
# buffers that may not be shared
# ---------------------------------------------------------------------------
def test_outputs_that_overlap_inputs_are_refused(handle):
    # a CTA would read what another one of the same sequence has written
    gen = torch.Generator(device="cuda").manual_seed(1)
    cache, _ = make_cache(gen, [8, 8], 2, 64, 16, 32)
    dst, _ = make_cache(gen, [0, 0], 2, 64, 16, 16)
    kn, vn = randn(gen, 2, 4, 2, 64), randn(gen, 2, 4, 2, 64)
    ints = torch.tensor([8, 8, 3, 3, 0, 0], dtype=torch.int32, device="cuda")
    floats = torch.zeros(2 * 2 * 32 + 2 * 2 * 16, device="cuda")
    scores = floats[:128].view(2, 2, 32)
    before = cache.k.clone()

    def refused(fn):
        with pytest.raises(api.Dflash2Error) as e:
            fn()
        assert e.value.status == -1

    def commit(new):
        return api.cache_commit(handle, kn, vn, cache, ints[:2], ints[2:4], new_len=new)

    def evict(new, ds):
        return api.cache_evict(handle, scores, cache, ints[:2], dst, 4, 1, new_len=new, dst_scores=ds)

    for new in (ints[:2], ints[1:3], ints[2:4], ints[3:5]):
        refused(lambda: commit(new))
    refused(lambda: evict(ints[1:3], None))
    refused(lambda: evict(ints[4:], floats[64:128].view(2, 2, 16)))
    refused(lambda: evict(ints[4:], floats[127:191].view(2, 2, 16)))
    torch.cuda.synchronize()
    assert torch.equal(cache.k.view(torch.int16), before.view(torch.int16)) and ints.tolist() == [8, 8, 3, 3, 0, 0]
    assert commit(ints[4:]).tolist() == [11, 11]
    assert evict(ints[4:], floats[128:].view(2, 2, 16))[1].tolist() == [4, 4]
    assert handle.device_error() == 0


@pytest.mark.parametrize("lens,T,heads,H,D", [([500], 1, 8, 2, 128), ([100, 0, 17], 40, 32, 4, 64)])
def test_a_capacity_far_above_the_lengths(handle, lens, T, heads, H, D):
    # how a call is cut goes by the capacity: clusters and whole items for a tight one, runs for a table of 65536 positions
    gen = torch.Generator(device="cuda").manual_seed(T)
    B = len(lens)
    tight, rows = make_cache(gen, lens, H, D, 64, max(lens))
    table = torch.full((B, 1024), -1, dtype=torch.int32, device="cuda")     # entries past a length are not looked at
    table[:, :tight.block_table.shape[1]] = tight.block_table
    q, kn, vn = randn(gen, B, T, heads, D), randn(gen, B, T, H, D), randn(gen, B, T, H, D)
    want = definition(q, rows, kn, vn, None, D ** -0.5)
    for cache in (tight, api.KVCache(tight.k, tight.v, table)):
        out, lse = api.tree_attention(handle, q, cache, lengths(lens), kn, vn)
        check(out, want)
        scores = torch.zeros(B, H, 512, device="cuda")
        api.cache_scores(handle, q, lse, cache, lengths(lens), scores)
        # a row's weights on the cache and on the block's own nodes are 1 together
        total = scores.sum((1, 2)).double()
        for b in range(B):
            z = torch.einsum("thgd,jhd->thgj", q[b].double().reshape(T, H, -1, D), rows[b][0].double()) * D ** -0.5
            w = torch.exp(z - lse[b].double().reshape(T, H, -1, 1)).sum()
            assert (total[b] - w).abs() <= 1e-4 * w
    assert handle.device_error() == 0
