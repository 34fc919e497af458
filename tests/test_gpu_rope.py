"""Rotary positions and the append of rotated keys, against 64-bit arithmetic.

Tolerance: one rounding to bf16, 2^-8 |y|, and what fp32 loses before it: the angle's fraction of a turn is rounded to
2^-32 turns and to 24 bits (2^-25 of half a turn: pi 2^-25 rad), sincospif is off by at most 2 ulp (2^-23), the factor,
two products and a sum by 2^-24 each: together below 2^-21 (|x1| + |x2|) factor."""
import math

import numpy as np
import pytest

from draft_selection_dflash2_gb300 import api
from gpu_common import handle, torch  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rates(rd, theta, scaling=None):
    """Radians per position, as the header defines them (plain loops)."""
    got = []
    for i in range(rd // 2):
        f = theta ** (-2 * i / rd)
        s = scaling or {"kind": "none"}
        if s["kind"] == "linear":
            f /= s["factor"]
        elif s["kind"] == "ntk":
            f = (theta * s["factor"] ** (rd / (rd - 2))) ** (-2 * i / rd)
        elif s["kind"] == "yarn":
            def index(n):
                return rd * math.log(s["original"] / (2 * math.pi * n)) / (2 * math.log(theta))
            lo, hi = max(math.floor(index(s["fast"])), 0), min(math.ceil(index(s["slow"])), rd - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0), 1)
            f = f * (r / s["factor"] + 1 - r)
        elif s["kind"] == "wavelength":
            t = (s["original"] * f / (2 * math.pi) - s["low"]) / (s["high"] - s["low"])
            t = min(max(t, 0), 1)
            f = (1 - t) * f / s["factor"] + t * f
        got.append(f)
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def rotated(x, pos, rd, inter, f, factor=1.0, inverse=False):
    """(y, tolerance) in 64 bits; x [B, T, H, D], pos int64 [B, T].  The angle is reduced exactly enough: far positions are
    split so that each product keeps 64 bits' precision."""
    hi, lo = pos // 65536 * 65536, pos % 65536
    turn = 2 * math.pi
    a = (torch.remainder(hi.double()[..., None] * f, turn) + torch.remainder(lo.double()[..., None] * f, turn))[:, :, None]
    if inverse:
        a = -a
    c, s = a.cos() * factor, a.sin() * factor
    y = x.double()
    one, two = (y[..., 0:rd:2], y[..., 1:rd:2]) if inter else (y[..., :rd // 2], y[..., rd // 2:rd])
    both = torch.stack([one * c - two * s, two * c + one * s], -1)
    size = (one.abs() + two.abs()) * factor
    tol = torch.zeros_like(y)
    if inter:
        y[..., :rd], tol[..., :rd] = both.flatten(-2), size.repeat_interleave(2, -1)
    else:
        y[..., :rd], tol[..., :rd] = torch.cat([both[..., 0], both[..., 1]], -1), torch.cat([size, size], -1)
    # a far position's angle in 64 bits is itself off by 2^-52 of it
    far = 2.0 ** -52 * float(pos.abs().max()) if pos.numel() else 0.0
    return y, tol * (2.0 ** -21 + far) + y.abs() * 2.0 ** -8 * (tol > 0)


def check(got, want, tol, what=""):
    bad = ~((got.double() - want).abs() <= tol) & ~(got.double() == want)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float((got.double() - want).abs().max())}"


@pytest.mark.parametrize("B,T,H,D,rd,inter", [
    (1, 1, 1, 64, 64, False), (1, 1, 40, 128, 128, True), (3, 5, 7, 128, 64, False), (2, 17, 9, 80, 20, False),
    (2, 17, 9, 80, 40, True), (2, 3, 5, 96, 24, False), (2, 3, 5, 72, 72, False), (1, 2, 3, 8, 2, False), (1, 2, 3, 8, 2, True),
    (2, 2, 2, 512, 512, False), (2, 3, 2, 88, 6, True), (40, 130, 3, 128, 128, False), (7, 801, 2, 64, 32, True),
    (1, 3, 90, 256, 256, True)])
def test_rope(handle, B, T, H, D, rd, inter):
    g = torch.Generator(device="cuda").manual_seed(B * 1000 + T)
    x = torch.randn(B, T, H + 2, D, generator=g, device="cuda").to(BF)[:, :, 1:H + 1]
    base = torch.randint(-1000, 200000, (B,), generator=g, device="cuda", dtype=torch.int32)
    depth = torch.randint(0, 50, (B, T), generator=g, device="cuda", dtype=torch.int32)
    r, f = api.Rope(rd, theta=10000.0, interleaved=inter), rates(rd, 10000.0)
    for dep, inverse in ((None, False), (depth, False), (depth, True)):
        pos = base[:, None].long() + (torch.arange(T, device="cuda")[None] if dep is None else dep.long())
        got = api.rope(handle, x, r, base, dep, inverse=inverse)
        check(got, *rotated(x, pos, rd, inter, f, inverse=inverse))
    # no base, and in place
    want = api.rope(handle, x, r)
    check(want, *rotated(x, torch.arange(T, device="cuda")[None].expand(B, T), rd, inter, f))
    around = x.clone()
    whole = torch.full((B, T, H + 2, D), 7.0, dtype=BF, device="cuda")
    whole[:, :, 1:H + 1] = around
    view = whole[:, :, 1:H + 1]
    assert api.rope(handle, view, r, out=view) is view
    assert torch.equal(view, want) and (whole[:, :, 0] == 7).all() and (whole[:, :, -1] == 7).all()
    assert handle.device_error() == 0


@pytest.mark.parametrize("scaling", [
    {"kind": "linear", "factor": 4.0}, {"kind": "ntk", "factor": 3.0}, {"kind": "yarn", "factor": 4.0, "original": 4096},
    {"kind": "yarn", "factor": 16.0, "original": 2048, "fast": 16.0, "slow": 2.0},
    {"kind": "wavelength", "factor": 8.0, "original": 8192, "low": 1.0, "high": 4.0}])
@pytest.mark.parametrize("theta", [10000.0, 1000000.0])
def test_scaled_rates(handle, scaling, theta):
    r = api.Rope(128, theta=theta, scaling=scaling)
    full = {"fast": 32.0, "slow": 1.0, **scaling}
    want_factor = 0.1 * math.log(scaling["factor"]) + 1 if scaling["kind"] == "yarn" else 1.0
    assert r.factor == pytest.approx(want_factor, rel=1e-6)
    x = torch.randn(2, 9, 3, 128, device="cuda").to(BF)
    base = torch.tensor([0, 500000], dtype=torch.int32, device="cuda")
    pos = base[:, None].long() + torch.arange(9, device="cuda")
    check(api.rope(handle, x, r, base), *rotated(x, pos, 128, False, rates(128, theta, full), r.factor))


def test_far_positions_and_special_values(handle):
    """Angles at the ends of int32; NaN and infinities stay in their pairs, and the rest of the head is copied bit by bit."""
    x = torch.randn(4, 2, 2, 128, device="cuda").to(BF)
    base = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 1 << 30], dtype=torch.int32, device="cuda")
    r = api.Rope(64)
    pos = base[:, None].long() + torch.arange(2, device="cuda")
    check(api.rope(handle, x, r, base), *rotated(x, pos, 64, False, rates(64, 10000.0)))
    bits = x.view(torch.int16)
    bits[..., 64:] = torch.randint(-2 ** 15, 2 ** 15, bits[..., 64:].shape, device="cuda", dtype=torch.int16)
    x[0, 0, 0, 3] = float("nan")
    x[0, 0, 1, 5] = float("inf")
    y = api.rope(handle, x, r, base)
    assert torch.equal(y.view(torch.int16)[..., 64:], bits[..., 64:])
    odd = ~torch.isfinite(y[..., :64].float())
    want = torch.zeros_like(odd)
    want[0, 0, 0, [3, 35]] = True
    want[0, 0, 1, [5, 37]] = True
    assert torch.equal(odd, want)


def test_the_inverse_is_the_gradient(handle):
    """<g, R x> = <R^T g, x> for every pair, and R^T by differences of the 64-bit form."""
    B, T, H, D = 2, 3, 2, 64
    x = torch.randn(B, T, H, D, device="cuda").to(BF)
    grad = torch.randn(B, T, H, D, device="cuda").to(BF)
    base = torch.tensor([5, 70000], dtype=torch.int32, device="cuda")
    scaling = {"kind": "yarn", "factor": 4.0, "original": 4096}
    for inter in (False, True):
        r = api.Rope(32, interleaved=inter, scaling=scaling)
        f = rates(32, 10000.0, {"fast": 32.0, "slow": 1.0, **scaling})
        pos = base[:, None].long() + torch.arange(T, device="cuda")
        got = api.rope(handle, grad, r, base, inverse=True)
        check(got, *rotated(grad, pos, 32, inter, f, r.factor, inverse=True))
        # by differences: the map is linear, so a step of 1 in one input is exact
        for e in (0, 1, 15, 16, 31, 32, 63):
            step = x.double()
            step[..., e] += 1.0
            d = rotated(step, pos, 32, inter, f, r.factor)[0] - rotated(x, pos, 32, inter, f, r.factor)[0]
            want = (d * grad.double()).sum(-1)
            tol = 2.0 ** -8 * want.abs() + 2.0 ** -20 * (d.abs() * grad.double().abs()).sum(-1) + 1e-9
            assert ((got[..., e].double() - want).abs() <= tol).all()


def test_empty_calls_and_refusals(handle):
    r = api.Rope(64)
    for shape in ((0, 3, 2, 64), (2, 0, 2, 64), (2, 3, 0, 64)):
        assert api.rope(handle, torch.zeros(shape, dtype=BF, device="cuda"), r).shape == shape
    x = torch.zeros(2, 3, 4, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        api.rope(handle, x.float(), r)
    with pytest.raises(ValueError):
        api.rope(handle, x, r, out=x[:, :2])
    with pytest.raises(ValueError):
        api.rope(handle, x, r, base=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        api.rope(handle, x, r, base=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        api.rope(handle, x.cpu(), r, out=x)
    with pytest.raises(api.Dflash2Error):                       # ranges that only overlap
        api.rope(handle, x[:, :2], r, out=x[:, 1:])
    with pytest.raises(api.Dflash2Error):                       # more than the head
        api.rope(handle, torch.zeros(1, 1, 1, 32, dtype=BF, device="cuda"), r)
    with pytest.raises(api.Dflash2Error):                       # rows not 16 bytes apart
        api.rope(handle, torch.zeros(1, 2, 2, 65, dtype=BF, device="cuda")[..., :64], r)
    assert handle.device_error() == 0


# ------------------------------------------------------------------------------------------- append
def pool(B, capacity, page, H, D, seed=0):
    """Cache with random contents, and its slots' places: [B, capacity] page and row."""
    rng = np.random.default_rng(seed)
    if page == 0:
        k = torch.randn(B, capacity, H, D, device="cuda").to(BF)
        v = torch.randn(B, capacity, H, D, device="cuda").to(BF)
        at = torch.arange(capacity, device="cuda")
        return api.KVCache(k, v), torch.arange(B, device="cuda")[:, None].expand(B, capacity), at[None].expand(B, capacity)
    per = -(-capacity // page)
    pages = B * per + 3
    k = torch.randn(pages, page, H, D, device="cuda").to(BF)
    v = torch.randn(pages, page, H, D, device="cuda").to(BF)
    table = torch.from_numpy(rng.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)).cuda()
    at = torch.arange(per * page, device="cuda")
    return api.KVCache(k, v, table), table[:, at // page].long(), (at % page)[None].expand(B, per * page)


@pytest.mark.parametrize("B,T,heads,H,D,page,rd,inter,shifted", [
    (1, 1, 8, 8, 128, 16, 128, False, False), (5, 1, 0, 2, 64, 16, 64, True, True), (3, 33, 6, 2, 64, 32, 32, False, True),
    (4, 17, 24, 8, 128, 64, 20, False, False), (2, 200, 3, 1, 128, 0, 128, True, True), (300, 20, 2, 2, 64, 16, 64, False, True),
    (2, 5, 4, 4, 128, 128, 0, False, False)])
def test_append(handle, B, T, heads, H, D, page, rd, inter, shifted):
    rng = np.random.default_rng(B + T)
    cap = 150 + T
    cache, pages, rows = pool(B, cap, page, H, D)
    k0, v0 = cache.k.clone(), cache.v.clone()
    lens = rng.integers(0, 150, B)
    count = rng.integers(0, T + 1, B)
    count[0] = T
    if B > 1:
        count[1] = 0
    qkv = torch.randn(B, T, heads + 2 * H, D, device="cuda").to(BF)
    q, kn, vn = qkv.split([heads, H, H], 2)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    position = rng.integers(0, 300000, B) if shifted else lens
    r = api.Rope(rd, interleaved=inter) if rd else None
    scores = torch.ones(B, H, cap, device="cuda")
    q_out = torch.full((B, T, heads, D), 9.0, dtype=BF, device="cuda") if heads else None
    new_len, q_got = api.cache_append(handle, kn, vn, cache, i32(lens), r, i32(count), i32(position) if shifted else None,
                                      q if heads else None, q_out, scores)
    assert new_len.tolist() == (lens + count).tolist() and q_got is q_out
    pos = torch.from_numpy(position).cuda()[:, None] + torch.arange(T, device="cuda")
    f = rates(rd, 10000.0)
    taken = torch.arange(T, device="cuda")[None] < i32(count)[:, None]
    for b in range(B):
        n, m = int(lens[b]), int(count[b])
        pg, rw = pages[b, n:n + m], rows[b, n:n + m]
        want, tol = rotated(kn[b:b + 1, :m], pos[b:b + 1, :m], rd, inter, f)
        check(cache.k[pg, rw], want[0], tol[0], f"k of {b}")
        assert torch.equal(cache.v[pg, rw], vn[b, :m])
        k0[pg, rw], v0[pg, rw] = cache.k[pg, rw], cache.v[pg, rw]
        want_scores = torch.ones(H, cap, device="cuda")
        want_scores[:, n:n + m] = 0
        assert torch.equal(scores[b], want_scores)
    assert torch.equal(cache.k, k0) and torch.equal(cache.v, v0)          # nothing else was written
    if heads:
        want, tol = rotated(q, pos, rd, inter, f)
        left = ~taken[:, :, None, None].expand_as(q_out)
        want = torch.where(left, 9.0, want)
        check(q_out, want, torch.where(left, 0.0, tol), "q")
        same = q.clone().contiguous()
        api.cache_append(handle, kn, vn, cache, i32(lens), r, i32(count), i32(position) if shifted else None, same, same)
        assert torch.equal(torch.where(left, 9.0, same), q_out)           # in place
    assert handle.device_error() == 0


def test_append_without_rotation_is_a_commit(handle):
    B, T, H, D = 3, 9, 2, 64
    a, _, _ = pool(B, 64, 16, H, D)
    b = api.KVCache(a.k.clone(), a.v.clone(), a.block_table)
    kn, vn = (torch.randn(B, T, H, D, device="cuda").to(BF) for _ in range(2))
    lens, count = torch.tensor([0, 31, 50], dtype=torch.int32, device="cuda"), torch.tensor([9, 4, 0], dtype=torch.int32, device="cuda")
    n1, _ = api.cache_append(handle, kn, vn, a, lens, count=count)
    n2 = api.cache_commit(handle, kn, vn, b, lens, count=count)
    assert torch.equal(n1, n2) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_append_keeps_to_the_capacity_and_flags(handle):
    """Lengths, counts and pages out of range: clamped or dropped, flagged, and nothing else written."""
    B, T, H, D, page = 4, 8, 2, 64, 16
    cache, pages, rows = pool(B, 32, page, H, D)
    k0 = cache.k.clone()
    kn, vn = (torch.randn(B, T, H, D, device="cuda").to(BF) for _ in range(2))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    n, _ = api.cache_append(handle, kn, vn, cache, i32([30, 32, 40, -5]), count=i32([8, 8, 3, 2]))
    assert n.tolist() == [32, 32, 32, 2] and handle.device_error() == 0x10
    for b, (start, m) in enumerate([(30, 2), (32, 0), (32, 0), (0, 2)]):
        pg, rw = pages[b, start:start + m], rows[b, start:start + m]
        assert torch.equal(cache.k[pg, rw], kn[b, :m])
        k0[pg, rw] = kn[b, :m]
    assert torch.equal(cache.k, k0)
    n, _ = api.cache_append(handle, kn, vn, cache, i32([0, 0, 0, 0]), count=i32([-1, 99, 0, 0]))
    assert n.tolist() == [0, 8, 0, 0] and handle.device_error() == 0x10
    table = cache.block_table.clone()
    table[0, 0], table[1, 0] = -1, cache.k.shape[0]
    bad = api.KVCache(cache.k, cache.v, table)
    k0 = cache.k.clone()
    n, _ = api.cache_append(handle, kn, vn, bad, i32([12, 0, 0, 0]), count=i32([8, 8, 0, 0]))
    assert n.tolist() == [20, 8, 0, 0] and handle.device_error() == 0x8
    pg, rw = pages[0, 16:20], rows[0, 16:20]
    assert torch.equal(cache.k[pg, rw], kn[0, 4:])
    k0[pg, rw] = kn[0, 4:]
    assert torch.equal(cache.k, k0)
    # scores shorter than the cache bound the positions too
    scores = torch.ones(B, H, 20, device="cuda")
    n, _ = api.cache_append(handle, kn, vn, cache, i32([16, 0, 0, 0]), count=i32([8, 1, 0, 0]), scores=scores)
    assert n.tolist() == [20, 1, 0, 0] and handle.device_error() == 0x10
    assert (scores[0, :, 16:] == 0).all() and (scores[0, :, :16] == 1).all() and scores[1, :, 1:].min() == 1
    # no tokens at all
    n, _ = api.cache_append(handle, kn[:, :0], vn[:, :0], cache, i32([3, 4, 5, 6]))
    assert n.tolist() == [3, 4, 5, 6] and handle.device_error() == 0


def test_append_refusals(handle):
    B, T, H, D = 2, 4, 2, 64
    cache, _, _ = pool(B, 32, 16, H, D)
    kn, vn = (torch.zeros(B, T, H, D, dtype=BF, device="cuda") for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, T, 4, D, dtype=BF, device="cuda")
    for kw in (dict(new_len=lens), dict(count=lens.clone()), dict(q=q, q_out=q[:, :3])):
        if "count" in kw:
            kw["new_len"] = kw["count"]
        with pytest.raises((ValueError, api.Dflash2Error)):
            api.cache_append(handle, kn, vn, cache, lens, **kw)
    position = torch.zeros(B, dtype=torch.int32, device="cuda")
    with pytest.raises(api.Dflash2Error):
        api.cache_append(handle, kn, vn, cache, lens, position=position, new_len=position)
    with pytest.raises(ValueError):
        api.cache_append(handle, kn, vn[:, :, :1], cache, lens)
    with pytest.raises(ValueError):
        api.cache_append(handle, torch.zeros(3, T, H, D, dtype=BF, device="cuda"),
                         torch.zeros(3, T, H, D, dtype=BF, device="cuda"), cache, torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(api.Dflash2Error):
        api.cache_append(handle, kn, vn, cache, lens, rope=api.Rope(128))    # more than the head
    assert handle.device_error() == 0


def test_another_stream_and_a_graph(handle):
    """The calls run on the stream they are given, and a captured sequence of them replays on new contents."""
    B, T, H, D = 3, 5, 2, 128
    cache, pages, rows = pool(B, 64, 16, H, D)
    r = api.Rope(128)
    kn, vn = (torch.randn(B, T, H, D, device="cuda").to(BF) for _ in range(2))
    lens = torch.tensor([0, 3, 20], dtype=torch.int32, device="cuda")
    q = torch.randn(B, T, 4, D, device="cuda").to(BF)
    q_out, new_len = torch.zeros_like(q), torch.zeros_like(lens)
    want = api.rope(handle, q, r, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.rope(handle, q, r, lens, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.cache_append(handle, kn, vn, cache, lens, r, q=q, q_out=q_out, new_len=new_len)
    for seed in range(2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        kn.copy_(torch.randn(kn.shape, generator=g, device="cuda"))
        graph.replay()
        assert torch.equal(q_out, api.rope(handle, q, r, lens)) and new_len.tolist() == [5, 8, 25]
        for b in range(B):
            n = int(lens[b])
            assert torch.equal(cache.k[pages[b, n:n + T], rows[b, n:n + T]], api.rope(handle, kn, r, lens)[b])
