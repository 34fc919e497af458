"""Logit adjustment and token counts, against 64-bit arithmetic.

Tolerance: one rounding to bf16, 2^-8 |y|, and at most 6 fp32 roundings (quotient, two products, three sums) of terms
no larger than |x / r| + |x r| + f n + p + |bias|: 2^-21 of that sum."""
import numpy as np
import pytest

from draft_selection_dflash2_gb300 import api
from gpu_common import handle, torch  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def pad(n):
    return (n + 7) // 8 * 8


def bits_of(sees):
    """bool [..., n] -> words of 64 as int64."""
    n = sees.shape[-1]
    words = (n + 63) // 64
    full = np.zeros((*sees.shape[:-1], words * 64), np.uint8)
    full[..., :n] = sees
    return torch.from_numpy(np.packbits(full, -1, bitorder="little").view(np.int64).copy()).cuda()


def words_of(ok):
    n = ok.shape[-1]
    full = np.zeros((*ok.shape[:-1], (n + 31) // 32 * 32), np.uint8)
    full[..., :n] = ok
    return torch.from_numpy(np.packbits(full, -1, bitorder="little").view(np.int32).copy()).cuda()


def plain(x, counts, tokens, sees, rep, freq, pres, bias, ok):
    """(y, tolerance), numpy 64-bit, plain loops over rows."""
    B, T, V = x.shape
    y, size = x.astype(np.float64), np.abs(x.astype(np.float64))
    for b in range(B):
        for t in range(T):
            n = np.zeros(V) if counts is None else (counts[b] & 0x7FFFFFFF).astype(np.float64)
            if tokens is not None:
                for s in range(T):
                    if sees[b, t, s] and 0 <= tokens[b, s] < V:
                        n[tokens[b, s]] += 1
            known = n > 0
            if counts is not None:
                known = known | (counts[b] < 0)
            r, f, p = (float(v[b]) if v is not None else d for v, d in ((rep, 1), (freq, 0), (pres, 0)))
            row = y[b, t]
            row = np.where(known, np.where(row > 0, row / r, row * r), row)
            size[b, t] = np.where(np.isfinite(row), np.abs(row), 0)
            row = row - np.where(n > 0, f * n + p, 0)
            size[b, t] += f * n + p
            if bias is not None:
                row = row + bias[b if bias.shape[0] > 1 else 0]
                size[b, t] += np.abs(bias[b if bias.shape[0] > 1 else 0])
            if ok is not None:
                row = np.where(ok[b if ok.shape[0] > 1 else 0, t if ok.shape[1] > 1 else 0], row, -np.inf)
            y[b, t] = row
    return y, size * 2.0 ** -21 + np.where(np.isfinite(y), np.abs(y), 0) * 2.0 ** -8


def check(got, want, tol):
    got = got.double().cpu().numpy()
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        assert (same | (np.abs(got - want) <= tol)).all()


CASES = [  # B, T, V, tree, counts, tokens, params, bias rows, allowed shape
    (1, 1, 1, False, True, True, True, 1, (1, 1)), (2, 3, 13, False, True, True, True, 2, (2, 3)),
    (3, 17, 1000, False, True, True, True, 0, None), (2, 17, 4099, True, True, True, True, 1, (2, 17)),
    (2, 100, 333, True, False, True, True, 0, (1, 100)), (1, 128, 257, True, True, True, True, 1, (1, 1)),
    (1, 128, 40, False, False, True, True, 0, None), (4, 1, 5000, False, True, False, True, 0, None),
    (2, 5, 2048, False, True, True, False, 2, (2, 1)), (2, 5, 2056, False, False, False, False, 1, (2, 5)),
    (3, 64, 100, True, True, True, True, 3, (3, 64)), (2, 65, 100, True, True, True, True, 0, None),
    (2, 2, 30, False, False, False, False, 0, None)]


@pytest.mark.parametrize("B,T,V,tree,counted,drafted,params,bias_rows,allow", CASES)
@pytest.mark.parametrize("inplace", [False, True])
def test_logits_adjust(handle, B, T, V, tree, counted, drafted, params, bias_rows, allow, inplace):
    rng = np.random.default_rng(B * 100 + T)
    gen = torch.Generator(device="cuda").manual_seed(V)
    wide = (torch.randn(B, T, pad(V) + 8, generator=gen, device="cuda") * 3).to(BF)
    wide[..., ::7] *= 0.0
    if V > 12:
        wide[0, 0, 3], wide[0, 0, 5], wide[0, 0, 11] = float("inf"), -float("inf"), float("nan")
    x = wide[..., :V]
    x_host = x.float().cpu().numpy()
    counts = tokens = sees = rep = freq = pres = bias = ok = None
    if counted:
        counts = rng.integers(0, 3, (B, V)) * (rng.random((B, V)) < 0.3)
        counts = np.where(rng.random((B, V)) < 0.2, counts - 2 ** 31, counts).astype(np.int32)
    if drafted:
        tokens = rng.integers(0, V, (B, T)).astype(np.int32)
        tokens[:, T // 2:] = tokens[:, :T - T // 2]          # the same tokens again
        sees = np.tril(np.ones((T, T), bool))[None].repeat(B, 0)
        if tree:
            sees = (rng.random((B, T, T)) < 0.4)
    if params:
        rep, freq, pres = (rng.uniform(lo, hi, B).astype(np.float32) for lo, hi in ((0.7, 1.5), (-0.3, 1.0), (-0.2, 1.0)))
        freq, pres = np.abs(freq), np.abs(pres)
    if bias_rows:
        bias = (rng.normal(0, 3, (bias_rows, V)) * (rng.random((bias_rows, V)) < 0.5)).astype(np.float32)
        if V > 20:
            bias[0, 17] = -np.inf
    if allow:
        ok = rng.random((*allow, V)) < 0.5
        ok[0, 0] = False                                      # a row with nothing left
        if allow[1] > 1:
            ok[-1, -1] = True
    dev = lambda a, dt: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()  # noqa: E731

    def padded(a, dt):
        if a is None:
            return None
        t = torch.zeros(a.shape[0], pad(V) + 8, dtype=dt, device="cuda")
        t[:, :V] = dev(a, dt)
        return t[:, :V]
    want, tol = plain(x_host, counts, tokens, sees, rep, freq, pres, bias, ok)
    room = wide if inplace else torch.full_like(wide, 5.0)
    beyond = room[..., V:].clone()
    got = api.logits_adjust(handle, x, padded(counts, torch.int32), dev(tokens, torch.int32),
                            bits_of(sees) if tree and drafted else None, dev(rep, torch.float32), dev(freq, torch.float32),
                            dev(pres, torch.float32), padded(bias, torch.float32), None if ok is None else words_of(ok),
                            out=room[..., :V])
    check(got, want, tol)
    assert torch.equal(room[..., V:].view(torch.int16), beyond.view(torch.int16))   # columns past V are left alone
    assert handle.device_error() == 0


def test_in_place_and_out_of_place_agree(handle):
    B, T, V = 3, 9, 3001
    rng = np.random.default_rng(0)
    x = torch.randn(B, T, pad(V), device="cuda").to(BF)[..., :V]
    counts = torch.zeros(B, pad(V), dtype=torch.int32, device="cuda")[:, :V]
    api.token_counts(handle, torch.from_numpy(rng.integers(0, V, (B, 50)).astype(np.int32)).cuda(), counts)
    kw = dict(counts=counts, tokens=torch.from_numpy(rng.integers(0, V, (B, T)).astype(np.int32)).cuda(),
              repetition=torch.full((B,), 1.2, device="cuda"), presence=torch.full((B,), 0.3, device="cuda"),
              allowed=words_of(rng.random((B, T, V)) < 0.99))
    a = api.logits_adjust(handle, x, **kw)
    b = api.logits_adjust(handle, x, out=x, **kw)
    assert b is x and torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_bad_tokens_are_flagged_and_count_nothing(handle):
    B, T, V = 2, 4, 100
    x = torch.ones(B, T, 104, dtype=BF, device="cuda")[..., :V]
    tokens = torch.tensor([[0, -1, V, 5], [2 ** 31 - 1, 1, 1, 1]], dtype=torch.int32, device="cuda")
    got = api.logits_adjust(handle, x, tokens=tokens, presence=torch.full((B,), 0.5, device="cuda"))
    assert handle.device_error() == 0x1
    want = torch.ones(B, T, V)
    want[0, :, 0] = 0.5
    want[0, 3, 5] = 0.5
    want[1, 1:, 1] = 0.5
    assert torch.equal(got.float().cpu(), want)


def test_token_counts(handle):
    B, N, V = 3, 40, 17
    rng = np.random.default_rng(1)
    tokens = rng.integers(0, V, (B, N)).astype(np.int32)
    count = np.array([40, 0, 7], np.int32)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    counts = torch.zeros(B, 24, dtype=torch.int32, device="cuda")
    counts[:, V:] = 77
    want = np.zeros((B, V), np.int64)
    api.token_counts(handle, dev(tokens), counts[:, :V], count=dev(count))
    for b in range(B):
        np.add.at(want[b], tokens[b, :count[b]], 1)
    assert counts[:, :V].cpu().numpy().tolist() == want.tolist() and (counts[:, V:] == 77).all()
    path = rng.integers(0, N, (B, N)).astype(np.int32)
    api.token_counts(handle, dev(tokens), counts[:, :V], count=dev(count), path=dev(path))
    for b in range(B):
        np.add.at(want[b], tokens[b, path[b, :count[b]]], 1)
    assert counts[:, :V].cpu().numpy().tolist() == want.tolist()
    prompt = rng.integers(0, 5, (B, 3000)).astype(np.int32)
    api.token_counts(handle, dev(prompt), counts[:, :V], prompt=True)
    want[:, :5] -= 2 ** 31
    assert counts[:, :V].cpu().numpy().tolist() == want.tolist() and (counts[:, V:] == 77).all()
    api.token_counts(handle, dev(tokens), counts[:, :V])          # a prompt's tokens are counted beside the flag
    for b in range(B):
        np.add.at(want[b], tokens[b], 1)
    assert counts[:, :V].cpu().numpy().tolist() == want.tolist() and handle.device_error() == 0


def test_token_counts_flags(handle):
    V = 10
    counts = torch.zeros(2, V, dtype=torch.int32, device="cuda")
    tokens = torch.tensor([[1, V, -1, 2], [3, 3, 3, 3]], dtype=torch.int32, device="cuda")
    api.token_counts(handle, tokens, counts)
    assert handle.device_error() == 0x1
    assert counts[0].tolist() == [0, 1, 1, 0, 0, 0, 0, 0, 0, 0] and counts[1, 3] == 4
    api.token_counts(handle, tokens, counts, count=torch.tensor([-2, 9], dtype=torch.int32, device="cuda"))
    assert handle.device_error() == 0x10 and counts[1, 3] == 8 and counts[0].sum() == 2
    path = torch.tensor([[0, 9, 0, 0], [-3, 0, 0, 0]], dtype=torch.int32, device="cuda")
    api.token_counts(handle, tokens, counts, count=torch.tensor([2, 1], dtype=torch.int32, device="cuda"), path=path)
    assert handle.device_error() == 0x20 and counts[0, 1] == 2 and counts[0, 2] == 2 and counts[1, 3] == 9


def test_empty_calls_and_refusals(handle):
    V = 16
    x = torch.zeros(2, 3, V, dtype=BF, device="cuda")
    for shape in ((0, 3, V), (2, 0, V), (2, 3, 0)):
        assert api.logits_adjust(handle, torch.zeros(shape, dtype=BF, device="cuda")).shape == shape
    counts = torch.zeros(2, V, dtype=torch.int32, device="cuda")
    assert api.token_counts(handle, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), counts) is counts
    f = torch.zeros(2, device="cuda")
    for kw in (dict(counts=counts[:, :8]), dict(counts=counts.long()), dict(tokens=torch.zeros(2, 2, dtype=torch.int32, device="cuda")),
               dict(repetition=f[:1]), dict(bias=torch.zeros(3, V, device="cuda")), dict(presence=f.cpu()),
               dict(allowed=torch.zeros(2, 3, 2, dtype=torch.int32, device="cuda")), dict(out=x.float())):
        with pytest.raises(ValueError):
            api.logits_adjust(handle, x, **kw)
    with pytest.raises(api.Dflash2Error):                      # rows that are not 16 bytes apart
        api.logits_adjust(handle, torch.zeros(2, 3, 17, dtype=BF, device="cuda"))
    with pytest.raises(api.Dflash2Error):                      # ranges that only overlap
        api.logits_adjust(handle, x[:, :2], out=x[:, 1:])
    with pytest.raises(api.Dflash2Error):                      # a mask without tokens
        api.logits_adjust(handle, x, tree_mask=torch.zeros(2, 3, 1, dtype=torch.int64, device="cuda"))
    with pytest.raises(api.Dflash2Error):
        api.logits_adjust(handle, torch.zeros(1, 129, V, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        api.token_counts(handle, torch.zeros(2, 3, dtype=torch.int64, device="cuda"), counts)
    with pytest.raises(ValueError):
        api.token_counts(handle, torch.zeros(1, 3, dtype=torch.int32, device="cuda"), counts)
    assert handle.device_error() == 0


def test_a_graph_replays_on_new_contents(handle):
    B, T, V = 2, 5, 1000
    x = torch.randn(B, T, V, device="cuda").to(BF)
    out, counts = torch.zeros_like(x), torch.zeros(B, V, dtype=torch.int32, device="cuda")
    tokens = torch.randint(0, V, (B, T), dtype=torch.int32, device="cuda")
    kw = dict(counts=counts, tokens=tokens, frequency=torch.tensor([0.5, 1.0], device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.logits_adjust(handle, x, out=out, **kw)
        api.token_counts(handle, tokens, counts)
    for step in range(3):
        x.normal_()
        tokens.random_(0, V)
        before = counts.clone()
        want = api.logits_adjust(handle, x, **{**kw, "counts": before})
        graph.replay()
        assert torch.equal(out, want) and int(counts.sum()) == (step + 1) * B * T
