"""Host-side checks of the rotary, append, logit and count entry points: no device is needed.

A made-up handle stands in for a real one: a refused call answers before anything asks for a device, and an accepted one
gets as far as asking (DFLASH2_ERR_CUDA where there is none)."""
import ctypes
import math

import pytest

from draft_selection_dflash2_gb300 import _lib, build

INVALID, UNSUPPORTED, MISALIGNED = -1, -2, -3


class FakeHandle(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("num_sms", ctypes.c_int), ("err", ctypes.c_void_p)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def h():
    # a device that no machine has: an accepted call stops at the check of the current device
    return ctypes.byref(FakeHandle(1 << 20, 152, 4096))


def past_the_checks(status):
    return status in (-4, INVALID)


def table(rotary=64, turns=4096, factor=1.0):
    return ctypes.byref(_lib.RopeTableStruct(turns, rotary, 0, factor))


ROPE = dict(rope=table(), x=4096, xb=512, xt=256, xh=64, out=1 << 20, ob=512, ot=256, oh=64, base=None, depth=None, B=2, T=2,
            heads=4, dim=64, inverse=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rope=None), INVALID), (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(heads=-1), INVALID), (dict(dim=0), INVALID),
    (dict(dim=60), UNSUPPORTED), (dict(dim=520), UNSUPPORTED), (dict(heads=65537), UNSUPPORTED),
    (dict(B=1 << 31), UNSUPPORTED), (dict(B=1 << 16, T=1 << 16), UNSUPPORTED), (dict(rope=table(62 + 4)), INVALID),
    (dict(rope=table(7)), INVALID), (dict(rope=table(0)), INVALID), (dict(rope=table(turns=None)), INVALID),
    (dict(rope=table(turns=4100)), MISALIGNED), (dict(rope=table(factor=math.inf)), INVALID), (dict(x=None), INVALID),
    (dict(out=None), INVALID), (dict(x=4104), MISALIGNED), (dict(out=4104 + (1 << 20)), MISALIGNED), (dict(base=2), MISALIGNED),
    (dict(depth=6), MISALIGNED), (dict(xt=63), INVALID), (dict(xt=260), MISALIGNED), (dict(oh=68), MISALIGNED),
    (dict(out=4096 + 512), INVALID), (dict(out=4096, oh=128), INVALID)])
def test_rope_refuses(lib, h, change, status):
    assert lib.dflash2_rope(h, *{**ROPE, **change}.values()) == status


@pytest.mark.parametrize("change", [dict(B=0), dict(T=0), dict(heads=0)])
def test_rope_of_nothing(lib, h, change):
    assert lib.dflash2_rope(h, *{**ROPE, **change, "x": None, "out": None}.values()) == 0


def test_accepted_calls_reach_the_device_check(lib, h):
    assert past_the_checks(lib.dflash2_rope(h, *ROPE.values()))
    assert past_the_checks(lib.dflash2_rope(h, *{**ROPE, "out": 4096}.values()))
    assert past_the_checks(lib.dflash2_cache_append(h, *append_args().values()))
    assert past_the_checks(lib.dflash2_logits_adjust(h, *LOGITS.values()))
    assert past_the_checks(lib.dflash2_token_counts(h, *COUNTS.values()))


def cache(**kw):
    s = _lib.KvCacheStruct(4096, 8192, 8, 16, 2, 64, 2048, 128, 64, 4096, 4, 4)
    for name, value in kw.items():
        setattr(s, name, value)
    return ctypes.byref(s)


def append_args(**kw):
    a = dict(k=1 << 20, v=1 << 21, nb=512, nt=128, nh=64, cache=cache(), len=4096, rope=table(), count=None, position=None, B=2,
             T=4, q=None, qb=0, qt=0, qh=0, qo=None, ob=0, ot=0, oh=0, heads=0, scores=None, ld=0, new_len=8192, stream=None)
    a.update(kw)
    return a


Q = dict(q=1 << 22, qb=1024, qt=256, qh=64, qo=1 << 23, ob=1024, ot=256, oh=64, heads=4)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(B=65536), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(B=60000, T=1 << 20), UNSUPPORTED), (dict(cache=None), INVALID), (dict(cache=cache(head_dim=96)), UNSUPPORTED),
    (dict(cache=cache(page_size=24)), UNSUPPORTED), (dict(cache=cache(table_ld=3)), INVALID), (dict(rope=table(128)), INVALID),
    (dict(len=None), INVALID), (dict(new_len=None), INVALID), (dict(k=None), INVALID), (dict(new_len=4096), INVALID),
    (dict(new_len=4100), INVALID), (dict(count=8192), INVALID), (dict(position=8188), INVALID), (dict(nt=60), INVALID), (dict(nt=124), MISALIGNED),
    (dict(k=1 << 20 | 8), MISALIGNED), (dict(len=4098), MISALIGNED), (dict(scores=16384, ld=-1), INVALID),
    (dict(q=1 << 22), INVALID), ({**Q, "heads": 0}, INVALID), ({**Q, "q": 8}, MISALIGNED), ({**Q, "qo": (1 << 22) + 256}, INVALID),
    (dict(k=4096 + 256), INVALID), (dict(v=8192 + 512), INVALID), (dict(v=4096), INVALID),   # in the cache
    ({**Q, "heads": 65537}, UNSUPPORTED), ({**Q, "qt": 32}, INVALID)])
def test_append_refuses(lib, h, change, status):
    assert lib.dflash2_cache_append(h, *append_args(**change).values()) == status


LOGITS = dict(x=4096, xb=4096, xt=1024, B=2, T=4, V=1000, counts=1 << 20, cld=1008, tokens=4096, mask=4096, rep=4096, freq=4096,
              pres=4096, bias=1 << 20, bld=0, allowed=4096, ab=128, at=32, out=1 << 21, ob=4096, ot=1024, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(V=-1), INVALID), (dict(tokens=None), INVALID), (dict(T=129), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(V=(1 << 31) - 4096), UNSUPPORTED), (dict(B=60000, V=1 << 30), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(xt=992), INVALID), (dict(xt=1004), MISALIGNED),
    (dict(cld=992), INVALID), (dict(cld=1004), MISALIGNED), (dict(bld=992), INVALID), (dict(bld=1004), MISALIGNED),
    (dict(ab=31), INVALID), (dict(at=31), INVALID), (dict(at=-1), INVALID), (dict(x=4104), MISALIGNED),
    (dict(counts=(1 << 20) + 8), MISALIGNED), (dict(bias=(1 << 20) + 4), MISALIGNED), (dict(mask=4), MISALIGNED),
    (dict(tokens=2), MISALIGNED), (dict(rep=2), MISALIGNED), (dict(allowed=2), MISALIGNED), (dict(out=4096 + 2048), INVALID),
    (dict(out=4096, ot=2048, ob=8192), INVALID)])
def test_logits_refuses(lib, h, change, status):
    assert lib.dflash2_logits_adjust(h, *{**LOGITS, **change}.values()) == status


PREFIX = dict(q=1 << 20, qb=1024, qt=256, qh=64, cache=cache(), len=4096, plen=4096, pstart=4096, groups=2, k=1 << 21, v=1 << 22,
              nb=512, nt=128, nh=64, mask=None, B=2, T=4, heads=4, scale=0.125, out=1 << 23, lse=None, ws=1 << 24,
              bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(groups=-1), INVALID), (dict(groups=3), INVALID), (dict(pstart=None), INVALID), (dict(plen=None), INVALID),
    (dict(q=None), INVALID), (dict(len=None), INVALID), (dict(out=None), INVALID), (dict(k=None), INVALID),
    (dict(cache=None), INVALID), (dict(scale=0.0), INVALID), (dict(heads=3), INVALID), (dict(T=129), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(plen=4098), MISALIGNED), (dict(pstart=4098), MISALIGNED), (dict(ws=1 << 24 | 128), MISALIGNED),
    (dict(qt=60), INVALID), (dict(qt=260), MISALIGNED), (dict(bytes=1 << 10), -7), (dict(ws=None), -7),
    (dict(k=None, v=None, mask=4096), INVALID)])
def test_prefix_refuses(lib, h, change, status):
    assert lib.dflash2_prefix_attention(h, *{**PREFIX, **change}.values()) == status


def test_prefix_accepts(lib, h):
    for change in ({}, dict(groups=0, plen=None, pstart=None), dict(groups=1, pstart=None), dict(qb=2048)):
        assert past_the_checks(lib.dflash2_prefix_attention(h, *{**PREFIX, **change}.values()))
    assert lib.dflash2_prefix_attention(h, *{**PREFIX, "T": 0, "q": None}.values()) == 0
    assert lib.dflash2_prefix_attention(None, *PREFIX.values()) == INVALID
    size = lib.dflash2_prefix_attention_workspace
    assert size(None, 1, 1, 1, 1, 64) == 0 and size(h, 0, 1, 1, 1, 64) == 0 and size(h, 1, 129, 1, 1, 64) == 0
    assert size(h, 2, 4, 4, 2, 96) == 0 and size(h, 2, 4, 3, 2, 64) == 0
    assert size(h, 2, 4, 4, 2, 64) >= lib.dflash2_tree_attention_workspace(h, 2, 4, 4, 2, 64) > 0


COUNTS = dict(tokens=4096, count=None, path=None, B=2, N=10, V=100, prompt=0, counts=8192, ld=100, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(V=-1), INVALID), (dict(B=65536), UNSUPPORTED), (dict(N=1 << 30), UNSUPPORTED),
    (dict(V=1 << 31), UNSUPPORTED), (dict(tokens=None), INVALID), (dict(counts=None), INVALID), (dict(ld=99), INVALID),
    (dict(tokens=2), MISALIGNED), (dict(count=2), MISALIGNED), (dict(path=2), MISALIGNED), (dict(counts=2), MISALIGNED)])
def test_counts_refuses(lib, h, change, status):
    assert lib.dflash2_token_counts(h, *{**COUNTS, **change}.values()) == status


def test_null_handle(lib):
    assert lib.dflash2_rope(None, *ROPE.values()) == INVALID
    assert lib.dflash2_cache_append(None, *append_args().values()) == INVALID
    assert lib.dflash2_logits_adjust(None, *LOGITS.values()) == INVALID
    assert lib.dflash2_token_counts(None, *COUNTS.values()) == INVALID


def turns(lib, rd, theta, **kw):
    s = _lib.RopeScalingStruct(**kw)
    got, factor = (ctypes.c_uint64 * max(rd // 2, 1))(), ctypes.c_float()
    return lib.dflash2_rope_turns(rd, theta, ctypes.byref(s), got, ctypes.byref(factor)), list(got), factor.value


def test_rates(lib):
    """Rates as turns per position times 2^64, within 2^-45 of the formula and the cut to whole numbers: a rate that is cut by
    less than 1 and taken `factor` times is off by less than the factor, and the one it is compared with by less than 1."""
    for rd in (2, 20, 128, 512):
        status, got, factor = turns(lib, rd, 10000.0)
        assert status == 0 and factor == 1.0
        for i, x in enumerate(got):
            want = 10000.0 ** (-2 * i / rd) / (2 * math.pi) * 2.0 ** 64
            assert abs(x - want) <= 2.0 ** -45 * want + 1
    _, plain, _ = turns(lib, 128, 10000.0)
    _, linear, _ = turns(lib, 128, 10000.0, kind=1, factor=4.0)
    assert all(abs(a - 4 * b) <= 2.0 ** -45 * a + 4 for a, b in zip(plain, linear))
    _, ntk, _ = turns(lib, 128, 10000.0, kind=2, factor=4.0)
    assert ntk[0] == plain[0] and abs(ntk[-1] * 4 - plain[-1]) <= 2.0 ** -40 * plain[-1] + 5     # the slowest pair is slowed by the factor
    _, yarn, factor = turns(lib, 128, 10000.0, kind=3, factor=4.0, original=4096, fast=32, slow=1)
    assert yarn[0] == plain[0] and abs(4 * yarn[-1] - plain[-1]) <= 2.0 ** -40 * plain[-1] + 5
    assert factor == pytest.approx(0.1 * math.log(4) + 1, rel=1e-6)
    _, wave, _ = turns(lib, 128, 500000.0, kind=4, factor=8.0, original=8192, low=1, high=4)
    _, plain, _ = turns(lib, 128, 500000.0)
    assert wave[0] == plain[0] and abs(8 * wave[-1] - plain[-1]) <= 2.0 ** -40 * plain[-1] + 9
    assert all(a >= b for a, b in zip(plain, wave))


@pytest.mark.parametrize("rd,theta,kw,status", [
    (0, 1e4, {}, INVALID), (-2, 1e4, {}, INVALID), (7, 1e4, {}, INVALID), (514, 1e4, {}, UNSUPPORTED), (64, 1.0, {}, INVALID),
    (64, math.inf, {}, INVALID), (64, math.nan, {}, INVALID), (64, 1e4, dict(kind=5), INVALID), (64, 1e4, dict(kind=-1), INVALID),
    (64, 1e4, dict(kind=1, factor=0.5), INVALID), (64, 1e4, dict(kind=1, factor=math.nan), INVALID),
    (2, 1e4, dict(kind=2, factor=2), UNSUPPORTED), (64, 1e4, dict(kind=3, factor=2, original=0, fast=32, slow=1), INVALID),
    (64, 1e4, dict(kind=3, factor=2, original=4096, fast=1, slow=1), INVALID),
    (64, 1e4, dict(kind=3, factor=2, original=4096, fast=2, slow=0), INVALID),
    (64, 1e4, dict(kind=4, factor=2, original=4096, low=4, high=1), INVALID),
    (64, 1e300, dict(kind=2, factor=1e300), INVALID)])
def test_rates_refuse(lib, rd, theta, kw, status):
    assert turns(lib, rd, theta, **kw)[0] == status


def test_structs_mirror_the_header():
    import re
    text = re.sub(r"/\*.*?\*/", "", open(_lib.HEADER).read(), flags=re.S)
    kinds = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "float": ctypes.c_float, "double": ctypes.c_double}
    for name, struct in (("dflash2_rope_table", _lib.RopeTableStruct), ("dflash2_rope_scaling", _lib.RopeScalingStruct)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        fields = []
        for decl in filter(None, (f.strip() for f in body.split(";"))):
            kind, names = re.match(r"((?:const )?\w+ ?\*?) *(.*)$", decl).groups()
            fields += [(n.strip(), kinds.get(kind.strip(), ctypes.c_void_p)) for n in names.split(",")]
        assert fields == list(struct._fields_)


def test_scalings_are_checked_by_name():
    from draft_selection_dflash2_gb300 import api
    for scaling in ({"kind": "other"}, {}, {"kind": "linear", "original": 4}, {"kind": "yarn", "low": 1}):
        with pytest.raises(ValueError):
            api.Rope(64, scaling=scaling)
    with pytest.raises(ValueError):
        api.Rope(1024)
