"""Host-side checks of the cache operators that need no device."""
import ctypes
import re

import pytest

from draft_selection_dflash2_gb300 import _lib, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_null_handle_is_rejected_without_a_device(lib):
    null, one = ctypes.c_void_p(None), ctypes.c_void_p(256)
    cache = ctypes.byref(_lib.KvCacheStruct())
    assert lib.dflash2_tree_attention(null, one, 64, 64, 64, cache, one, one, one, 64, 64, 64, null, 1, 1, 1, 1.0, one,
                                      one, one, 1 << 30, null) == -1
    assert lib.dflash2_cache_commit(null, one, one, 64, 64, 64, cache, one, null, null, 1, 1, null, 0, one, null) == -1
    assert lib.dflash2_cache_scores(null, one, 64, 64, 64, one, cache, one, null, null, 1, 1, 1, 1.0, one, 1, null) == -1
    assert lib.dflash2_cache_evict(null, one, 1, cache, one, cache, 1, 1, 0, one, one, one, 1, null) == -1
    assert lib.dflash2_tree_attention_workspace(null, 1, 1, 1, 1, 64) == 0


def test_the_struct_mirrors_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(_lib.HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct dflash2_kv_cache \{(.*?)\} dflash2_kv_cache;", text, re.S).group(1)
    fields = [re.match(r"(.*?)(\w+)$", f.strip()).groups() for f in body.split(";") if f.strip()]
    want = {"int64_t": ctypes.c_int64}
    assert [n for _, n in fields] == [n for n, _ in _lib.KvCacheStruct._fields_]
    for (decl, name), (_, ctype) in zip(fields, _lib.KvCacheStruct._fields_):
        assert ctype is want.get(decl.strip(), ctypes.c_void_p), name


def test_the_binding_refuses_what_is_not_on_a_device():
    import torch
    from draft_selection_dflash2_gb300 import api
    x = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.KVCache(x, x)
    with pytest.raises(ValueError):
        api.KVCache(x, x[:1])
