"""Host-side argument checks of the sampling and cache entry points: a bad call is refused before anything is
launched (so these run without a GPU; the pointers are never followed)."""
import ctypes

import pytest

from lossless_draft_verification_online_amd import _native
from lossless_draft_verification_online_amd.build import LIBRARY, is_stale

OK, INVALID, UNSUPPORTED, LIMIT, WORKSPACE = 0, -1, -2, -3, -4
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    if is_stale():
        pytest.fail(f"{LIBRARY} is missing or older than its sources; run __graft_entry__.build()")
    return _native.lib()


def _sample(lib, opt=None, **kw):
    a = dict(logits=P, n=4, stride=1000, V=1000, dtype=0, T=1.0, u=P, tokens=P, prob=P, ws=P, bytes=0)
    a.update(kw)
    o = None
    if opt is not None:
        o = _native.SdvSampleOptions(**opt)
    return lib.sdv_sample(a["logits"], a["n"], a["stride"], a["V"], a["dtype"], a["T"], a["u"],
                          None if o is None else ctypes.byref(o), a["tokens"], a["prob"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw", [dict(logits=None), dict(logits=P + 1), dict(dtype=1, logits=P + 2), dict(u=None),
                                dict(tokens=None), dict(prob=None), dict(n=0), dict(n=-1), dict(V=0), dict(stride=999),
                                dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(opt=dict(n_slots=3)),
                                dict(opt=dict(slots=P, n_slots=-1))])
def test_sample_invalid(lib, kw):
    assert _sample(lib, **kw) == INVALID


def test_sample_other_refusals(lib):
    assert _sample(lib, dtype=2) == UNSUPPORTED
    assert _sample(lib, V=2 ** 31 - 1, stride=2 ** 31) == LIMIT
    assert _sample(lib, n=2 ** 31, stride=1000) == LIMIT
    assert _sample(lib, n=2 ** 30, V=100_000, stride=100_000) == LIMIT
    assert _sample(lib, stride=2 ** 41) == LIMIT
    need = lib.sdv_sample_workspace_bytes(4, 1000, 0)
    assert need > 0
    assert _sample(lib) == WORKSPACE  # 0 bytes
    assert _sample(lib, bytes=need - 1) == WORKSPACE
    assert _sample(lib, ws=None, bytes=need) == WORKSPACE
    assert _sample(lib, ws=P + 4, bytes=need) == WORKSPACE
    # a scalar temperature is not looked at beside per-row ones
    assert _sample(lib, T=-1.0, opt=dict(temperature=P)) == WORKSPACE
    for bad in ((0, 10, 0), (1, 0, 0), (1, 10, 5)):
        assert lib.sdv_sample_workspace_bytes(*bad) == 0


def _cache(**kw):
    a = dict(keys=P, values=P, page_table=P, cache_len=P, n_pages=10, max_pages=4, page_size=16, n_kv_heads=2,
             head_dim=64, dtype=0)
    a.update(kw)
    return _native.SdvCache(**a)


BAD_CACHES = [dict(keys=None), dict(values=None), dict(page_table=None), dict(cache_len=None), dict(keys=P + 2),
              dict(values=P + 8), dict(n_pages=0), dict(max_pages=0), dict(page_size=0), dict(page_size=12),
              dict(page_size=2048), dict(n_kv_heads=0), dict(head_dim=96), dict(head_dim=32)]


def _append(lib, cache=None, **kw):
    a = dict(B=3, n_d=5, cu=P, parents=None, k=P, ks=128, v=P, vs=128, f=None, rotary=0, inter=0, q=None, qs=0, n_q=0,
             qo=None)
    a.update(kw)
    c = _cache(**(cache or {}))
    return lib.sdv_kv_append(ctypes.byref(c), a["B"], a["n_d"], a["cu"], a["parents"], a["k"], a["ks"], a["v"], a["vs"],
                             a["f"], a["rotary"], a["inter"], a["q"], a["qs"], a["n_q"], a["qo"], None)


def _attend(lib, cache=None, **kw):
    a = dict(B=3, n_d=5, cu=P, parents=None, q=P, qs=256, n_q=4, scale=1.0, window=0, sinks=0, out=2 * P, ws=None, bytes=0)
    a.update(kw)
    c = _cache(**(cache or {}))
    return lib.sdv_attend(ctypes.byref(c), a["B"], a["n_d"], a["cu"], a["parents"], a["q"], a["qs"], a["n_q"], a["scale"],
                          a["window"], a["sinks"], a["out"], a["ws"], a["bytes"], None)


def _settle(lib, cache=None, **kw):
    a = dict(layers=1, B=3, n_d=5, cu=P, acc=P, nodes=P, new=P)
    a.update(kw)
    c = _cache(**(cache or {}))
    return lib.sdv_kv_settle(ctypes.byref(c), a["layers"], a["B"], a["n_d"], a["cu"], a["acc"], a["nodes"], a["new"], None)


@pytest.mark.parametrize("call", [_append, _attend, _settle])
def test_cache_checks(lib, call):
    for bad in BAD_CACHES:
        assert call(lib, cache=bad) == INVALID, bad
    assert call(lib, cache=dict(dtype=3)) == UNSUPPORTED
    for bad in (dict(B=0), dict(n_d=-1), dict(cu=None)):
        assert call(lib, **bad) == INVALID, bad
    assert call(lib, n_d=2 ** 31 - 2) == LIMIT
    assert call(lib, cache=dict(n_kv_heads=1025)) == LIMIT
    assert call(lib, cache=dict(n_pages=2 ** 31)) == LIMIT


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=P + 4), dict(ks=127), dict(vs=120), dict(ks=132),
                                dict(f=P), dict(rotary=64), dict(f=P, rotary=24), dict(f=P, rotary=80), dict(f=P, rotary=-16),
                                dict(n_q=4), dict(n_q=4, q=P, qs=256), dict(n_q=4, qo=P), dict(n_q=4, q=P, qs=255, qo=2 * P),
                                dict(n_q=4, q=P, qs=512, qo=P), dict(q=P), dict(n_q=-1)])
def test_append_invalid(lib, kw):
    assert _append(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(q=None), dict(out=None), dict(q=P + 2), dict(out=P + 2), dict(qs=255), dict(qs=260),
                                dict(n_q=0), dict(n_q=5), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(out=P)])
def test_attend_invalid(lib, kw):
    assert _attend(lib, **kw) == INVALID


def test_attend_workspace(lib):
    c = _cache(max_pages=1000)
    need = lib.sdv_attend_workspace_bytes(ctypes.byref(c), 3, 5, 4, 0, 0)
    assert need > 0  # a long cache of few heads is split
    for kw in (dict(ws=None, bytes=need), dict(ws=P, bytes=need - 1), dict(ws=P + 4, bytes=need)):
        assert _attend(lib, cache=dict(max_pages=1000), **kw) == WORKSPACE
    assert lib.sdv_attend_workspace_bytes(ctypes.byref(c), 3, 5, 5, 0, 0) == 0
    assert lib.sdv_attend_workspace_bytes(None, 3, 5, 4, 0, 0) == 0


@pytest.mark.parametrize("kw", [dict(layers=0), dict(acc=None), dict(nodes=None), dict(new=None)])
def test_settle_invalid(lib, kw):
    assert _settle(lib, **kw) == INVALID
    assert _settle(lib, layers=20000) == LIMIT
