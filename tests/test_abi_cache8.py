"""Host-side argument checks of the calls over a cache in 8 bits, and of the pages' call: nothing is launched, and the
pointers are never followed."""
import ctypes

import pytest

from lossless_draft_verification_online_amd import _native
from test_abi_drafting import BAD_CACHES, INVALID, LIMIT, P, UNSUPPORTED, WORKSPACE, _cache, lib  # noqa: F401

FAR = 1 << 20


def _cache8(cache=None, **kw):
    a = dict(key_scales=P, value_scales=P, block=8)
    a.update(kw)
    return _native.SdvCache8(_cache(**(cache or {})), a["key_scales"], a["value_scales"], a["block"])


def _append(lib, cache=None, c8=None, **kw):  # noqa: F811
    a = dict(B=3, n_d=5, cu=P, parents=None, k=P, ks=128, v=P, vs=128, f=None, rotary=0, inter=0, q=None, qs=0, n_q=0, qo=None)
    a.update(kw)
    c = _cache8(cache, **(c8 or {}))
    return lib.sdv_kv_append8(ctypes.byref(c), a["B"], a["n_d"], a["cu"], a["parents"], a["k"], a["ks"], a["v"], a["vs"],
                              a["f"], a["rotary"], a["inter"], a["q"], a["qs"], a["n_q"], a["qo"], None)


def _attend(lib, cache=None, c8=None, **kw):  # noqa: F811
    a = dict(B=3, n_d=5, cu=P, parents=None, q=P, qs=256, n_q=4, scale=1.0, window=0, sinks=0, out=2 * P, ws=None, bytes=0)
    a.update(kw)
    c = _cache8(cache, **(c8 or {}))
    return lib.sdv_attend8(ctypes.byref(c), a["B"], a["n_d"], a["cu"], a["parents"], a["q"], a["qs"], a["n_q"], a["scale"],
                           a["window"], a["sinks"], a["out"], a["ws"], a["bytes"], None)


def _settle(lib, cache=None, c8=None, **kw):  # noqa: F811
    a = dict(layers=1, B=3, n_d=5, cu=P, acc=P, nodes=P, new=P)
    a.update(kw)
    c = _cache8(cache, **(c8 or {}))
    return lib.sdv_kv_settle8(ctypes.byref(c), a["layers"], a["B"], a["n_d"], a["cu"], a["acc"], a["nodes"], a["new"], None)


def _pages(lib, **kw):  # noqa: F811
    a = dict(table=P, B=3, max_pages=4, page=16, len=P + FAR, n_d=5, cu=P + 2 * FAR, n_pages=10, ring=P + 3 * FAR,
             state=P + 4 * FAR, window=0, sinks=0, placed=P + 5 * FAR, slots=P + 6 * FAR, ws=None, bytes=0)
    a.update(kw)
    return lib.sdv_kv_pages(a["table"], a["B"], a["max_pages"], a["page"], a["len"], a["n_d"], a["cu"], a["n_pages"], a["ring"],
                            a["state"], a["window"], a["sinks"], a["placed"], a["slots"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("call", [_append, _attend, _settle])
def test_cache_checks(lib, call):  # noqa: F811
    for bad in BAD_CACHES:
        assert call(lib, cache=bad) == INVALID, bad
    for bad in (dict(key_scales=None), dict(value_scales=None), dict(block=0), dict(block=-1), dict(block=3), dict(block=32),
                dict(block=128)):
        assert call(lib, c8=bad) == INVALID, bad
    assert call(lib, c8=dict(block=128), cache=dict(page_size=1024)) == INVALID
    assert call(lib, cache=dict(dtype=3)) == UNSUPPORTED
    for bad in (dict(B=0), dict(n_d=-1), dict(cu=None)):
        assert call(lib, **bad) == INVALID, bad
    assert call(lib, n_d=2 ** 31 - 2) == LIMIT
    assert call(lib, cache=dict(n_kv_heads=1025)) == LIMIT
    assert call(lib, cache=dict(n_pages=2 ** 31)) == LIMIT


def test_no_cache(lib):  # noqa: F811
    assert lib.sdv_kv_append8(None, 3, 5, P, None, P, 128, P, 128, None, 0, 0, None, 0, 0, None, None) == INVALID
    assert lib.sdv_attend8(None, 3, 5, P, None, P, 256, 4, 1.0, 0, 0, 2 * P, None, 0, None) == INVALID
    assert lib.sdv_kv_settle8(None, 1, 3, 5, P, P, P, P, None) == INVALID
    assert lib.sdv_attend8_workspace_bytes(None, 3, 5, 4, 0, 0) == 0


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=P + 4), dict(ks=127), dict(vs=120), dict(ks=132),
                                dict(f=P), dict(rotary=64), dict(f=P, rotary=24), dict(f=P, rotary=80), dict(f=P, rotary=-16),
                                dict(n_q=4), dict(n_q=4, q=P, qs=256), dict(n_q=4, qo=P), dict(n_q=4, q=P, qs=255, qo=2 * P),
                                dict(n_q=4, q=P, qs=512, qo=P), dict(q=P), dict(n_q=-1)])
def test_append_invalid(lib, kw):  # noqa: F811
    assert _append(lib, **kw) == INVALID


def test_append_launches_below_2_to_32_threads(lib):  # noqa: F811
    assert _append(lib, n_d=2 ** 24 - 3) == LIMIT
    # a unit of one token: two of a request's and one of a row, in a workgroup for each four of its heads
    assert _append(lib, n_d=2 ** 23, c8=dict(block=1), cache=dict(n_kv_heads=8), ks=512, vs=512) == LIMIT
    assert _append(lib, n_d=2 ** 23, n_q=4, q=P, qs=256, qo=2 * P, c8=dict(block=1)) == LIMIT


@pytest.mark.parametrize("kw", [dict(q=None), dict(out=None), dict(q=P + 2), dict(out=P + 2), dict(qs=255), dict(qs=260),
                                dict(n_q=0), dict(n_q=5), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(out=P)])
def test_attend_invalid(lib, kw):  # noqa: F811
    assert _attend(lib, **kw) == INVALID


def test_attend_limits(lib):  # noqa: F811
    assert _attend(lib, n_d=2 ** 27, cache=dict(dtype=1)) == LIMIT
    assert _attend(lib, n_d=2 ** 27, parents=P) == LIMIT


def test_attend_workspace(lib):  # noqa: F811
    c = _cache8(dict(max_pages=1000))
    need = lib.sdv_attend8_workspace_bytes(ctypes.byref(c), 3, 5, 4, 0, 0)
    assert need > 0  # a long cache of few heads is split
    for kw in (dict(ws=None, bytes=need), dict(ws=P, bytes=need - 1), dict(ws=P + 4, bytes=need)):
        assert _attend(lib, cache=dict(max_pages=1000), **kw) == WORKSPACE
    assert lib.sdv_attend8_workspace_bytes(ctypes.byref(c), 3, 5, 5, 0, 0) == 0


@pytest.mark.parametrize("kw", [dict(layers=0), dict(acc=None), dict(nodes=None), dict(new=None)])
def test_settle_invalid(lib, kw):  # noqa: F811
    assert _settle(lib, **kw) == INVALID
    assert _settle(lib, layers=20000) == LIMIT


APART = dict(cu=P + FAR, acc=P + 2 * FAR, nodes=P + 3 * FAR, new=P + 8 * FAR, cache=dict(cache_len=P + 4 * FAR, page_table=P + 5 * FAR))


@pytest.mark.parametrize("at", [P + 4 * FAR, P + 4 * FAR + 8, P + 2 * FAR, P + 2 * FAR - 4, P + FAR + 12, P + 3 * FAR + 16,
                                P + 5 * FAR + 44, P + 5 * FAR - 8])
def test_new_lengths_apart_from_what_is_read(lib, at):  # noqa: F811
    assert _settle(lib, **{**APART, "new": at}) == INVALID


@pytest.mark.parametrize("kw", [dict(table=None), dict(len=None), dict(cu=None), dict(ring=None), dict(state=None),
                                dict(placed=None), dict(B=0), dict(n_d=-1), dict(max_pages=0), dict(n_pages=0), dict(page=0),
                                dict(page=12), dict(page=2048), dict(window=-1), dict(sinks=-1), dict(table=P + 2),
                                dict(slots=P + 6 * FAR + 4), dict(placed=P + FAR), dict(placed=P + FAR + 8),
                                dict(state=P + 3 * FAR + 36), dict(slots=P), dict(table=P + 2 * FAR), dict(B=300, ws=P, bytes=FAR),
                                dict(B=300, ws=P + 6 * FAR - 16, bytes=FAR)])
def test_pages_invalid(lib, kw):  # noqa: F811
    assert _pages(lib, **kw) == INVALID


def test_pages_limits_and_workspace(lib):  # noqa: F811
    big = dict(table=1 << 44, len=1 << 45, cu=1 << 46, ring=1 << 47, state=1 << 48, placed=1 << 49, slots=1 << 50)
    assert _pages(lib, B=2 ** 24, **big) == LIMIT
    assert _pages(lib, n_d=2 ** 31 - 1024, **big) == LIMIT
    assert _pages(lib, n_pages=2 ** 31, **big) == LIMIT
    assert _pages(lib, max_pages=2 ** 31 - 1, **big) == LIMIT
    need = lib.sdv_kv_pages_workspace_bytes(3, 1000)
    assert need > 0
    for bad in ((0, 1000), (2 ** 24, 1000), (100, 0), (3, 4)):  # the last: few requests with short rows need none
        assert lib.sdv_kv_pages_workspace_bytes(*bad) == 0
    for kw in (dict(), dict(ws=P + 9 * FAR, bytes=need - 1), dict(ws=P + 9 * FAR + 4, bytes=need)):
        assert _pages(lib, max_pages=1000, **kw) == WORKSPACE
