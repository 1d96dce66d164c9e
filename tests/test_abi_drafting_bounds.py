"""Host-side refusals of the sampling and cache entry points that concern memory and launch sizes: nothing is launched, and
the pointers are never followed."""
import pytest

from test_abi_drafting import INVALID, LIMIT, P, WORKSPACE, _append, _attend, _sample, _settle, lib  # noqa: F401

FAR = 1 << 20
APART = dict(cu=P + FAR, acc=P + 2 * FAR, nodes=P + 3 * FAR, new=P + 8 * FAR,
             cache=dict(cache_len=P + 4 * FAR, page_table=P + 5 * FAR))


@pytest.mark.parametrize("at", [P + 4 * FAR, P + 4 * FAR + 8, P + 4 * FAR - 8, P + 2 * FAR, P + 2 * FAR - 4, P + FAR + 12,
                                P + 3 * FAR + 16, P + 3 * FAR - 8, P + 5 * FAR + 44, P + 5 * FAR - 8])
def test_new_lengths_apart_from_what_is_read(lib, at):  # noqa: F811
    """3 requests, 5 draft rows, tables of 4 pages: lengths in place, or overlapping the first or last word of an input."""
    assert _settle(lib, **{**APART, "new": at}) == INVALID
    assert _settle(lib, **{**APART, "new": at, "layers": 20000}) == LIMIT


@pytest.mark.parametrize("n,V,dtype,probs", [
    (2 ** 24, 1000, 1, False), (2 ** 22, 8000, 0, False), (2 ** 22, 16000, 1, False), (2 ** 22, 100_000, 0, False),
    (2 ** 22 - 1, 160_000, 0, False), (2 ** 22 - 1, 80_000, 1, False), (342_393, 100_000, 0, True), (171_197, 100_000, 1, True)])
def test_sample_launches_below_2_to_32_threads(lib, n, V, dtype, probs):  # noqa: F811
    """The first size that does not fit, and the last that does (which then lacks its workspace)."""
    opt = dict(probs=P) if probs else {}
    assert _sample(lib, n=n, V=V, stride=V, dtype=dtype, opt=opt) == LIMIT
    n = {2 ** 22 - 1: 3_000_000}.get(n, n - 1)
    assert _sample(lib, n=n, V=V, stride=V, dtype=dtype, opt=opt) == WORKSPACE


def test_cache_launches_below_2_to_32_threads(lib):  # noqa: F811
    assert _append(lib, n_d=2 ** 24 - 3) == LIMIT
    assert _settle(lib, **{**APART, "B": 2 ** 24, "cu": P + 2 ** 30}) == LIMIT
    assert _attend(lib, n_d=2 ** 26, cache=dict(dtype=1)) == LIMIT
    assert _attend(lib, n_d=2 ** 27, parents=P) == LIMIT
