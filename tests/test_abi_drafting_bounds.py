"""Host-side refusals of the sampling and cache entry points that concern memory and launch sizes: nothing is launched, and
the pointers are never followed."""
import pytest

from test_abi_drafting import INVALID, LIMIT, P, _settle, lib  # noqa: F401

FAR = 1 << 20
APART = dict(cu=P + FAR, acc=P + 2 * FAR, nodes=P + 3 * FAR, new=P + 8 * FAR,
             cache=dict(cache_len=P + 4 * FAR, page_table=P + 5 * FAR))


@pytest.mark.parametrize("at", [P + 4 * FAR, P + 4 * FAR + 8, P + 4 * FAR - 8, P + 2 * FAR, P + 2 * FAR - 4, P + FAR + 12,
                                P + 3 * FAR + 16, P + 3 * FAR - 8, P + 5 * FAR + 44, P + 5 * FAR - 8])
def test_new_lengths_apart_from_what_is_read(lib, at):  # noqa: F811
    """3 requests, 5 draft rows, tables of 4 pages: lengths in place, or overlapping the first or last word of an input."""
    assert _settle(lib, **{**APART, "new": at}) == INVALID
    assert _settle(lib, **{**APART, "new": at, "layers": 20000}) == LIMIT
