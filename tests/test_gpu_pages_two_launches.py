"""Arguments that are not valid, and rings that run out or over, where the pages' call takes two launches: rows of the table too long
for one, or more requests, against the oracle."""
import numpy as np
import pytest

import lossless_draft_verification_online_amd as sdv
from oracle import cache8 as oracle
from test_gpu_pages import Pages
from test_gpu_pages_many import batch, wanted

pytestmark = pytest.mark.gpu

WIDE = 1000  # entries of a row


def more_requests(ks, lens):
    """Requests enough for two launches, the given ones first."""
    return ks + [k % 5 for k in range(20)], lens + [3 * k for k in range(20)]


def check(p, rows):
    """p.check() with the slots of `rows` only."""
    args = p.args()
    placed, slots = sdv.kv_pages(*args[:3], p.n_d, *args[3:], p.page)
    want = oracle.pages(p.table, p.page, p.len, p.n_d, p.cu, p.ring, p.state)
    for x, y in zip((args[0], args[3], args[4], placed), want):
        assert np.array_equal(x.cpu().numpy(), y)
    assert np.array_equal(slots.cpu().numpy()[rows], want[4][rows])


@pytest.fixture(params=["long rows", "many requests"])
def pages(request):
    def make(ks, lens, page, seed, **kw):
        if request.param == "long rows":
            kw["width"] = WIDE
        else:
            ks, lens = more_requests(ks, lens)
        return Pages(ks, lens, page, seed, **kw)

    return make


@pytest.mark.parametrize("bad", [[0, 3, 2, 10], [0, -5, 5, 10], [0, 3, 50, 10], [4, 3, 2, 1], [-1, -1, -1, -1], [0, 3, 5, -1],
                                 [2 ** 31 - 1, 3, 5, 10], [0, 3, -2 ** 31, 10]])
def test_offsets_that_are_not_valid(pages, bad):
    p = pages([3, 2, 5], [30, 7, 15], 4, 7, spare=120)
    p.cu[:4] = bad
    # of two requests that name one row, any is served: an offset of 50 lies within the larger batch, whose other requests go on at 10
    lo, hi = p.cu[:-1].astype(np.int64), p.cu[1:].astype(np.int64)
    named = np.zeros(p.n_d + len(lo), dtype=np.int64)
    for i in np.flatnonzero((lo >= 0) & (hi >= lo) & (hi <= p.n_d)):
        named[lo[i] + i:hi[i] + i + 1] += 1
    check(p, named < 2)


@pytest.mark.parametrize("state", [[-1, 3], [10 ** 6, 3], [0, -1], [0, 2 ** 31 - 1], [2 ** 31 - 1, 0], [-2 ** 31, -2 ** 31]])
def test_a_ring_out_of_its_bounds(pages, state):
    p = pages([3, 2, 5], [30, 7, 15], 4, 8, spare=120)
    p.state[:] = state
    before = p.table.copy(), p.ring.copy()
    got = p.check()
    assert (got[3] == -1).all() and (got[4] == -1).all()
    assert np.array_equal(got[0], before[0]) and np.array_equal(got[1], before[1]) and got[2].tolist() == state


def test_what_is_passed_over(pages):
    p = pages([3, 2, 9, 1], [40, 100, 77, 33], 16, 5, spare=120)
    p.len[:4] = [40, -2, 2 ** 31 - 1, 2 ** 31 - 1024 - 1]
    assert p.check()[3][:4].tolist() == [1, -1, -1, -1]
    p.len[1] = 2 ** 30  # its rows end behind the table
    assert p.check()[3][:4].tolist() == [1, 0, -1, -1]


def test_numbers_that_are_no_pages(pages):
    p = pages([3, 2, 5], [30, 7, 15], 4, 9, spare=120)
    p.table[0, 2], p.table[0, 7], p.table[2, 3] = 2 ** 31 - 1, -2 ** 31, len(p.ring)
    p.ring[(p.state[0] + 1) % len(p.ring)] = 10 ** 6  # taken, and no page
    assert (p.check()[4] == -1).any()


def test_more_pages_than_the_ring_holds(pages):
    p = pages([0, 0, 0], [100, 100, 100], 4, 10, spare=3)
    p.table[:, :20] = 5
    p.len[:] = -1
    got = p.check()
    assert got[2][1] == len(p.ring)


@pytest.mark.parametrize("spare", [0, 1, 3, 4, 9])
def test_a_ring_that_runs_out(pages, spare):
    got = pages([20, 0, 70, 0, 5, 0], [8, 16, 3, 5, 31, 16], 16, 3, spare=spare).check()
    assert (got[3] == 0).any() or spare == 9


@pytest.mark.parametrize("last", [0, 100, 254, 255, 256, 300, 511, 512, 599])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_a_ring_that_runs_out_among_hundreds(last, more):
    """The ring holds what the requests up to `last` want, or a page less or more."""
    B = 600
    want = wanted(batch(B, 3, 4 * B))
    spare = max(int(want[last]) + more, 0)
    got = batch(B, 3, spare).check()
    most = np.searchsorted(want, spare, side="right") - 1
    assert got[3][:most + 1].all() and (most == B - 1 or not got[3].all())


@pytest.mark.parametrize("B", [17, 255, 256, 257, 600])
def test_requests_that_end_and_come_back(B):
    p = batch(B, B, 3 * B)
    rng = np.random.default_rng(B)
    for _ in range(6):
        p.check()
        p.len = np.where(rng.random(B) < 0.3, -1, np.where(p.len < 0, 0, (p.len + rng.integers(1, 6, B)) % 25)).astype(np.int32)
