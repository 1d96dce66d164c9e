"""Pages of many thousands of requests, whose sums a launch of their own adds up, against the oracle, and the time that they take."""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache_helpers import DEV
from test_gpu_pages import Pages

pytestmark = pytest.mark.gpu


def batch(B, seed, spare):
    """Requests that want no page, one or two, of pages of 4 slots."""
    rng = np.random.default_rng(seed)
    return Pages(rng.integers(0, 6, B), rng.integers(0, 20, B), 4, seed, width=8, spare=spare, window=int(rng.choice([0, 7])), sinks=2)


def wanted(p):
    """How many pages the requests before each and it want."""
    k = np.arange(p.width)
    ks = np.diff(p.cu)
    rows = (k >= p.len[:, None] // 4) & (k <= (p.len + ks)[:, None] // 4) & (p.table < 0)
    return np.cumsum(rows.sum(1))


@pytest.mark.parametrize("B", [10240, 10241, 12288, 20000])
def test_many_thousands(B):
    p = batch(B, B, 3 * B)
    assert (p.check()[3] == 1).all()
    rng = np.random.default_rng(1)
    p.len = np.where(rng.random(B) < 0.2, -1, np.minimum(p.len + 3, 24)).astype(np.int32)
    p.check()


@pytest.mark.parametrize("last", [0, 700, 1022, 1023, 1024, 2047, 5000, 11263, 12344])
@pytest.mark.parametrize("more", [0, 1])
def test_a_ring_that_runs_out_among_thousands(last, more):
    """The ring holds what the requests up to `last` want, or one page more."""
    B = 12345
    spare = int(wanted(batch(B, 5, 4 * B))[last]) + more
    p = batch(B, 5, spare)
    got = p.check()
    most = np.searchsorted(wanted(batch(B, 5, 4 * B)), spare, side="right") - 1
    assert got[3][:most + 1].all() and most >= last


@pytest.mark.parametrize("state", [[-1, 3], [0, 2 ** 31 - 1]])
def test_thousands_with_a_ring_out_of_its_bounds(state):
    p = batch(11000, 6, 100)
    p.state[:] = state
    got = p.check()
    assert (got[3] == -1).all() and (got[4] == -1).all()


def test_thousands_of_which_some_are_passed_over():
    p = batch(11000, 7, 33000)
    p.cu[[5, 1024, 4000]] = [-3, 2 ** 31 - 1, 1]
    p.len[[9, 1025, 10999]] = [-2, 2 ** 31 - 1, -1]
    got = p.check()
    assert (got[3] == -1).any()


def test_time_grows_with_the_requests():
    """Eight times the requests take about eight times as long, not sixty-four (38 times when each workgroup added up all before it)."""
    def time(B):
        table = torch.full((B, 4), -1, dtype=torch.int32, device=DEV)
        length = torch.full((B,), 20, dtype=torch.int32, device=DEV)
        cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
        ring, state = torch.arange(4 * B, dtype=torch.int32, device=DEV), torch.tensor([0, 0], dtype=torch.int32, device=DEV)
        times = []
        for _ in range(6):
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            for _ in range(4):
                sdv.kv_pages(table, length, cu, B, ring, state, 16)
            end.record()
            torch.cuda.synchronize()
            times.append(begin.elapsed_time(end))
        return min(times)

    assert time(65536) < 20 * time(8192)
