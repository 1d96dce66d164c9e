"""A round's pages from the requests' lengths, on the GPU against the oracle: whole numbers, all equal."""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache_helpers import DEV
from oracle import cache8 as oracle

pytestmark = pytest.mark.gpu


class Pages:
    """Tables that hold what lens need, the other pages in a ring in random order."""

    def __init__(self, ks, lens, page, seed, width=None, spare=5, window=0, sinks=0):
        rng = np.random.default_rng(seed)
        self.page, self.window, self.sinks = page, window, sinks
        self.len = np.array(lens, dtype=np.int32)
        self.cu = np.concatenate([[0], np.cumsum(ks)]).astype(np.int32)
        self.n_d = int(self.cu[-1])
        need = [-(-max(n, 0) // page) for n in lens]
        self.width = width or max(-(-(n + k + 1) // page) for n, k in zip(lens, ks)) + 1
        n_pages = sum(need) + spare
        order = rng.permutation(n_pages).astype(np.int32)
        self.table = np.full((len(ks), self.width), -1, dtype=np.int32)
        at = 0
        for i, m in enumerate(need):
            self.table[i, :m] = order[at:at + m]
            at += m
        first = int(rng.integers(n_pages))
        self.ring = np.full(n_pages, -7, dtype=np.int32)
        self.ring[(first + np.arange(spare)) % n_pages] = order[at:]
        self.state = np.array([first, spare], dtype=np.int32)

    def args(self):
        t = lambda x: torch.from_numpy(np.array(x)).to(DEV)  # noqa: E731
        return t(self.table), t(self.len), t(self.cu), t(self.ring), t(self.state)

    def check(self):
        table, length, cu, ring, state = self.args()
        placed, slots = sdv.kv_pages(table, length, cu, self.n_d, ring, state, self.page, window=self.window, sinks=self.sinks)
        want = oracle.pages(self.table, self.page, self.len, self.n_d, self.cu, self.ring, self.state, self.window, self.sinks)
        got = [x.cpu().numpy() for x in (table, ring, state, placed, slots)]
        for name, x, y in zip(("table", "ring", "state", "placed", "slots"), got, want):
            assert np.array_equal(x, y), (name, np.argwhere(x != y)[:5], x[x != y][:5], y[x != y][:5])
        self.table, self.ring, self.state = got[:3]
        return got


@pytest.mark.parametrize("page", [1, 2, 16, 1024])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (30, 4), (100, 40), (64, 10000)])
def test_pages(page, window, sinks):
    Pages([0, 3, 40, 0, 100, 7], [0, 17, 300, 31, 0, 640], page, page + window, spare=400, window=window, sinks=sinks).check()


def test_one_request():
    for n, k in ((0, 0), (15, 0), (16, 0), (15, 1), (1000, 4), (0, 5000)):
        got = Pages([k], [n], 16, n, spare=400).check()
        assert got[3].tolist() == [1] and (got[4] >= 0).all()


@pytest.mark.parametrize("spare", [0, 1, 3, 4, 9])
def test_a_ring_that_runs_out(spare):
    got = Pages([20, 0, 70, 0, 5, 0], [8, 16, 3, 5, 31, 16], 16, 3, spare=spare).check()
    assert (got[3] == 0).any() or spare == 9


def test_requests_that_end_and_that_are_rolled_back():
    p = Pages([3, 0, 9, 0, 2], [40, 100, 77, 33, 12], 16, 4, spare=20)
    p.check()
    p.len[:] = [41, -1, 20, 0, -1]  # drafts that were not taken, ended requests, one that starts again
    got = p.check()
    assert got[3].tolist() == [1, 0, 1, 1, 0] and (got[0][[1, 4]] == -1).all()
    p.check()


def test_what_is_passed_over():
    p = Pages([3, 2, 9, 1], [40, 100, 77, 33], 16, 5, spare=20)
    p.len[:] = [40, -2, 2 ** 31 - 1, 2 ** 31 - 1024 - 1]
    got = p.check()
    assert got[3].tolist() == [1, -1, -1, -1]
    p = Pages([3, 2, 9], [40, 100, 77], 16, 6, spare=20, width=7)
    got = p.check()  # the second request's rows end behind the table
    assert got[3].tolist() == [1, 1, 1]
    p = Pages([3, 12, 9], [40, 100, 77], 16, 6, spare=20, width=7)
    assert p.check()[3].tolist() == [1, 0, 1]
    p.len[1] = 2 ** 30
    assert p.check()[3].tolist() == [1, 0, 1]


@pytest.mark.parametrize("bad", [[0, 3, 2, 10], [0, -5, 5, 10], [0, 3, 50, 10], [4, 3, 2, 1], [-1, -1, -1, -1], [0, 3, 5, -1],
                                 [2 ** 31 - 1, 3, 5, 10], [0, 3, -2 ** 31, 10]])
def test_offsets_that_are_not_valid(bad):
    p = Pages([3, 2, 5], [30, 7, 15], 4, 7, spare=20)
    p.cu = np.array(bad, dtype=np.int32)
    p.check()


@pytest.mark.parametrize("state", [[-1, 3], [25, 3], [0, -1], [0, 2 ** 31 - 1], [2 ** 31 - 1, 0], [-2 ** 31, -2 ** 31]])
def test_a_ring_out_of_its_bounds(state):
    p = Pages([3, 2, 5], [30, 7, 15], 4, 8, spare=10)
    p.state[:] = state
    before = p.table.copy()
    got = p.check()
    assert (got[3] == -1).all() and (got[4] == -1).all() and np.array_equal(got[0], before)


def test_numbers_that_are_no_pages():
    p = Pages([3, 2, 5], [30, 7, 15], 4, 9, spare=20)
    p.table[0, 2], p.table[0, 7], p.table[2, 3] = 2 ** 31 - 1, -2 ** 31, len(p.ring)
    p.ring[(p.state[0] + 1) % len(p.ring)] = 10 ** 6  # taken, and no page
    got = p.check()
    assert (got[4] == -1).any()


def test_more_pages_than_the_ring_holds():
    """The same page in several places (which a caller never does) does not write beyond the ring."""
    p = Pages([0, 0, 0], [100, 100, 100], 4, 10, spare=3)
    p.table[:, :20] = 5
    p.len[:] = -1
    got = p.check()
    assert got[2][1] == len(p.ring)


def test_many_requests_and_long_tables():
    rng = np.random.default_rng(11)
    for B, top, page in ((1, 100000, 1), (70, 3000, 2), (300, 900, 16), (1500, 40, 16), (64, 100, 16), (65, 100, 16)):
        ks, lens = rng.integers(0, 9, B), rng.integers(0, top, B)
        p = Pages(ks, lens, page, B, spare=B * 6, window=int(rng.choice([0, 50])), sinks=3)
        p.check()
        p.len = np.where(rng.random(B) < 0.2, -1, p.len + 1 + ks // 2).astype(np.int32)
        p.check()


def test_rounds_keep_every_page():
    """Whatever the rounds do, each page is in one place: a table or the ring."""
    rng = np.random.default_rng(12)
    B, page = 20, 4
    p = Pages([0] * B, [0] * B, page, 12, width=64, spare=150, window=24, sinks=2)
    p.len[:] = rng.integers(0, 30, B)
    for step in range(40):
        ks = rng.integers(0, 12, B)
        p.cu = np.concatenate([[0], np.cumsum(ks)]).astype(np.int32)
        p.n_d = int(p.cu[-1])
        table, ring, state, placed, slots = p.check()
        held = table[table >= 0].tolist() + [int(ring[(state[0] + x) % len(ring)]) for x in range(state[1])]
        assert sorted(held) == list(range(len(ring)))
        grown = p.len + 1 + rng.integers(0, ks + 1)
        p.len = np.where(placed == 1, grown, p.len).astype(np.int32)
        p.len = np.where((rng.random(B) < 0.05) | (p.len > 230), -1, np.where(p.len < 0, 0, p.len)).astype(np.int32)


def test_rows_of_a_padded_batch():
    p = Pages([3, 2], [30, 7], 4, 13, spare=20)
    p.n_d += 9  # rows that no request names
    got = p.check()
    assert (got[4][7:] == -1).all()


def test_without_slots():
    import ctypes

    from lossless_draft_verification_online_amd import _native
    p = Pages([3, 2, 9], [30, 7, 60], 4, 14, spare=20)
    table, length, cu, ring, state = p.args()
    placed = torch.empty(3, dtype=torch.int32, device=DEV)
    ws = torch.empty(_native.lib().sdv_kv_pages_workspace_bytes(300, 64), dtype=torch.uint8, device=DEV)
    at = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    rc = _native.lib().sdv_kv_pages(at(table), 3, p.width, 4, at(length), p.n_d, at(cu), len(p.ring), at(ring), at(state), 0, 0,
                                    at(placed), None, at(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    got = p.check()
    assert np.array_equal(table.cpu().numpy(), got[0]) and np.array_equal(placed.cpu().numpy(), got[3])


@pytest.mark.parametrize("B", [3, 200])
def test_graph_replays(B):
    rng = np.random.default_rng(B)
    p = Pages(rng.integers(0, 9, B), rng.integers(0, 200, B), 16, 15, spare=3 * B, window=64, sinks=4)
    table, length, cu, ring, state = p.args()

    def call():
        return sdv.kv_pages(table, length, cu, p.n_d, ring, state, 16, window=64, sinks=4)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = call()
            graphs.append((g, out))
    torch.cuda.synchronize()
    for step in range(5):
        p.len = np.maximum(p.len + rng.integers(-3, 9, B), -1).astype(np.int32)
        length.copy_(torch.from_numpy(p.len))
        got = p.check()
        torch.cuda.synchronize()
        graphs[step % 2][0].replay()
        torch.cuda.synchronize()
        for x, y in zip((table, ring, state, *graphs[step % 2][1]), got):
            assert np.array_equal(x.cpu().numpy(), y)


def test_refusals():
    p = Pages([3, 2], [30, 7], 4, 16, spare=20)
    table, length, cu, ring, state = p.args()

    def call(**kw):
        a = dict(table=table, length=length, cu=cu, n_d=p.n_d, ring=ring, state=state, page=4)
        a.update({k: kw.pop(k) for k in list(kw) if k in a})
        return sdv.kv_pages(a["table"], a["length"], a["cu"], a["n_d"], a["ring"], a["state"], a["page"], **kw)

    for kw in (dict(table=table.long()), dict(table=table[:1]), dict(table=table.t()), dict(length=length.long()),
               dict(length=length[:1]), dict(cu=cu[:2]), dict(ring=ring.long()), dict(state=state[:1]), dict(n_d=-1),
               dict(table=table.cpu()), dict(slots=torch.empty(3, dtype=torch.int64, device=DEV)),
               dict(placed=torch.empty(2, dtype=torch.int64, device=DEV))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(page=0), dict(page=12), dict(page=2048), dict(window=-1), dict(sinks=-1), dict(placed=length),
               dict(state=ring[:2]), dict(length=state)):
        with pytest.raises(sdv.SdvError):
            call(**kw)
    call()
    many = Pages([0] * 40, [9] * 40, 4, 16)
    table, length, cu, ring, state = many.args()
    with pytest.raises(sdv.SdvError):
        call(table=table, length=length, cu=cu, n_d=0, ring=ring, state=state,
             workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError):
            call(table=table, length=length, cu=cu, n_d=0, ring=ring, state=state, workspace=ws)


@pytest.mark.parametrize("width", [640, 4100, 16385, 50003])
@pytest.mark.parametrize("kept", [1.0, 0.02, 0.0004])
def test_entries_that_change_here_and_there(width, kept):
    """Rows of the table of which few entries, or runs of them, are returned and taken, at every distance from each other."""
    rng = np.random.default_rng(width)
    lens = [(width - 20) * 4, (width - 20) * 2, 64, (width - 20) * 3 + 1]
    p = Pages([30, 17, 200, 3], lens, 4, 12, width=width, spare=300, window=97, sinks=9)
    p.table[rng.random(p.table.shape) > kept] = -1
    got = p.check()
    assert got[3].tolist() == [1, 1, 1, 1]
    p.len[:] = [lens[0] // 3, lens[1] + 5, -1, lens[3] + 2]
    p.table[0, rng.integers(width, size=7)] = got[1][:7]
    assert p.check()[3].tolist() == [1, 1, 0, 1]
