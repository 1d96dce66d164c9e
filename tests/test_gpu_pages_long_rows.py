"""Rows of the table of tens of thousands of entries, of which a wave marks in 64 bits where something changes: every place of its part,
the last ones among them, at the widths where a bit comes to stand for more entries.  Against the oracle."""
import numpy as np
import pytest

from test_gpu_pages import Pages

pytestmark = pytest.mark.gpu

# parts of a quarter each, in chunks of 64 entries: 64, 65, 128, 129, 130, 256 .. 260 and 513 chunks
WIDTHS = [16384, 16385, 32768, 32769, 33000, 33024, 33025, 65536, 65537, 66304, 66305, 131073]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("B", [1, 5])
def test_pages_at_the_ends_of_the_parts(width, B):
    part = -(-width // 256) * 64
    ends = [min((w + 1) * part, width) for w in range(4)]
    rng = np.random.default_rng(width + B)
    # drafts whose pages lie in the last chunks of a part, and some that lie anywhere
    lens = ([e - 70 for e in ends] + [int(rng.integers(width - 70))])[:B] if B > 1 else [ends[0] - 70]
    ks = [66] * len(lens)
    p = Pages(ks, lens, 1, width, width=width, spare=80 * len(lens))
    assert (p.check()[3] == 1).all()
    p.len = (p.len - 5).astype(np.int32)  # drafts that were not taken
    p.cu = np.arange(len(lens) + 1, dtype=np.int32)
    p.n_d = len(lens)
    p.check()
    p.len = (p.len - 60).astype(np.int32)
    got = p.check()
    # every page is in one place
    table, ring, state = got[:3]
    held = table[table >= 0].tolist() + [int(ring[(state[0] + x) % len(ring)]) for x in range(state[1])]
    assert sorted(held) == list(range(len(ring)))


@pytest.mark.parametrize("width", [32769, 33024, 65537, 66000])
def test_ended_requests_return_all_pages(width):
    p = Pages([0, 0, 0], [width - 3, width // 2, width // 4 + 60], 1, width, width=width, spare=10)
    p.len[:] = [-1, 40, -1]
    got = p.check()
    assert got[2][1] == len(p.ring) - 41 and (got[0][[0, 2]] == -1).all()
