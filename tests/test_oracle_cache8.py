"""Pins of the oracle of the cache in 8 bits: the codes against torch's, the scales' limits, requantising, pages by hand."""
import math

import numpy as np
import pytest
import torch

from oracle import cache8 as oracle


def test_codes_are_torchs():
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, oracle.DECODED, equal_nan=True)


def test_nearest_codes_are_torchs():
    x = np.concatenate([np.random.default_rng(0).standard_normal(20000) * 2.0 ** np.random.default_rng(1).integers(-12, 8, 20000),
                        oracle.DECODED[np.isfinite(oracle.DECODED)]])
    p = oracle.DECODED[:127]
    x = np.concatenate([x, (p[1:] + p[:-1]) / 2, -(p[1:] + p[:-1]) / 2]).astype(np.float32)  # ties
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.encode(x), want)


def test_what_lies_beyond_the_codes():
    got = oracle.DECODED[oracle.encode([449.0, 1e30, -1e30, math.inf, -math.inf, math.nan, 2.0 ** -10, 2.0 ** -10 * 1.01])]
    assert got[:3].tolist() == [448.0, 448.0, -448.0] and np.isnan(got[3:6]).all() and got[6:].tolist() == [0.0, 2.0 ** -9]


@pytest.mark.parametrize("limit", [oracle.KEY_LIMIT, oracle.VALUE_LIMIT])
def test_least_scale(limit):
    for e in range(-117, 119):
        edge = limit * 2.0 ** e
        assert oracle.least_byte(edge, limit) == e + 127
        assert oracle.least_byte(np.nextafter(edge, math.inf), limit) == e + 128
    assert oracle.least_byte(0.0, limit) == 10 and oracle.least_byte(2.0 ** -149, limit) == 10
    assert oracle.least_byte(float(np.finfo(np.float32).max), limit) == 246


def test_a_rotation_fits_under_the_keys_limit():
    assert oracle.KEY_LIMIT * math.sqrt(2) < oracle.VALUE_LIMIT < (oracle.KEY_LIMIT + 1) * math.sqrt(2)


def test_codes_keep_their_values_under_larger_scales():
    c = np.arange(256, dtype=np.uint8)
    for shift in range(0, 20):
        v, w = oracle.DECODED[c], oracle.DECODED[oracle.shifted(c, shift)] * 2.0 ** shift
        normal = np.abs(v) * 2.0 ** -shift >= 2.0 ** -6
        assert np.array_equal(v[normal], w[normal])
        finite = np.isfinite(v)
        assert (np.abs(v - w)[finite] <= 2.0 ** (shift - 10)).all() and np.isnan(w[~finite]).all()


def test_pages_by_hand():
    table = np.array([[4, -1, -1, -1], [2, 7, 0, -1], [5, 6, -1, -1]], dtype=np.int32)
    ring, state = np.array([9, 1, 3, 8, 0, 0, 0, 0, 0, 0], dtype=np.int32), np.array([1, 3], dtype=np.int32)
    # request 0: 3 tokens, 3 more rows on pages of 4; request 1 rolled back to 2; request 2 ended
    t, r, s, placed, slots = oracle.pages(table, 4, [3, 2, -1], 2, [0, 2, 2, 2], ring, state)
    assert t.tolist() == [[4, 1, -1, -1], [2, -1, -1, -1], [-1, -1, -1, -1]]
    assert placed.tolist() == [1, 1, 0] and slots.tolist() == [19, 4, 5, 10, -1]
    assert s.tolist() == [2, 6] and [int(r[(2 + x) % 10]) for x in range(6)] == [3, 8, 7, 0, 5, 6]
    # under a window of 2 and 1 sink: the page of slots 0 .. 3 stays, that of 4 .. 7 goes
    t, r, s, placed, slots = oracle.pages([[4, 5, 6, -1]], 4, [11], 1, [0, 1], ring, state, window=2, sinks=1)
    assert t.tolist() == [[4, -1, 6, 1]] and slots.tolist() == [27, 4] and s.tolist() == [2, 3]
    # no pages for the second request's rows, nor for those behind it; one that takes none is placed
    t, r, s, placed, slots = oracle.pages([[-1, -1], [-1, -1], [-1, -1], [4, -1]], 2, [0, 0, 0, 0], 5, [0, 1, 4, 5, 5],
                                          np.array([3, 0, 0, 0, 0, 0, 0]), np.array([6, 2]))
    assert placed.tolist() == [1, 0, 0, 1] and t[1:].tolist() == [[-1, -1], [-1, -1], [4, -1]] and s.tolist() == [0, 1]
