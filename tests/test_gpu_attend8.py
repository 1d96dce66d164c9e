"""Attention over the paged cache in 8 bits, on the GPU against the binary64 oracle over the codes' values.

Tolerances are those of test_gpu_attend: a code times its scale is exact in bf16, so its products are as exact as a bf16
cache's.  With binary32 rows a query and a weight are three bf16 numbers whose sum they are, so a product loses nothing either, but
its three parts are added one after another: three times the roundings of a sum of D (or n) terms.
"""
import math

import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache8_helpers import DEV, Batch8, host
from cache_helpers import DT, np64
from oracle import cache8 as oracle
from oracle.cache import attend as attend64

pytestmark = pytest.mark.gpu


def check(b, window=0, sinks=0, scale=None, q=None, mine=None, out=None):
    D = b.kc.shape[-1]
    got = b.attend(q, window=window, sinks=sinks, scale=scale, out=out)
    s = D ** -0.5 if scale is None else scale
    k, v = b.values()
    ref, mag, span = attend64(np64(b.q), k, v, b.table, b.len, b.cu, s, window, sinks, b.parents)
    n = int(b.len.max()) + int(max(b.ks)) + 1
    times = 3 if b.dtype == "fp32" else 1
    rel = times * (D + 2) * 2.0 ** -24 * span[..., None] + 2.0 ** -22 * (n / 32 + 4) + times * n * 2.0 ** -24
    tol = mag * rel + np.abs(ref) * 2.0 ** -24 + 1e-30
    if b.dtype == "bf16":
        tol += 2.0 ** -8 * mag + 2.0 ** -8 * np.abs(ref)
    bad = ~(np.abs(np64(got) - ref) <= tol)
    if mine is not None:
        bad &= mine[:, None, None]
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], np64(got)[bad][:4], ref[bad][:4], tol[bad][:4])
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 4), (3, 7), (1, 16), (2, 20)])
def test_heads(Hkv, G, D, dtype):
    check(Batch8([0, 3, 8, 1], [0, 17, 300, 31], Hkv, D, 16, 16, dtype, D + G, Hq=Hkv * G))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 5), (1, 0), (1, 1), (33, 0), (64, 4), (100, 40), (5000, 3), (200, 10000)])
def test_windows_and_sinks(window, sinks, dtype):
    check(Batch8([0, 3, 12, 0, 5], [0, 97, 640, 31, 200], 2, 64, 16, 8, dtype, window + sinks, Hq=8), window, sinks)


@pytest.mark.parametrize("page,block", [(1, 1), (2, 1), (8, 8), (16, 1), (16, 4), (32, 32), (128, 64), (1024, 2)])
def test_pages_and_blocks(page, block):
    check(Batch8([0, 2, 7], [1, 130, 777], 2, 128, page, block, "bf16", page, Hq=4), 300, 7)
    check(Batch8([0, 2, 7], [1, 130, 777], 2, 64, page, block, "fp32", page, Hq=4))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (40, 60), (2, 105)])
def test_trees(window, sinks, dtype):
    check(Batch8([0, 64, 12, 30, 1], [3, 100, 0, 63, 7], 2, 64, 16, 8, dtype, window, tree=True, Hq=6), window, sinks)


def test_every_code_and_scale():
    """All finite codes under scales that lie 2^24 apart; and the least and largest scales."""
    rng = np.random.default_rng(0)
    for dtype in ("bf16", "fp32"):
        b = Batch8([3, 9, 0], [70, 33, 200], 2, 128, 16, 4, dtype, 51, Hq=8)
        for c in (b.kc, b.vc):
            c[:] = rng.integers(0, 127, c.shape) | (rng.integers(0, 2, c.shape) << 7)
        b.ks8[:] = rng.integers(105, 120, b.ks8.shape)
        b.vs8[:] = rng.integers(115, 139, b.vs8.shape)
        check(b)
        # bytes beyond the bounds are read as the bounds
        b.ks8[:] = rng.choice([10, 9, 0, 100], b.ks8.shape)
        b.vs8[:] = rng.choice([10, 3, 60], b.vs8.shape)
        check(b, scale=1.0)
        b.vc[:] = rng.integers(0, 8, b.vc.shape)  # subnormal codes
        b.vs8[:] = rng.choice([246, 250, 255], b.vs8.shape)
        check(b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompts(dtype):
    check(Batch8([300, 0, 97], [40, 0, 0], 2, 64, 32, 16, dtype, 1, Hq=4))
    check(Batch8([513], [200], 1, 128, 64, 64, dtype, 2, Hq=5), 128, 4)
    check(Batch8([258, 130], [0, 77], 1, 256, 16, 8, dtype, 3, Hq=2), 50, 0)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 3), (64, 0), (100, 40), (90, 200), (5000, 3)])
def test_prompts_under_windows(window, sinks):
    check(Batch8([127, 300, 64], [33, 500, 0], 1, 128, 16, 16, "bf16", window, Hq=8), window, sinks)
    b = Batch8([127, 300, 64], [33, 500, 0], 2, 64, 64, 8, "bf16", window, Hq=6)
    b.table[1, 2:4] = [-1, b.n_pages]  # pages that are missing
    check(b, window, sinks)


# Batches of 256 columns of a request and more, and 256 workgroups of 128 of them, which the prompts' kernel takes.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [0, 1, 29, 64, 128, 129])
def test_many_heads_of_few_tiles(length, D):
    check(Batch8([27, 31, 33], [length, length + 37, length + 64], 24, D, 16, 4, "bf16", length, Hq=384))


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 3), (64, 0), (100, 40), (90, 200), (5000, 3)])
def test_many_heads_under_windows(window, sinks):
    check(Batch8([127, 300, 64], [33, 500, 0], 8, 128, 16, 16, "bf16", window, Hq=64), window, sinks)
    b = Batch8([127, 300, 64], [33, 500, 0], 16, 64, 64, 32, "bf16", window, Hq=64)
    b.table[1, 2:4] = [-1, b.n_pages]  # pages that are missing
    check(b, window, sinks, scale=-0.2)


@pytest.mark.parametrize("D,page,block", [(64, 16, 1), (128, 32, 2), (128, 128, 64), (64, 1024, 8)])
def test_many_heads_of_other_blocks(D, page, block):
    b = Batch8([127, 300, 64], [33, 200, 0], 8, D, page, block, "bf16", page, Hq=64)
    rng = np.random.default_rng(page)
    b.ks8[:], b.vs8[:] = rng.integers(112, 122, b.ks8.shape), rng.integers(110, 130, b.vs8.shape)
    check(b, 150, 5)


def test_prompts_of_many_requests():
    ks = [(5 * i) % 40 for i in range(150)]
    b = Batch8(ks, [(7 * i) % 90 for i in range(150)], 1, 64, 16, 16, "bf16", 22, Hq=16)
    b.len[70] = -1
    out = check(b, 48, 2)
    lo = int(b.cu[70]) + 70
    assert not out[lo:lo + ks[70] + 1].any()
    b.len[70] = 2 ** 31 - 1024 - ks[70]
    assert torch.equal(b.attend(window=48, sinks=2), out)


def test_long_caches_are_split():
    check(Batch8([0], [9000], 1, 128, 16, 16, "bf16", 4, Hq=8))
    check(Batch8([4, 0], [5000, 20], 1, 64, 16, 4, "fp32", 5, Hq=4), 4096, 4)
    check(Batch8([0, 1], [6000, 0], 1, 256, 64, 32, "bf16", 6, Hq=4))
    check(Batch8([2, 1], [6000, 40], 1, 128, 128, 64, "fp32", 7, Hq=20))
    check(Batch8([2, 1, 8], [1700, 40, 1600], 3, 128, 16, 16, "bf16", 8, Hq=12))
    check(Batch8([70], [3000], 2, 64, 16, 16, "bf16", 9, Hq=8), 0, 0)  # many columns of one request
    check(Batch8([0, 0], [20000, 7], 1, 128, 64, 64, "bf16", 10, Hq=4))  # units of many pieces
    check(Batch8([20, 64], [2500, 3000], 1, 64, 16, 8, "fp32", 11, tree=True, Hq=4), 2000, 3)


def test_long_caches_of_many_requests():
    """More requests than a wave has lanes, some of them empty or not valid, in ranges."""
    rng = np.random.default_rng(9)
    for B, dtype in ((70, "bf16"), (100, "fp32"), (130, "bf16")):
        lens = np.where(rng.random(B) < 0.08, rng.integers(3000, 4500, B), rng.integers(0, 60, B))
        lens[-1] = 6500
        b = Batch8(rng.integers(0, 4, B), lens, 1, 64, 16, 16, dtype, B, Hq=4)
        b.len[5] = -1
        check(b)


def test_many_requests():
    rng = np.random.default_rng(7)
    check(Batch8(rng.integers(0, 6, 200), rng.integers(0, 90, 200), 1, 64, 16, 16, "bf16", 8, Hq=4), 40, 2)
    check(Batch8(rng.integers(0, 6, 100), rng.integers(0, 2000, 100), 1, 64, 16, 16, "bf16", 8, Hq=4))


def test_strided_queries_and_scales():
    b = Batch8([3, 1], [50, 20], 2, 64, 16, 16, "bf16", 9, Hq=4)
    wide = torch.randn((b.rows, 9, 64)).to(torch.bfloat16)
    wide[:, :4] = b.q
    check(b, q=wide.to(DEV)[:, :4])
    prompt = Batch8([130, 70], [50, 20], 2, 64, 16, 16, "bf16", 9, Hq=4)
    many = Batch8([130, 70], [50, 20], 24, 64, 16, 16, "bf16", 9, Hq=192)
    for scale in (0.0, 1.0, -0.5):
        check(b, scale=scale)
        check(prompt, 60, 3, scale=scale)
        check(many, 60, 3, scale=scale)
    b = Batch8([3, 1], [500, 20], 2, 64, 16, 16, "fp32", 10, Hq=4)
    b.q *= 30  # far apart scores: most weights vanish
    check(b, scale=1.0)
    check(b, scale=-1.0)


CASES = [([2, 0, 5], False, 128, "bf16", 4, 2), ([2, 0, 5], False, 128, "fp32", 4, 2), ([2, 0, 5], False, 64, "bf16", 8, 2),
         ([2, 0, 5], True, 256, "bf16", 4, 2), ([200, 100, 260], False, 128, "bf16", 128, 16),
         ([200, 100, 260], False, 64, "bf16", 128, 16)]


@pytest.mark.parametrize("ks,tree,D,dtype,Hq,Hkv", CASES)
def test_what_no_row_sees_may_hold_anything(ks, tree, D, dtype, Hq, Hkv):
    """NaN codes behind the last row, before the window, in pages of nobody and in freed places, under any scale."""
    b = Batch8(ks, [70, 9, 333], Hkv, D, 16, 4, dtype, 11, Hq=Hq, tree=tree)
    window, sinks = 64, 4
    want = check(b, window, sinks)
    seen = np.zeros((b.n_pages, 16), dtype=bool)
    for i, _, K, L, _, _ in oracle.requests(b.cu, b.len, b.n_d, b.parents):
        for s in range(L + K + 1):
            if s < sinks or s > L - window:
                seen[oracle.place(b.table[i], b.n_pages, 16, s)] = True
    for c in (b.kc, b.vc):
        c[np.broadcast_to(~seen[:, None, :, None], c.shape)] = 0xff
    blocks = seen.reshape(b.n_pages, 4, 4).any(-1)
    for c in (b.ks8, b.vs8):
        c[np.broadcast_to(~blocks[:, None], c.shape)] = 255
    assert torch.equal(b.attend(window=window, sinks=sinks), want)


@pytest.mark.parametrize("ks,tree,D,dtype,page,Hq", [
    ([12, 5, 3], False, 64, "bf16", 16, 2), ([12, 5, 3], False, 128, "bf16", 16, 8), ([12, 5, 3], False, 128, "bf16", 4, 8),
    ([12, 5, 3], False, 256, "bf16", 32, 4), ([12, 5, 3], False, 64, "fp32", 16, 8), ([12, 5, 3], False, 256, "fp32", 16, 2),
    ([30, 12, 9], True, 64, "bf16", 16, 8), ([30, 12, 9], True, 64, "fp32", 16, 8),
    ([200, 150, 260], False, 128, "bf16", 16, 16), ([200, 150, 260], False, 64, "bf16", 64, 16)])
def test_rows_that_do_not_see_a_value(ks, tree, D, dtype, page, Hq):
    """A value of one slot that is no number reaches the rows that see the slot, and no other."""
    Hkv = 2 if Hq < 16 else 4
    b = Batch8(ks, [70, 33, 130], Hkv, D, page, 4, dtype, 31, tree=tree, Hq=Hq if Hq < 16 else 64)
    window, sinks = 40, 2
    want = b.attend(window=window, sinks=sinks).float().cpu()
    hit = torch.zeros(b.rows, dtype=torch.bool)
    for i, row0, K, L, d, see in oracle.requests(b.cu, b.len, b.n_d, b.parents):
        for slot in (L + K // 2, max(L - 36, sinks)):  # a draft's own, and one that leaves the window on the way
            place = oracle.place(b.table[i], b.n_pages, page, slot)
            b.vc[place[0], :, place[1], 3] = 0x7f
            for j in range(K + 1):
                position = slot if slot < L else L + d[slot - L]
                seen = slot < L or slot - L in see[j]
                hit[row0 + j] |= seen and L + d[j] - position < window
    out = b.attend(window=window, sinks=sinks).float().cpu()
    assert hit.any() and not hit.all()
    assert torch.equal(out[~hit], want[~hit])
    assert torch.isnan(out[hit][..., 3]).all()
    rest = [k for k in range(D) if k != 3]
    assert torch.equal(out[hit][..., rest], want[hit][..., rest])


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "fp32"), (128, "fp32")])
def test_keys_that_are_no_numbers(D, dtype):
    b = Batch8([12, 5, 30], [1500, 33, 2900], 2, D, 16, 16, dtype, 32, Hq=8)
    want = b.attend().float().cpu()
    hit = torch.zeros(b.rows, dtype=torch.bool)
    for i, row0, K, L, _, _ in oracle.requests(b.cu, b.len, b.n_d):
        place = oracle.place(b.table[i], b.n_pages, 16, L + K // 2)
        b.vc[place[0], :, place[1], 5] = 0xff
        b.kc[place[0], :, place[1], 7] = 0x7f
        hit[row0 + K // 2:row0 + K + 1] = True
    out = b.attend().float().cpu()
    assert torch.equal(out[~hit], want[~hit]) and torch.isnan(out[hit]).all()


def test_queries_that_are_not_finite():
    for dtype in ("bf16", "fp32"):
        b = Batch8([3, 0], [40, 20], 2, 64, 16, 16, dtype, 33, Hq=4)
        want = b.attend().float().cpu()
        b.q[1, 2, 7], b.q[2, 0, 9], b.q[4, 3] = math.inf, math.nan, torch.finfo(DT[dtype]).max
        out = b.attend().float().cpu()
        same = torch.ones(out.shape[:2], dtype=torch.bool)
        same[1, 2] = same[2, 0] = same[4, 3] = False
        assert torch.equal(out[same], want[same])
        assert torch.isnan(out[1, 2]).all() and torch.isnan(out[2, 0]).all()


def test_pages_that_left_the_window_and_pages_that_are_missing():
    b = Batch8([2, 0, 5], [70, 200, 333], 2, 64, 16, 8, "bf16", 12, Hq=4)
    want = check(b, 64, 3)
    b.table[1, 1:8] = -1  # slots 16 .. 127: out of the window of position 200
    b.table[2, 1:16] = [-1, b.n_pages, 2 ** 31 - 1, -2 ** 31, -7] * 3
    assert torch.equal(check(b, 64, 3), want)
    b.table[0, 1] = -1  # missing inside the window: not seen
    b.table[2, :] = -1  # nothing left to see: zeros
    out = check(b, 64, 3)
    assert not out[4:].any() and out[:3].any()


def test_requests_that_are_passed_over():
    b = Batch8([2, 1, 5, 3], [70, 20, 33, 4], 2, 64, 16, 8, "bf16", 13, Hq=4)
    b.len[1] = -3
    assert not check(b)[3:5].any()
    b = Batch8([2, 3, 5], [70, 20, 33], 2, 64, 16, 8, "bf16", 14, Hq=4, tree=True)
    b.parents[3] = 1
    assert not check(b)[3:7].any()
    b = Batch8([70, 3], [10, 20], 2, 64, 16, 8, "bf16", 15, Hq=4, tree=True)
    assert not check(b)[:71].any()
    b = Batch8([3, 2, 5], [30, 7, 15], 1, 64, 16, 8, "bf16", 16, Hq=2)
    b.len[0] = 16 * b.table.shape[1] - 1  # rows behind the table's end
    check(b)


SMALL = [[0, 3, 2, 10], [0, -5, 5, 10], [0, 3, 50, 10], [4, 3, 2, 1], [-1, -1, -1, -1], [0, 3, -5, 10], [0, 3, 5, -1],
         [0, 3, -2 ** 31, 10], [-7, 3, 5, 10], [0, 2 ** 31 - 1, 5, 10], [2 ** 31 - 1, 3, 5, 10]]


def check_offsets(b, window=0, sinks=0):
    mine = np.zeros(b.rows, dtype=bool)
    for _, row0, K, *_ in oracle.requests(b.cu, b.len, b.n_d, b.parents):
        mine[row0:row0 + K + 1] = True
    out = torch.full(b.q.shape, 5.0, dtype=DT[b.dtype], device=DEV)
    check(b, window, sinks, mine=mine, out=out)
    assert (out[torch.from_numpy(~mine)] == 5.0).all()


@pytest.mark.parametrize("bad", SMALL)
@pytest.mark.parametrize("dtype,Hq,page", [("bf16", 2, 16), ("fp32", 16, 16), ("bf16", 16, 4)])
def test_offsets_that_are_not_valid(bad, dtype, Hq, page):
    b = Batch8([3, 2, 5], [30, 7, 15], 1, 64, page, 2, dtype, 16, Hq=Hq)
    b.cu = np.array(bad, dtype=np.int32)
    check_offsets(b)


@pytest.mark.parametrize("at,bad", [(1, -5), (1, 10 ** 6), (2, -5), (2, 2 ** 31 - 1), (3, -1), (0, -5)])
def test_prompts_beside_an_offset(at, bad):
    b = Batch8([27, 31, 33], [20, 57, 84], 24, 64, 16, 16, "bf16", at, Hq=384)
    b.cu[at] = bad
    check_offsets(b)
    ks = [(5 * i) % 40 + 8 for i in range(150)]
    b = Batch8(ks, [(7 * i) % 90 for i in range(150)], 1, 64, 16, 16, "bf16", 22, Hq=16)
    b.cu[at * 49] = bad
    check_offsets(b, 48, 2)


@pytest.mark.parametrize("ks,lens,dtype", [([3, 0, 7], [20, 90, 5], "bf16"), ([3, 0, 7], [20, 90, 5], "fp32"),
                                           ([3, 0, 7], [20, 1900, 5], "bf16"), ([200, 130, 70], [20, 90, 5], "bf16")])
def test_rows_behind_the_last_request_stay(ks, lens, dtype):
    b = Batch8(ks, lens, 16, 64, 16, 16, dtype, 40, Hq=128)
    want = b.attend()
    out = torch.full((b.rows + 9,) + b.q.shape[1:], 5.0, dtype=DT[dtype], device=DEV)
    b.attend(torch.cat([b.q, b.q[:9]]).to(DEV), out=out)
    assert (out[b.rows:] == 5.0).all()
    assert (out[:b.rows].float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()


@pytest.mark.parametrize("ks,lens,dtype", [([3, 0, 7], [20, 90, 5], "bf16"), ([3, 0, 7], [20, 90, 5], "fp32"),
                                           ([3, 0, 7], [20, 1900, 5], "bf16"), ([400, 230, 170], [20, 90, 5], "bf16")])
def test_caches_of_more_than_32_bit_offsets(ks, lens, dtype):
    b = Batch8(ks, lens, 8, 128, 16, 4, dtype, 41, Hq=64)
    want = b.attend()
    first = (2 ** 32 + 2 ** 31) // (8 * 16 * 128)  # pages from 6 GiB on
    big = []
    for t in b.caches():
        x = torch.empty((first + b.n_pages,) + t.shape[1:], dtype=torch.uint8, device=DEV)
        x[first:] = t.view(torch.uint8)
        big.append(x.view(t.dtype))
    b.table = np.where(b.table >= 0, b.table + first, b.table).astype(np.int32)
    assert torch.equal(b.attend(caches=big), want)


def test_it_is_the_attention_over_a_bf16_cache_of_the_same_values():
    b = Batch8([4, 0, 2], [100, 50, 30], 2, 128, 16, 16, "bf16", 17, Hq=4)
    table, length, cu = b.index_args()
    k, v = (torch.from_numpy(x).to(torch.bfloat16).to(DEV) for x in b.values())  # exact
    want = sdv.attend(b.q.to(DEV), k, v, table, length, cu, window=40, sinks=2)
    got = b.attend(window=40, sinks=2)
    assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
    assert torch.equal(b.attend(window=40, sinks=2), got)


@pytest.mark.parametrize("ks,lens", [([4, 0, 2], [3000, 50, 30]), ([130, 100, 90], [300, 50, 30])])
def test_graph_replays(ks, lens):
    b = Batch8(ks, lens, 16, 128, 16, 16, "bf16", 18, Hq=128)
    table, length, cu = b.index_args()
    q = b.q.to(DEV)
    kc, vc, ks8, vs8 = b.caches()

    def call():
        return sdv.attend(q, kc, vc, table, length, cu, key_scales=ks8, value_scales=vs8)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        call()
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = call()
            graphs.append((g, out))
    torch.cuda.synchronize()
    for step in range(4):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(step)))
        length.copy_(torch.tensor([lens[0] - 7 * step, 50, 30 + step // 2], dtype=torch.int32))
        want = call()
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out, want)


def test_refusals():
    b = Batch8([2, 0], [5, 7], 2, 64, 16, 8, "bf16", 19, Hq=4)
    q = b.q.to(DEV)
    b.attend(q)
    for bad in (q[:1], q[:, :3], q.transpose(0, 1), q[:, :, :32]):
        with pytest.raises(ValueError):
            b.attend(bad)
    with pytest.raises(TypeError):
        b.attend(q.half())
    for kw in (dict(window=-1), dict(sinks=-1), dict(scale=math.inf), dict(scale=math.nan)):
        with pytest.raises(sdv.SdvError):
            b.attend(q, **kw)
    with pytest.raises(ValueError):
        b.attend(q, out=torch.empty_like(q)[:2])
    kc, vc, ks, vs = b.caches()
    table, length, cu = b.index_args()
    for kw in (dict(key_scales=ks), dict(key_scales=ks, value_scales=vs[:1]), dict(key_scales=ks.float(), value_scales=vs)):
        with pytest.raises(ValueError):
            sdv.attend(q, kc, vc, table, length, cu, **kw)
    with pytest.raises(TypeError):
        sdv.attend(q, kc, vc, table, length, cu)
    long = Batch8([0], [9000], 1, 128, 16, 16, "bf16", 4, Hq=8)
    with pytest.raises(sdv.SdvError):
        long.attend(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert host(ks).shape == (b.n_pages, 2, 2)


def test_a_workspace_that_the_gpu_does_not_hold_as_one_piece():
    b = Batch8([0], [9000], 1, 128, 16, 16, "bf16", 4, Hq=8)
    for ws in (torch.empty(1 << 24, dtype=torch.uint8), torch.empty(1 << 24, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError):
            b.attend(workspace=ws)
    assert torch.equal(b.attend(workspace=torch.empty(1 << 24, dtype=torch.uint8, device=DEV)), b.attend())
