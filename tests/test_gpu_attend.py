"""Attention over the paged cache on the GPU against the binary64 oracle.

Tolerance of an output value o = sum p v with A = sum p |v|.  A score is a binary32 sum of D products (bf16
products are exact in binary32), so it is off by at most (D + 2) 2^-24 sum |q k| scale, and so is its weight
relatively; the exponential and the running rescales add 2^-22 per step of the longest chain of maxima (at
most the number of 32-token tiles a wave takes, joined over waves and splits); the sums over the n visible
tokens n 2^-24.  With bf16 a weight is rounded to 2^-8 for its product, and the result to 2^-8 of itself.
"""
import math

import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from oracle import cache as oracle
from cache_helpers import DEV, DT, Batch, np64

pytestmark = pytest.mark.gpu


def check(b, dtype, window=0, sinks=0, scale=None, q=None):
    table, length, cu = b.index_args()
    D = b.kc.shape[-1]
    args = (q if q is not None else b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, cu)
    out = sdv.attend(*args, parents=b.tree_arg(), scale=scale, window=window, sinks=sinks)
    s = D ** -0.5 if scale is None else scale
    ref, mag, span = oracle.attend(np64(b.q), np64(b.kc), np64(b.vc), b.table, b.len, b.cu, s, window, sinks, b.parents)
    n = int(b.len.max()) + int(max(b.ks)) + 1
    rel = (D + 2) * 2.0 ** -24 * span[..., None] + 2.0 ** -22 * (n / 32 + 4) + n * 2.0 ** -24
    tol = mag * rel + np.abs(ref) * 2.0 ** -24 + 1e-30
    if dtype == "bf16":
        tol += 2.0 ** -8 * mag + 2.0 ** -8 * np.abs(ref)
    got = np64(out)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 4), (3, 7), (1, 16), (2, 20)])
def test_heads(Hkv, G, D, dtype):
    check(Batch([0, 3, 8, 1], [0, 17, 300, 31], Hkv, D, 16, dtype, D + G, Hq=Hkv * G), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 5), (1, 0), (1, 1), (33, 0), (64, 4), (100, 40), (5000, 3), (200, 10000)])
def test_windows_and_sinks(window, sinks, dtype):
    check(Batch([0, 3, 12, 0, 5], [0, 97, 640, 31, 200], 2, 64, 16, dtype, window + sinks, Hq=8), dtype, window, sinks)


@pytest.mark.parametrize("page", [1, 2, 8, 32, 128, 1024])
def test_pages(page):
    check(Batch([0, 2, 7], [1, 130, 777], 2, 128, page, "bf16", page, Hq=4), "bf16", 300, 7)
    check(Batch([0, 2, 7], [1, 130, 777], 2, 64, page, "fp32", page, Hq=4), "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (40, 60), (2, 105)])
def test_trees(window, sinks, dtype):
    check(Batch([0, 64, 12, 30, 1], [3, 100, 0, 63, 7], 2, 64, 16, dtype, window, tree=True, Hq=6), dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompts(dtype):
    check(Batch([300, 0, 97], [40, 0, 0], 2, 64, 32, dtype, 1, Hq=4), dtype)
    check(Batch([513], [200], 1, 128, 64, dtype, 2, Hq=5), dtype, 128, 4)
    check(Batch([258, 130], [0, 77], 1, 256, 16, dtype, 3, Hq=2), dtype, 50, 0)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 3), (64, 0), (100, 40), (90, 200), (5000, 3)])
def test_prompts_under_windows(window, sinks):
    check(Batch([127, 300, 64], [33, 500, 0], 1, 128, 16, "bf16", window, Hq=8), "bf16", window, sinks)
    b = Batch([127, 300, 64], [33, 500, 0], 2, 64, 64, "bf16", window, Hq=6)
    b.table[1, 2:4] = [-1, b.n_pages]  # pages that are missing
    check(b, "bf16", window, sinks)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [0, 1, 29, 64, 128, 129])
def test_prompts_of_few_tiles(length, D):
    check(Batch([27, 31, 33], [length, length + 37, length + 64], 2, D, 16, "bf16", length, Hq=8), "bf16")


# Batches of 128 workgroups of 128 columns and more, which the prompts' kernel takes.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [0, 1, 29, 64, 128, 129])
def test_many_heads_of_few_tiles(length, D):
    check(Batch([27, 31, 33], [length, length + 37, length + 64], 48, D, 16, "bf16", length, Hq=192), "bf16")


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 3), (64, 0), (100, 40), (90, 200), (5000, 3)])
def test_many_heads_under_windows(window, sinks):
    check(Batch([127, 300, 64], [33, 500, 0], 4, 128, 16, "bf16", window, Hq=32), "bf16", window, sinks)
    b = Batch([127, 300, 64], [33, 500, 0], 8, 64, 64, "bf16", window, Hq=32)
    b.table[1, 2:4] = [-1, b.n_pages]  # pages that are missing
    check(b, "bf16", window, sinks, scale=-0.2)


def test_what_no_row_of_many_heads_sees_may_hold_anything():
    b = Batch([200, 100], [300, 9], 16, 128, 16, "bf16", 20, Hq=128)
    window, sinks = 64, 3
    args = b.index_args()

    def run(length):
        return sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), args[0], length, args[2], window=window, sinks=sinks)

    want = check(b, "bf16", window, sinks)
    seen = np.zeros((b.n_pages, 16), dtype=bool)
    for i, _, K, L, _, _ in oracle.requests(b.cu, b.len, b.n_d):
        for s in range(L + K + 1):
            if s < sinks or s > L - window:
                seen[oracle.place(b.table[i], b.n_pages, 16, s)] = True
    for c in (b.kc, b.vc):
        c[torch.from_numpy(~seen)[:, None, :, None].expand(c.shape)] = float("nan")
    assert torch.equal(run(args[1]), want)
    b.len[0] = -1
    out = run(torch.from_numpy(b.len).to(DEV))
    assert not out[:201].any() and torch.equal(out[201:], want[201:])


def test_many_heads_with_offsets_that_are_not_valid():
    b = Batch([100, 130, 100], [30, 0, 70], 16, 64, 16, "bf16", 23, Hq=128)
    table, length, cu = b.index_args()
    q, kc, vc = b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV)
    want = sdv.attend(q, kc, vc, table, length, cu)
    for bad in ([0, 100, 230, 331], [0, 100, 90, 330], [0, -5, 230, 330], [400, 300, 200, 100], [-1, -1, -1, -1],
                [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 5]):
        out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=DEV)
        sdv.attend(q, kc, vc, table, length, torch.tensor(bad, dtype=torch.int32, device=DEV), out=out)
        if bad[:3] == [0, 100, 230]:  # the requests before are as they were
            assert torch.equal(out[:232], want[:232]) and (out[232:] == 5.0).all()


def test_prompts_of_many_requests():
    ks = [(5 * i) % 40 for i in range(150)]
    b = Batch(ks, [(7 * i) % 90 for i in range(150)], 1, 64, 16, "bf16", 22, Hq=16)
    b.len[70] = -1
    out = check(b, "bf16", 48, 2)
    lo = int(b.cu[70]) + 70
    assert not out[lo:lo + ks[70] + 1].any()
    b.len[70] = 2 ** 31 - 1024 - ks[70]
    table, length, cu = b.index_args()
    assert torch.equal(sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, cu, window=48, sinks=2), out)


def test_what_no_row_of_a_prompt_sees_may_hold_anything():
    b = Batch([200, 100], [300, 9], 2, 128, 16, "bf16", 20, Hq=4)
    window, sinks = 64, 3
    want = check(b, "bf16", window, sinks)
    seen = np.zeros((b.n_pages, 16), dtype=bool)
    for i, _, K, L, _, _ in oracle.requests(b.cu, b.len, b.n_d):
        for s in range(L + K + 1):
            if s < sinks or s > L - window:
                seen[oracle.place(b.table[i], b.n_pages, 16, s)] = True
    for c in (b.kc, b.vc):
        c[torch.from_numpy(~seen)[:, None, :, None].expand(c.shape)] = float("nan")
    table, length, cu = b.index_args()
    out = sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, cu, window=window, sinks=sinks)
    assert torch.equal(out, want)
    b.len[0] = -1
    length = torch.from_numpy(b.len).to(DEV)
    out = sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, cu, window=window, sinks=sinks)
    assert not out[:201].any() and torch.equal(out[201:], want[201:])


def test_long_caches_are_split():
    check(Batch([0], [9000], 1, 128, 16, "bf16", 4, Hq=8), "bf16")
    check(Batch([4, 0], [5000, 20], 1, 64, 16, "fp32", 5, Hq=4), "fp32", 4096, 4)
    check(Batch([0, 1], [6000, 0], 1, 256, 64, "bf16", 6, Hq=4), "bf16", 0, 0)


def test_many_requests():
    rng = np.random.default_rng(7)
    check(Batch(rng.integers(0, 6, 200), rng.integers(0, 90, 200), 1, 64, 16, "bf16", 8, Hq=4), "bf16", 40, 2)


def test_strided_queries_and_scales():
    b = Batch([3, 1], [50, 20], 2, 64, 16, "bf16", 9, Hq=4)
    wide = torch.randn((b.rows, 9, 64)).to(torch.bfloat16)
    wide[:, :4] = b.q
    check(b, "bf16", q=wide.to(DEV)[:, :4])
    prompt = Batch([130, 70], [50, 20], 2, 64, 16, "bf16", 9, Hq=4)
    for scale in (0.0, 1.0, -0.5):
        check(b, "bf16", scale=scale)
        check(prompt, "bf16", 60, 3, scale=scale)
    b = Batch([3, 1], [500, 20], 2, 64, 16, "fp32", 10, Hq=4)
    b.q *= 30  # far apart scores: most weights vanish
    check(b, "fp32", scale=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_what_no_row_sees_may_hold_anything(dtype):
    """NaN and infinities behind the last row, before the window, in pages of nobody and in freed places."""
    b = Batch([2, 0, 5], [70, 9, 333], 2, 128, 16, dtype, 11, Hq=4)
    window, sinks = 64, 3
    want = check(b, dtype, window, sinks)
    seen = np.zeros((b.n_pages, 16), dtype=bool)
    for i, _, K, L, _, _ in oracle.requests(b.cu, b.len, b.n_d):
        for s in range(L + K + 1):
            if s < sinks or s > L - window:
                p = oracle.place(b.table[i], b.n_pages, 16, s)
                seen[p] = True
    for c in (b.kc, b.vc):
        hole = torch.from_numpy(~seen)[:, None, :, None].expand(c.shape)
        c[hole] = torch.tensor([float("nan"), float("inf"), -float("inf")]).to(c.dtype).repeat(c.numel())[:int(hole.sum())]
    table, length, cu = b.index_args()
    out = sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, cu, window=window, sinks=sinks)
    assert torch.equal(out, want)


def test_pages_that_left_the_window_and_pages_that_are_missing():
    b = Batch([2, 0, 5], [70, 200, 333], 2, 64, 16, "bf16", 12, Hq=4)
    want = check(b, "bf16", 64, 3)
    b.table[1, 1:8] = -1  # slots 16 .. 127: out of the window of position 200
    b.table[2, 1:16] = [-1, b.n_pages, 2 ** 31 - 1, -2 ** 31, -7] * 3
    assert torch.equal(check(b, "bf16", 64, 3), want)
    b.table[0, 1] = -1  # missing inside the window: not seen
    b.table[2, :] = -1  # nothing left to see: zeros
    out = check(b, "bf16", 64, 3)
    assert not out[4:].any() and out[:3].any()


def test_requests_that_are_passed_over():
    b = Batch([2, 1, 5, 3], [70, 20, 33, 4], 2, 64, 16, "bf16", 13, Hq=4)
    b.len[1] = -3
    assert not check(b, "bf16")[3:5].any()
    b = Batch([2, 3, 5], [70, 20, 33], 2, 64, 16, "bf16", 14, Hq=4, tree=True)
    b.parents[3] = 1
    assert not check(b, "bf16")[3:7].any()
    b = Batch([70, 3], [10, 20], 2, 64, 16, "bf16", 15, Hq=4, tree=True)
    assert not check(b, "bf16")[:71].any()
    b = Batch([3, 2, 5], [30, 7, 15], 1, 64, 16, "bf16", 16, Hq=2)
    b.len[0] = 16 * b.table.shape[1] - 1  # rows behind the table's end
    check(b, "bf16")
    table, length, _ = b.index_args()
    for bad in ([0, 3, 2, 10], [0, -5, 5, 10], [0, 3, 50, 10], [4, 3, 2, 1], [-1, -1, -1, -1]):
        out = torch.full((13, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
        sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, torch.tensor(bad, dtype=torch.int32, device=DEV),
                   out=out)
        torch.cuda.synchronize()


def test_a_row_does_not_depend_on_its_batch():
    b = Batch([4, 0, 2], [100, 50, 30], 2, 128, 16, "fp32", 17, Hq=4)
    table, length, cu = b.index_args()
    args = (b.kc.to(DEV), b.vc.to(DEV))
    first = sdv.attend(b.q.to(DEV), *args, table, length, cu, window=40, sinks=2)
    again = sdv.attend(b.q.to(DEV), *args, table, length, cu, window=40, sinks=2)
    assert torch.equal(first, again)
    one = sdv.attend(b.q[5:6].to(DEV), *args, table[1:2].contiguous(), length[1:2].contiguous(),
                     torch.zeros(2, dtype=torch.int32, device=DEV), window=40, sinks=2)
    assert (one - first[5:6]).abs().max() <= 2.0 ** -18 * first.abs().max()


def test_graph_replays():
    b = Batch([4, 0, 2], [3000, 50, 30], 2, 128, 16, "bf16", 18, Hq=4)
    table, length, cu = b.index_args()
    q, kc, vc = b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        sdv.attend(q, kc, vc, table, length, cu)
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = sdv.attend(q, kc, vc, table, length, cu)
            graphs.append((g, out))
    torch.cuda.synchronize()
    for step in range(4):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(step)))
        length.copy_(torch.tensor([3000 - 7 * step, 50, 30 + step // 2], dtype=torch.int32))
        want = sdv.attend(q, kc, vc, table, length, cu)
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out, want)


def test_refusals():
    b = Batch([2, 0], [5, 7], 2, 64, 16, "bf16", 19, Hq=4)
    table, length, cu = b.index_args()
    q, kc, vc = b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV)
    for bad in (q.float(), q[:1], q[:, :3], q.transpose(0, 1), q[:, :, :32]):
        with pytest.raises(ValueError):
            sdv.attend(bad, kc, vc, table, length, cu)
    for kw in (dict(window=-1), dict(sinks=-1), dict(scale=math.inf), dict(scale=math.nan)):
        with pytest.raises(sdv.SdvError):
            sdv.attend(q, kc, vc, table, length, cu, **kw)
    with pytest.raises(ValueError):
        sdv.attend(q, kc, vc, table, length, cu, out=torch.empty_like(q)[:2])
    long = Batch([0], [9000], 1, 128, 16, "bf16", 4, Hq=8)
    table, length, cu = long.index_args()
    with pytest.raises(sdv.SdvError):
        sdv.attend(long.q.to(DEV), long.kc.to(DEV), long.vc.to(DEV), table, length, cu,
                   workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
@pytest.mark.parametrize("ks,tree,D,dtype,page,Hq", [
    ([12, 5, 3], False, 64, "bf16", 16, 2), ([12, 5, 3], False, 128, "bf16", 16, 8), ([12, 5, 3], False, 128, "bf16", 4, 8),
    ([12, 5, 3], False, 256, "bf16", 32, 4), ([12, 5, 3], False, 64, "fp32", 16, 8), ([12, 5, 3], False, 256, "fp32", 16, 2),
    ([30, 12, 9], True, 64, "bf16", 16, 8), ([30, 12, 9], True, 64, "fp32", 16, 8),
    ([200, 150, 260], False, 128, "bf16", 16, 16), ([200, 150, 260], False, 64, "bf16", 64, 16)])
def test_rows_that_do_not_see_a_value(ks, tree, D, dtype, page, Hq, poison):
    # a value of one slot that is not finite reaches the rows that see the slot, and no other
    Hkv = 2 if Hq < 16 else 4
    b = Batch(ks, [70, 33, 130], Hkv, D, page, dtype, 31, tree=tree, Hq=Hq if Hq < 16 else 64)
    table, length, cu = b.index_args()
    window, sinks = 40, 2

    def run():
        return sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, cu, parents=b.tree_arg(), window=window,
                          sinks=sinks).float().cpu()

    want = run()
    hit = torch.zeros(b.rows, dtype=torch.bool)
    for i, row0, K, L, d, see in oracle.requests(b.cu, b.len, b.n_d, b.parents):
        for slot in (L + K // 2, max(L - 36, sinks)):  # a draft's own, and one that leaves the window on the way
            place = oracle.place(b.table[i], b.n_pages, page, slot)
            b.vc[place[0], :, place[1], 3] = poison
            for j in range(K + 1):
                position = slot if slot < L else L + d[slot - L]
                seen = slot < L or slot - L in see[j]
                hit[row0 + j] |= seen and L + d[j] - position < window
    out = run()
    assert hit.any() and not hit.all()
    assert torch.equal(out[~hit], want[~hit])
    assert not torch.isfinite(out[hit][..., 3]).any()
    rest = [k for k in range(D) if k != 3]
    assert torch.equal(out[hit][..., rest], want[hit][..., rest])


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "fp32"), (128, "fp32")])
def test_rows_of_long_caches_that_do_not_see_a_value(D, dtype):
    b = Batch([12, 5, 30], [1500, 33, 2900], 2, D, 16, dtype, 32, Hq=8)
    table, length, cu = b.index_args()
    want = sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, cu).float().cpu()
    hit = torch.zeros(b.rows, dtype=torch.bool)
    for i, row0, K, L, _, _ in oracle.requests(b.cu, b.len, b.n_d):
        place = oracle.place(b.table[i], b.n_pages, 16, L + K // 2)
        b.vc[place[0], :, place[1], 5] = math.nan
        b.kc[place[0], :, place[1], 7] = math.nan
        hit[row0 + K // 2:row0 + K + 1] = True
    out = sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, cu).float().cpu()
    assert torch.equal(out[~hit], want[~hit]) and torch.isnan(out[hit]).all()


@pytest.mark.parametrize("ks,lens,dtype", [([3, 0, 7], [20, 90, 5], "bf16"), ([3, 0, 7], [20, 90, 5], "fp32"),
                                           ([3, 0, 7], [20, 1900, 5], "bf16"), ([200, 130, 70], [20, 90, 5], "bf16")])
def test_rows_behind_the_last_request_stay(ks, lens, dtype):
    b = Batch(ks, lens, 8, 64, 16, dtype, 40, Hq=64)
    table, length, cu = b.index_args()
    want = sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, cu)
    q = torch.cat([b.q, b.q[:9]]).to(DEV)
    out = torch.full(q.shape, 5.0, dtype=DT[dtype], device=DEV)
    sdv.attend(q, b.kc.to(DEV), b.vc.to(DEV), table, length, cu, out=out)
    assert (out[b.rows:] == 5.0).all()
    assert (out[:b.rows].float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()


@pytest.mark.parametrize("ks,lens,dtype", [([3, 0, 7], [20, 90, 5], "bf16"), ([3, 0, 7], [20, 90, 5], "fp32"),
                                           ([3, 0, 7], [20, 1900, 5], "bf16"), ([400, 230, 170], [20, 90, 5], "bf16")])
def test_caches_of_more_than_32_bit_offsets(ks, lens, dtype):
    b = Batch(ks, lens, 8, 128, 16, dtype, 41, Hq=32)
    table, length, cu = b.index_args()
    q = b.q.to(DEV)
    want = sdv.attend(q, b.kc.to(DEV), b.vc.to(DEV), table, length, cu)
    page = 8 * 16 * 128 * (2 if dtype == "bf16" else 4)
    first = (2 ** 32 + 2 ** 31) // page  # pages from 6 GiB on
    caches = []
    for c in (b.kc, b.vc):
        big = torch.empty((first + b.n_pages,) + c.shape[1:], dtype=c.dtype, device=DEV)
        big[first:] = c.to(DEV)
        caches.append(big)
    far = torch.where(table >= 0, table + first, table)
    assert torch.equal(sdv.attend(q, *caches, far, length, cu), want)
    k, v = b.k.to(DEV), b.v.to(DEV)
    near = [b.kc.to(DEV), b.vc.to(DEV)]
    sdv.kv_append(k, v, *near, table, length, cu)
    sdv.kv_append(k, v, *caches, far, length, cu)
    assert torch.equal(caches[0][first:], near[0]) and torch.equal(caches[1][first:], near[1])
