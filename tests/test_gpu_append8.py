"""Appending to the paged cache in 8 bits, on the GPU against the oracle.

Scales come from the rows as given, and a code is that of the value in binary64: the kernel goes on in binary64 where binary32 does
not tell on which side of a border it lies (its angles are off by 2^-53 of a position, 1e-9 at the farthest here, so that no value of a
test lies within its error of a border but by a chance of 1e-3 in all), so both are the oracle's.  Queries: off by 2^-20 (|a| + |b|)
(the bound of test_gpu_kv_cache), and one rounding to their type (bf16 2^-8, binary32 2^-24).
"""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache8_helpers import DEV, SCALES, Batch8, host
from cache_helpers import DT, np64
from oracle import cache8 as oracle
from test_gpu_kv_cache import freq, near

pytestmark = pytest.mark.gpu


def same(got, want):
    """Bytes of codes that stand for the same numbers."""
    return np.array_equal(oracle.DECODED[got], oracle.DECODED[want], equal_nan=True)


def compare(b, caches, q_out, rotary, interleaved):
    f = freq(rotary).double().numpy()
    rk, rv, rks, rvs, rq, exact = oracle.append8(np64(b.k), np64(b.v), b.kc, b.vc, b.ks8, b.vs8, b.block, b.table, b.len,
                                                 b.cu, f, interleaved, b.parents, None if b.q is None else np64(b.q))
    gk, gv, gks, gvs = (host(t) for t in caches)
    assert np.array_equal(gks, rks) and np.array_equal(gvs, rvs)
    assert same(gv, rv)
    assert same(gk, rk), (np.argwhere(gk != rk)[:4], gk[gk != rk][:4], rk[gk != rk][:4], exact[gk != rk][:4])
    if q_out is not None:
        seen = np.isfinite(rq)
        big = 2 * max(float(b.q[torch.isfinite(b.q)].abs().max()), 1.0)
        near(np64(q_out)[seen], rq[seen], big, b.dtype)


def run(b, rotary=64, interleaved=False, fused=True):
    Hkv = b.k.shape[1]
    q, k, v = (x.to(DEV) for x in (b.q, b.k, b.v))
    if fused:  # slices of one projection's output
        qkv = torch.cat([q, k, v], 1)
        q, k, v = qkv[:, :b.q.shape[1]], qkv[:, b.q.shape[1]:-Hkv], qkv[:, -Hkv:]
    caches = b.caches()
    q_out = b.append(caches, freq(rotary).to(DEV) if rotary else None, k=k, v=v, interleaved=interleaved, queries=q)
    compare(b, caches, q_out, rotary, interleaved)
    return caches, q_out


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rotary", [(64, 64), (128, 128), (128, 64), (256, 16), (64, 0), (256, 256)])
def test_append(D, rotary, interleaved, dtype):
    run(Batch8([0, 3, 8, 1, 0], [0, 17, 100, 31, 1], 2, D, 16, 16, dtype, D + rotary, Hq=6), rotary, interleaved)


@pytest.mark.parametrize("page,block", [(1, 1), (2, 1), (2, 2), (16, 1), (16, 4), (64, 32), (64, 64), (128, 64), (1024, 64)])
@pytest.mark.parametrize("tree", [False, True])
def test_pages_blocks_and_trees(page, block, tree):
    run(Batch8([0, 64, 9, 20], [3, 150, 0, 129], 3, 64, page, block, "bf16", page + block, tree=tree, Hq=3), fused=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_blocks_that_were_begun(dtype):
    """Larger rows raise the block's scale and bring the held codes to it; smaller rows leave both."""
    for size in (2.0 ** 6, 1.0, 2.0 ** -9, 0.0):
        b = Batch8([2, 0, 5, 30], [7, 16, 31, 45], 2, 64, 32, 16, dtype, 5, Hq=2)
        b.k, b.v = b.k * size, b.v * size
        run(b)
    b = Batch8([2, 3], [7, 9], 1, 64, 16, 16, dtype, 6, Hq=1)
    b.kc[:] = np.random.default_rng(0).integers(0, 256, b.kc.shape)  # every code, NaN among them
    b.ks8[:], b.vs8[:] = 10, 90
    run(b, 0)


def test_scales_that_were_never_written():
    """Bytes outside [10, 246] in a begun block are read as the nearest inside; a fresh block's are not read."""
    for byte in (0, 5, 250, 255):
        b = Batch8([2, 3, 1], [7, 16, 3], 1, 64, 16, 16, "bf16", 7, Hq=1)
        b.ks8[:], b.vs8[:] = byte, byte
        run(b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_smallest_and_largest_rows(dtype):
    for size in (1e-38, 2.0 ** -126, 1e-36, 1e30, 2.0 ** 120, 8e37):
        b = Batch8([2, 0, 5], [7, 16, 31], 2, 64, 16, 8, dtype, 8, Hq=2)
        b.k, b.v = (b.k.clamp(-3, 3) * size).to(DT[dtype]), (b.v.clamp(-3, 3) * size).to(DT[dtype])
        run(b, 0)
    b = Batch8([2, 0], [7, 16], 1, 64, 16, 8, dtype, 8, Hq=1)
    b.k[:], b.v[:] = torch.finfo(DT[dtype]).max, -torch.finfo(DT[dtype]).max
    run(b, 0)


def test_limits_of_a_scale():
    """Rows whose largest value is 316 or 448 times a power of two take that one, the next number above the next one."""
    b = Batch8([0] * 6, [0] * 6, 1, 64, 16, 16, "fp32", 9, Hq=1)
    top = torch.tensor([316.0, 448.0, 316.0 * 2 ** -30, 448.0 * 2 ** 40, 1.0, 0.0])
    up = torch.nextafter(top, torch.tensor(float("inf")))
    for t in (top, up):
        b.k = b.k.clamp(-0.5, 0.5) * t[:, None, None]
        b.v = b.k.clone()
        b.k[:, 0, 5] = t
        b.v[:, 0, 60] = -t
        run(b, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rotary", [0, 64])
def test_rows_that_are_not_finite(dtype, rotary):
    b = Batch8([2, 0, 5], [7, 16, 31], 2, 64, 16, 8, dtype, 10, Hq=2)
    inf, nan = float("inf"), float("nan")
    for x in (b.k, b.v):
        x[0, 0, 3], x[1, 0, 40], x[3, 1, 0], x[5, 1, 63] = inf, -inf, nan, nan
    b.k[6] = nan  # a row of nothing else
    b.v[6] = inf
    run(b, rotary)


def test_prompts_and_many_requests():
    run(Batch8([700, 0, 333], [5, 0, 400], 1, 64, 32, 32, "bf16", 1, Hq=5), 32, True)
    run(Batch8([130], [61], 2, 256, 64, 64, "fp32", 1, Hq=1), 256)
    rng = np.random.default_rng(2)
    run(Batch8(rng.integers(0, 4, 300), rng.integers(0, 90, 300), 1, 64, 16, 4, "fp32", 3, Hq=1))


def test_far_positions_keep_their_angle():
    b = Batch8([2], [100], 1, 64, 16, 16, "fp32", 4, Hq=1)
    L = 3_000_000
    b.table = np.concatenate([np.full((1, L // 16), -1, dtype=np.int32), b.table], 1)
    b.lens, b.len = [L + 100], np.array([L + 100], dtype=np.int32)
    run(b)


def test_what_has_no_place_is_left():
    """Freed pages, slots beyond the table, requests passed over: nothing is written for them."""
    b = Batch8([3, 2, 5, 4], [30, 7, 15, 11], 2, 64, 16, 8, "bf16", 5, Hq=2)
    b.table[0, 1] = -1
    b.table[0, 2] = b.n_pages
    b.table[2, 1] = 2 ** 31 - 1
    b.len[1] = -1
    b.len[3] = 16 * b.table.shape[1] - 2  # the table ends inside the request
    run(b)
    b = Batch8([3, 2, 5], [30, 7, 15], 2, 64, 16, 8, "bf16", 6, Hq=2, tree=True)
    b.parents[4] = 1  # request 1: a parent that does not precede its node
    b.parents[3] = 0
    run(b, 64, True)
    run(Batch8([70, 2], [30, 7], 1, 64, 16, 8, "bf16", 7, Hq=1, tree=True))  # more nodes than a tree may hold


SMALL = [[0, 3, 2, 10], [0, -5, 5, 10], [0, 3, 50, 10], [4, 3, 2, 1], [-1, -1, -1, -1], [0, 3, -5, 10], [0, 3, 5, -1],
         [0, 3, -2 ** 31, 10], [-7, 3, 5, 10], [0, 2 ** 31 - 1, 5, 10], [2 ** 31 - 1, 3, 5, 10]]


@pytest.mark.parametrize("bad", SMALL)
@pytest.mark.parametrize("block", [1, 16])
def test_offsets_that_are_not_valid(bad, block):
    b = Batch8([3, 2, 5], [30, 7, 15], 1, 64, 16, block, "bf16", 8, Hq=1)
    b.table = np.concatenate([b.table, np.full((3, 1), -1, dtype=np.int32)], 1)
    b.cu = np.array(bad, dtype=np.int32)
    caches = b.caches()
    q_out = torch.full(b.q.shape, 5.0, dtype=torch.bfloat16, device=DEV)
    b.append(caches, freq(64).to(DEV), queries=b.q.to(DEV), queries_out=q_out)
    compare(b, caches, q_out, 64, False)
    named = np.zeros(b.rows, dtype=bool)
    for _, row0, K, *_ in oracle.requests(b.cu, b.len, b.n_d):
        named[row0:row0 + K + 1] = True
    assert (q_out[torch.from_numpy(~named)] == 5.0).all()


@pytest.mark.parametrize("bad", [-5, -2 ** 31, 2 ** 30, 10 ** 6])
@pytest.mark.parametrize("B", [40, 100, 300])
def test_one_offset_of_many(B, bad):
    rng = np.random.default_rng(B)
    ks = rng.integers(0, 6, B)
    for at in (0, 7, B // 2 + 1, B):
        b = Batch8(ks, rng.integers(0, 60, B), 1, 64, 16, 8, "bf16", B + at, Hq=2)
        b.cu[at] = bad
        run(b)


def test_rows_behind_the_last_request_stay():
    b = Batch8([3, 0, 7], [20, 90, 5], 2, 64, 16, 16, "bf16", 40, Hq=4)
    table, length, cu = b.index_args()
    wide = lambda x: torch.cat([x, x[:9]]).to(DEV)  # noqa: E731
    caches, want = run(b)
    again = b.caches()
    q_out = torch.full((b.rows + 9, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    b.append(again, freq(64).to(DEV), k=wide(b.k), v=wide(b.v), queries=wide(b.q), queries_out=q_out)
    assert torch.equal(q_out[:b.rows], want) and (q_out[b.rows:] == 5.0).all()
    for x, y in zip(again, caches):
        assert np.array_equal(host(x), host(y))


def test_without_queries_and_in_place():
    for D, dtype in ((128, "bf16"), (64, "fp32"), (256, "bf16")):
        b = Batch8([30, 0], [30, 7], 2, D, 16, 16, dtype, 9, Hq=4)
        caches, want = run(b, D)
        f = freq(D).to(DEV)
        again = b.caches()
        assert b.append(again, f) is None
        q = b.q.to(DEV)
        assert b.append(b.caches(), f, queries=q, queries_out=q) is q
        assert torch.equal(q, want)
        for x, y in zip(again, caches):
            assert np.array_equal(host(x), host(y))


def test_appended_again_it_is_the_same():
    b = Batch8([3, 0, 7, 20], [20, 90, 5, 47], 2, 64, 32, 16, "bf16", 41, Hq=4)
    b.k, b.v = b.k * 50, b.v * 50
    caches, _ = run(b)
    first = [host(t).copy() for t in caches]
    b.append(caches, freq(64).to(DEV))
    for x, y in zip(caches, first):
        assert np.array_equal(host(x), y)


def test_scales_as_bytes_and_as_numbers():
    b = Batch8([3, 0, 7], [20, 90, 5], 2, 64, 16, 8, "bf16", 42, Hq=4)
    caches, want = run(b)
    kc, vc, ks, vs = b.caches()
    b.append((kc, vc, ks.view(torch.uint8), vs.view(torch.uint8)), freq(64).to(DEV))
    assert np.array_equal(host(ks), host(caches[2]))
    # what a scale of torch's type says is what the codes stand for
    assert np.array_equal(ks.view(SCALES).double().cpu().numpy()[0], oracle.scales(host(ks))[0])


def test_caches_beyond_32_bit_offsets():
    b = Batch8([4, 40], [14, 3], 2, 128, 16, 16, "bf16", 10, Hq=4)
    near_, _ = run(b)
    first = (2 ** 32 + 2 ** 31) // (2 * 16 * 128)
    big = []
    for t in b.caches():
        x = torch.zeros((first + b.n_pages,) + t.shape[1:], dtype=torch.uint8, device=DEV)
        x[first:] = t.view(torch.uint8)
        big.append(x.view(t.dtype))
    b.table = np.where(b.table >= 0, b.table + first, b.table).astype(np.int32)
    b.append(big, freq(64).to(DEV))
    for x, y in zip(big, near_):
        assert np.array_equal(host(x[first:]), host(y))
        assert not x[:first].view(torch.uint8).any()


def test_graph_replays():
    b = Batch8([4, 0, 20], [30, 50, 7], 2, 128, 16, 16, "bf16", 18, Hq=4)
    table, length, cu = b.index_args()
    k, v, q, f = b.k.to(DEV), b.v.to(DEV), b.q.to(DEV), freq(128).to(DEV)
    start = b.caches()

    def call(c):
        return sdv.kv_append(k, v, c[0], c[1], table, length, cu, key_scales=c[2], value_scales=c[3], inv_freq=f, queries=q)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mine = [t.clone() for t in start]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = call(mine)
    torch.cuda.synchronize()
    for step in range(4):
        k.copy_(torch.randn(k.shape, generator=torch.Generator().manual_seed(step)) * 2.0 ** step)
        length.copy_(torch.tensor([30 - step, 50 + step, 7], dtype=torch.int32))
        want = [t.clone() for t in start]
        want_q = call(want)
        for x, y in zip(mine, start):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_q)
        for x, y in zip(mine, want):
            assert np.array_equal(host(x), host(y))


def test_refusals():
    b = Batch8([2, 0], [5, 7], 2, 64, 16, 8, "bf16", 13, Hq=4)
    table, length, cu = b.index_args()
    k, v, q = (x.to(DEV) for x in (b.k, b.v, b.q))
    kc, vc, ks, vs = b.caches()

    def ok(**kw):
        a = dict(k=k, v=v, kc=kc, vc=vc, ks=ks, vs=vs, q=q)
        a.update(kw)
        return sdv.kv_append(a["k"], a["v"], a["kc"], a["vc"], table, length, cu, key_scales=a["ks"], value_scales=a["vs"],
                             queries=a["q"])

    ok()
    for kw in (dict(ks=None), dict(vs=None), dict(ks=ks[:1]), dict(vs=vs[:, :, :1]), dict(ks=ks.float()), dict(ks=ks.cpu()),
               dict(ks=ks.transpose(0, 1)), dict(ks=torch.zeros((b.n_pages, 2, 3), dtype=torch.uint8, device=DEV)),
               dict(v=v.float()), dict(q=q.float()), dict(vc=vc.view(torch.uint8)), dict(k=k[:1]), dict(kc=kc[:, :1])):
        with pytest.raises(ValueError):
            ok(**kw)
    for kw in (dict(kc=kc.to(torch.bfloat16), vc=vc.to(torch.bfloat16)), dict(k=k.half(), v=v.half(), q=q.half()),
               dict(kc=kc.view(torch.uint8), vc=vc.view(torch.uint8)), dict(ks=None, vs=None)):
        with pytest.raises(TypeError):
            ok(**kw)
    wide = torch.zeros((b.n_pages, 2, 16, 64), dtype=torch.uint8, device=DEV).view(kc.dtype)
    many = torch.zeros((b.n_pages, 2, 1), dtype=torch.uint8, device=DEV)
    ok(kc=wide, vc=wide.clone(), ks=many, vs=many.clone())
    big = torch.zeros((3, 2, 128, 64), dtype=torch.uint8, device=DEV).view(kc.dtype)
    one = torch.zeros((3, 2, 1), dtype=torch.uint8, device=DEV)
    with pytest.raises(sdv.SdvError):
        ok(kc=big, vc=big.clone(), ks=one, vs=one.clone())  # a block of 128 tokens
