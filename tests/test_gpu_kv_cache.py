"""Appending to the paged cache and settling a verified tree's path, on the GPU against the oracle.

Tolerances of a rotated value a c - b s: the angle in turns is rounded to binary32 after its reduction
(2^-25 turns, so 2 pi 2^-25 < 2^-22 in angle), sincospi is within 2 steps of 2^-24, and the two
products and the sum add three roundings: under 2^-20 (|a| + |b|).  Then one rounding to the cache's
type (bf16 2^-8, binary32 2^-24 of the value).  What is not rotated is copied, bit for bit.
"""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from oracle import cache as oracle
from cache_helpers import DEV, DT, Batch, np64

pytestmark = pytest.mark.gpu


def freq(rotary, base=10000.0):
    half = rotary // 2
    return torch.tensor(base ** (-np.arange(half) / max(half, 1)), dtype=torch.float32)


def near(got, ref, mag, dtype):
    tol = 2.0 ** -20 * mag + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(ref) + 1e-30
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])


def run_append(b, rotary, interleaved, dtype, fused=True):
    table, length, cu = b.index_args()
    f = freq(rotary)
    Hkv, D = b.k.shape[1:]
    if fused:  # slices of one projection's output
        qkv = torch.cat([b.q, b.k, b.v], 1).to(DEV)
        q, k, v = qkv[:, :b.q.shape[1]], qkv[:, b.q.shape[1]:-Hkv], qkv[:, -Hkv:]
    else:
        q, k, v = b.q.to(DEV), b.k.to(DEV), b.v.to(DEV)
    kc, vc = b.kc.to(DEV), b.vc.to(DEV)
    q_out = sdv.kv_append(k, v, kc, vc, table, length, cu, parents=b.tree_arg(), inv_freq=f.to(DEV) if rotary else None,
                          interleaved=interleaved, queries=q)
    rk, rv, rq = oracle.append(np64(b.k), np64(b.v), np64(b.kc), np64(b.vc), b.table, b.len, b.cu, f.double().numpy(),
                               interleaved, b.parents, np64(b.q))
    big = 2 * max(float(b.k.abs().max()), float(b.q.abs().max()), 1.0)
    touched = rk != np64(b.kc)
    got = np64(kc)
    near(got[touched], rk[touched], big, dtype)
    assert np.array_equal(got[~touched], rk[~touched])  # slots of no row are as they were
    assert np.array_equal(np64(vc), rv)
    seen = ~np.isnan(rq)
    near(np64(q_out)[seen], rq[seen], big, dtype)
    return kc, vc, q_out


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rotary", [(64, 64), (128, 128), (128, 64), (256, 16), (64, 0), (256, 256)])
def test_append(D, rotary, interleaved, dtype):
    run_append(Batch([0, 3, 8, 1, 0], [0, 17, 500, 31, 1], 2, D, 16, dtype, D + rotary, Hq=6), rotary, interleaved, dtype)


@pytest.mark.parametrize("page", [1, 2, 16, 128, 1024])
@pytest.mark.parametrize("tree", [False, True])
def test_append_pages_and_trees(page, tree):
    run_append(Batch([0, 64, 9, 20], [3, 1000, 0, 129], 3, 64, page, "bf16", page, tree=tree, Hq=3), 64, False, "bf16",
               fused=False)


def test_append_prompts_and_many_requests():
    run_append(Batch([700, 0, 333], [5, 0, 4000], 1, 64, 32, "bf16", 1, Hq=5), 32, True, "bf16")
    rng = np.random.default_rng(2)
    run_append(Batch(rng.integers(0, 4, 300), rng.integers(0, 90, 300), 1, 64, 16, "fp32", 3, Hq=1), 64, False, "fp32")


def test_far_positions_keep_their_angle():
    b = Batch([2], [100], 1, 64, 16, "fp32", 4, Hq=1)
    L = 3_000_000
    b.table = np.concatenate([np.full((1, L // 16), -1, dtype=np.int32), b.table], 1)
    b.lens, b.len = [L + 100], np.array([L + 100], dtype=np.int32)
    run_append(b, 64, False, "fp32")


def test_append_leaves_what_has_no_place():
    """Freed pages, slots beyond the table, requests passed over: nothing is written for them."""
    b = Batch([3, 2, 5, 4], [30, 7, 15, 11], 2, 64, 16, "bf16", 5, Hq=2)
    b.table[0, 1] = -1
    b.table[0, 2] = b.n_pages
    b.table[2, 1] = 2 ** 31 - 1
    b.len[1] = -1
    b.len[3] = 16 * b.table.shape[1] - 2  # the table ends inside the request
    run_append(b, 64, False, "bf16")
    b = Batch([3, 2, 5], [30, 7, 15], 2, 64, 16, "bf16", 6, Hq=2, tree=True)
    b.parents[4] = 1  # request 1: a parent that does not precede its node
    b.parents[3] = 0
    run_append(b, 64, True, "bf16")
    b = Batch([70, 2], [30, 7], 1, 64, 16, "bf16", 7, Hq=1, tree=True)  # more nodes than a tree may hold
    run_append(b, 64, False, "bf16")


def test_append_offsets_that_are_not_valid():
    b = Batch([3, 2, 5], [30, 7, 15], 1, 64, 16, "bf16", 8, Hq=1)
    table, length, cu = b.index_args()
    for bad in ([0, 3, 2, 10], [0, -5, 5, 10], [0, 3, 50, 10], [4, 3, 2, 1], [-1, -1, -1, -1]):
        kc, vc = b.kc.to(DEV), b.vc.to(DEV)
        sdv.kv_append(b.k.to(DEV), b.v.to(DEV), kc, vc, table, length, torch.tensor(bad, dtype=torch.int32, device=DEV),
                      queries=b.q.to(DEV))
        torch.cuda.synchronize()


def test_append_without_queries_and_in_place():
    b = Batch([3, 0], [30, 7], 2, 128, 16, "bf16", 9, Hq=4)
    kc, vc, want = run_append(b, 128, False, "bf16")
    table, length, cu = b.index_args()
    k2, v2, q = b.kc.to(DEV), b.vc.to(DEV), b.q.to(DEV)
    assert sdv.kv_append(b.k.to(DEV), b.v.to(DEV), k2, v2, table, length, cu, inv_freq=freq(128).to(DEV)) is None
    assert torch.equal(k2, kc) and torch.equal(v2, vc)
    assert sdv.kv_append(b.k.to(DEV), b.v.to(DEV), k2, v2, table, length, cu, inv_freq=freq(128).to(DEV), queries=q,
                         queries_out=q) is q
    assert torch.equal(q, want)


def test_a_cache_beyond_32_bit_offsets():
    """5 GiB per cache: the last pages lie behind 2^32 bytes and 2^31 values."""
    n_pages, page, Hkv, D = 5 * 2 ** 30 // (16 * 2 * 128 * 2), 16, 2, 128
    kc = torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    b = Batch([4], [14], Hkv, D, page, "bf16", 10, Hq=4)
    table = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32, device=DEV)
    _, length, cu = b.index_args()
    sdv.kv_append(b.k.to(DEV), b.v.to(DEV), kc, vc, table, length, cu)
    for j in range(5):
        pg, at = table[0, (14 + j) // 16], (14 + j) % 16
        assert torch.equal(kc[pg, :, at].cpu(), b.k[j]) and torch.equal(vc[pg, :, at].cpu(), b.v[j])
    small = [x[n_pages - 3:].clone() for x in (kc, vc)]
    q = b.q.to(DEV)
    want = sdv.attend(q, *small, table - (n_pages - 3), length, cu)
    assert torch.equal(sdv.attend(q, kc, vc, table, length, cu), want)


# ---------------------------------------------------------------------------------------- settle

def accepted(rng, b):
    acc, nodes = [], []
    for t in b.trees:
        path, here = [], -1
        while True:
            kids = [n for n, p in enumerate(t) if p == here]
            if not kids or rng.random() < 0.1:
                break
            here = int(rng.choice(kids))
            path.append(here)
        acc.append(len(path))
        nodes += path + [-1] * (len(t) - len(path))
    return np.array(acc, dtype=np.int32), np.array(nodes, dtype=np.int32)


def run_settle(b, acc, nodes):
    table, length, cu = b.index_args()
    kc, vc = b.kc.to(DEV), b.vc.to(DEV)
    new = sdv.kv_settle(kc, vc, table, length, cu, torch.from_numpy(acc).to(DEV), torch.from_numpy(nodes).to(DEV))
    one = b.kc.dim() == 4
    lift = lambda t: (t.float().numpy()[None] if one else t.float().numpy())  # noqa: E731
    rk, rv, rn = oracle.settle(lift(b.kc), lift(b.vc), b.table, b.len, b.cu, acc, nodes)
    assert np.array_equal(lift(kc.cpu()), rk) and np.array_equal(lift(vc.cpu()), rv)
    assert np.array_equal(new.cpu().numpy(), rn)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page,layers", [(1, 0), (16, 3), (64, 1)])
def test_settle(page, layers, D, dtype):
    rng = np.random.default_rng(page + D)
    b = Batch([0, 64, 12, 30, 1, 64], [5, 100, 0, 31, 7, 15], 2, D, page, dtype, page, tree=True, layers=layers)
    run_settle(b, *accepted(rng, b))


def test_settle_whole_chains_and_far_jumps():
    b = Batch([64, 64, 64], [3, 0, 16], 1, 128, 16, "bf16", 11, tree=True)
    nodes = np.full(192, -1, dtype=np.int32)
    nodes[:64] = np.arange(64)  # nothing moves
    nodes[64:96] = np.arange(32, 64)  # every source is a later place
    nodes[128:160] = np.arange(1, 64, 2)
    run_settle(b, np.array([64, 32, 32], dtype=np.int32), nodes)


def test_settle_passes_over_what_is_not_valid():
    b = Batch([5, 5, 5, 5, 5, 5], [9, 9, 9, 9, 9, 9], 2, 64, 16, "bf16", 12, tree=True)
    acc = np.array([-1, 6, 3, 2, 2, 2], dtype=np.int32)
    nodes = np.array([0, 1, 2, 3, 4] * 2 + [1, 1, 2, -1, -1] + [2, 7, -1, -1, -1] + [-1, 3, -1, -1, -1] + [3, 4, -1, -1, -1],
                     dtype=np.int32)
    b.len[5] = -2
    run_settle(b, acc, nodes)
    b.len[5] = 9
    b.table[5, 0] = -1
    run_settle(b, acc, nodes)


def test_refusals():
    b = Batch([2, 0], [5, 7], 2, 64, 16, "bf16", 13, Hq=4)
    table, length, cu = b.index_args()
    k, v, kc, vc, q = (x.to(DEV) for x in (b.k, b.v, b.kc, b.vc, b.q))
    f = freq(64).to(DEV)
    ok = lambda **kw: sdv.kv_append(kw.get("k", k), kw.get("v", v), kw.get("kc", kc), kw.get("vc", vc),  # noqa: E731
                                    kw.get("table", table), kw.get("len", length), kw.get("cu", cu),
                                    inv_freq=kw.get("f"), queries=kw.get("q"))
    ok(f=f, q=q)
    for kw in (dict(k=k.float()), dict(k=k[:, :1]), dict(v=v[:2]), dict(vc=vc[:1]), dict(table=table[:1]),
               dict(len=length.long()), dict(kc=kc.transpose(1, 2)), dict(q=q[:1]), dict(k=k.transpose(0, 1))):
        with pytest.raises(ValueError):
            ok(**kw)
    with pytest.raises(TypeError):
        ok(kc=kc.half())
    with pytest.raises(sdv.SdvError):
        ok(f=freq(24).to(DEV))  # a rotation of 24 values
    with pytest.raises(sdv.SdvError):
        ok(f=freq(128).to(DEV))  # more than a head
    wide = torch.zeros((4, 2 * 64 + 4), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sdv.SdvError):
        ok(k=wide[:, 4:].view(4, 2, 64))  # rows off the 16-byte grid
    odd = torch.zeros((4, 2, 12, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sdv.SdvError):
        ok(kc=odd, vc=odd)
    with pytest.raises(ValueError):
        sdv.kv_settle(kc, vc, table, length, cu, torch.zeros(2, dtype=torch.int64, device=DEV),
                      torch.zeros(2, dtype=torch.int32, device=DEV))
