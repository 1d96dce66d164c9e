"""Settling a verified tree's path in caches of 8 bits, on the GPU against the oracle: codes and scales are the oracle's."""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache8_helpers import DEV, Batch8, host
from oracle import cache8 as oracle
from test_gpu_append8 import same
from test_gpu_kv_cache import accepted

pytestmark = pytest.mark.gpu


def run(b, acc, nodes):
    table, length, cu = b.index_args()
    kc, vc, ks, vs = b.caches()
    new = sdv.kv_settle(kc, vc, table, length, cu, torch.from_numpy(acc).to(DEV), torch.from_numpy(nodes).to(DEV),
                        key_scales=ks, value_scales=vs)
    lift = (lambda x: x[None]) if b.kc.ndim == 4 else (lambda x: x)
    rk, rv, rks, rvs, rn = oracle.settle8(*(lift(x) for x in (b.kc, b.vc, b.ks8, b.vs8)), b.block, b.table, b.len, b.cu, acc,
                                          nodes)
    assert np.array_equal(new.cpu().numpy(), rn)
    assert np.array_equal(lift(host(ks)), rks) and np.array_equal(lift(host(vs)), rvs)
    assert same(lift(host(kc)), rk) and same(lift(host(vc)), rv)
    return kc, vc, ks, vs


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page,block,layers", [(1, 1, 0), (16, 16, 3), (16, 2, 0), (64, 64, 1), (128, 8, 1)])
def test_settle(page, block, layers, D):
    rng = np.random.default_rng(page + D)
    b = Batch8([0, 64, 12, 30, 1, 64], [5, 100, 0, 31, 7, 15], 2, D, page, block, "bf16", page, tree=True, layers=layers)
    for c in (b.ks8, b.vs8):
        c[:] = rng.integers(100, 130, c.shape)
    run(b, *accepted(rng, b))


def test_all_codes_and_scales():
    rng = np.random.default_rng(1)
    for low, high in ((10, 14), (100, 112), (0, 256)):
        b = Batch8([20, 30, 9, 40], [5, 33, 0, 31], 3, 64, 32, 16, "bf16", 3, tree=True)
        for c in (b.kc, b.vc):
            c[:] = rng.integers(0, 256, c.shape)
        for c in (b.ks8, b.vs8):
            c[:] = rng.integers(low, high, c.shape)
        run(b, *accepted(rng, b))


@pytest.mark.parametrize("block", [1, 4, 16])
def test_whole_chains_and_far_jumps(block):
    b = Batch8([64, 64, 64], [3, 0, 16], 1, 128, 16, block, "bf16", 11, tree=True)
    nodes = np.full(192, -1, dtype=np.int32)
    nodes[:64] = np.arange(64)  # nothing moves
    nodes[64:96] = np.arange(32, 64)  # every source is a later place
    nodes[128:160] = np.arange(1, 64, 2)
    run(b, np.array([64, 32, 32], dtype=np.int32), nodes)


def test_what_is_not_valid_is_passed_over():
    b = Batch8([5, 5, 5, 5, 5, 5], [9, 9, 9, 9, 9, 9], 2, 64, 16, 4, "bf16", 12, tree=True)
    acc = np.array([-1, 6, 3, 2, 2, 2], dtype=np.int32)
    nodes = np.array([0, 1, 2, 3, 4] * 2 + [1, 1, 2, -1, -1] + [2, 7, -1, -1, -1] + [-1, 3, -1, -1, -1] + [3, 4, -1, -1, -1],
                     dtype=np.int32)
    b.len[5] = -2
    run(b, acc, nodes)
    b.len[5] = 9
    b.table[5, 0] = -1
    run(b, acc, nodes)
    for bad in ([0, 5, 10, 15, 20, 25, 31], [0, 5, 4, 15, 20, 25, 30], [-1, 5, 10, 15, 20, 25, 30]):
        b.cu = np.array(bad, dtype=np.int32)
        run(b, acc, nodes)


def test_missing_pages():
    """A slot to come from without a page, and one to go to."""
    b = Batch8([12, 12, 12], [2, 2, 2], 2, 64, 4, 4, "bf16", 14, tree=True)
    b.ks8[:] = np.random.default_rng(2).integers(100, 120, b.ks8.shape)
    nodes = np.array([1, 3, 5, 8, 10, 11] + [-1] * 6, dtype=np.int32)
    b.table[0, 2] = -1  # slots 8 .. 11
    b.table[1, 0] = b.n_pages
    b.table[2, 1:3] = -1
    run(b, np.array([6, 6, 6], dtype=np.int32), np.tile(nodes, 3))


def test_refusals():
    b = Batch8([2, 0], [5, 7], 2, 64, 16, 8, "bf16", 13, tree=True)
    table, length, cu = b.index_args()
    kc, vc, ks, vs = b.caches()
    acc, nodes = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    assert sdv.kv_settle(kc, vc, table, length, cu, acc, nodes, key_scales=ks, value_scales=vs).tolist() == [6, 8]
    for kw in (dict(key_scales=ks), dict(key_scales=ks[None], value_scales=vs[None]), dict(key_scales=ks, value_scales=vs.float())):
        with pytest.raises(ValueError):
            sdv.kv_settle(kc, vc, table, length, cu, acc, nodes, **kw)
    with pytest.raises(TypeError):
        sdv.kv_settle(kc, vc, table, length, cu, acc, nodes)
