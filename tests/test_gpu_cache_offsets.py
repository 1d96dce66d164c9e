"""Offsets that are not valid, beside requests whose offsets are: the valid ones are served, and rows that none of them names
stay as they were.  A request is valid if 0 <= cu[i] <= cu[i + 1] <= n_draft_rows; tolerances as in test_gpu_attend and
test_gpu_kv_cache.
"""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache_helpers import DEV, DT, Batch, np64
from oracle import cache as oracle
from test_gpu_kv_cache import freq, near

pytestmark = pytest.mark.gpu
FILL = 5.0


def valid_rows(b):
    rows = np.zeros(b.rows, dtype=int)
    for _, row0, K, *_ in oracle.requests(b.cu, b.len, b.n_d, b.parents):
        rows[row0:row0 + K + 1] += 1
    assert rows.max(initial=0) <= 1  # no row of two requests
    return rows > 0


def run_append(b, dtype):
    table, length, cu = b.index_args()
    kc, vc = b.kc.to(DEV), b.vc.to(DEV)
    q_out = torch.full(b.q.shape, FILL, dtype=DT[dtype], device=DEV)
    sdv.kv_append(b.k.to(DEV), b.v.to(DEV), kc, vc, table, length, cu, parents=b.tree_arg(), inv_freq=freq(64).to(DEV),
                  queries=b.q.to(DEV), queries_out=q_out)
    rk, rv, rq = oracle.append(np64(b.k), np64(b.v), np64(b.kc), np64(b.vc), b.table, b.len, b.cu, freq(64).double().numpy(),
                               False, b.parents, np64(b.q))
    big = 2 * max(float(b.k.abs().max()), float(b.q.abs().max()))
    touched = rk != np64(b.kc)
    near(np64(kc)[touched], rk[touched], big, dtype)
    assert np.array_equal(np64(kc)[~touched], rk[~touched]) and np.array_equal(np64(vc), rv)
    mine = valid_rows(b)
    near(np64(q_out)[mine], rq[mine], big, dtype)
    assert (q_out[torch.from_numpy(~mine)] == FILL).all()


def run_attend(b, dtype, window=0, sinks=0):
    table, length, cu = b.index_args()
    out = torch.full(b.q.shape, FILL, dtype=DT[dtype], device=DEV)
    sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, cu, parents=b.tree_arg(), window=window, sinks=sinks,
               out=out)
    D = b.kc.shape[-1]
    ref, mag, span = oracle.attend(np64(b.q), np64(b.kc), np64(b.vc), b.table, b.len, b.cu, D ** -0.5, window, sinks,
                                   b.parents)
    n = int(b.len.max()) + int(max(b.ks)) + 1
    rel = (D + 2) * 2.0 ** -24 * span[..., None] + 2.0 ** -22 * (n / 32 + 4) + n * 2.0 ** -24
    tol = mag * rel + np.abs(ref) * 2.0 ** -24 + 1e-30
    if dtype == "bf16":
        tol += 2.0 ** -8 * mag + 2.0 ** -8 * np.abs(ref)
    mine = valid_rows(b)
    bad = ~(np.abs(np64(out) - ref) <= tol) & mine[:, None, None]
    assert not bad.any(), np.argwhere(bad)[:4]
    assert (out[torch.from_numpy(~mine)] == FILL).all()


def spoiled(b, places):
    b.cu = b.cu.copy()
    for at, value in places.items():
        b.cu[at] = value
    return b


SMALL = [[0, 3, 2, 10], [0, -5, 5, 10], [0, 3, 50, 10], [4, 3, 2, 1], [-1, -1, -1, -1], [0, 3, -5, 10], [0, 3, 5, -1],
         [0, 3, -2 ** 31, 10], [-7, 3, 5, 10], [0, 2 ** 31 - 1, 5, 10], [2 ** 31 - 1, 3, 5, 10]]


@pytest.mark.parametrize("bad", SMALL)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_few(bad, dtype):
    b = Batch([3, 2, 5], [30, 7, 15], 1, 64, 16, dtype, 8, Hq=1)
    b.table = np.concatenate([b.table, np.full((3, 1), -1, dtype=np.int32)], 1)
    b.cu = np.array(bad, dtype=np.int32)
    run_append(b, dtype)


@pytest.mark.parametrize("bad", SMALL)
@pytest.mark.parametrize("dtype,Hq,page", [("bf16", 2, 16), ("fp32", 16, 16), ("bf16", 16, 4)])
def test_attend_few(bad, dtype, Hq, page):
    b = Batch([3, 2, 5], [30, 7, 15], 1, 64, page, dtype, 16, Hq=Hq)
    b.cu = np.array(bad, dtype=np.int32)
    run_attend(b, dtype)


@pytest.mark.parametrize("bad", [-5, -2 ** 31, 2 ** 30, 10 ** 6])
@pytest.mark.parametrize("B", [40, 100, 300])
def test_one_offset_of_many(B, bad):
    """The requests before and behind are served, wherever the search for a row's request meets the spoiled offset."""
    rng = np.random.default_rng(B)
    ks = rng.integers(0, 6, B)
    for at in (0, 7, B // 2 + 1, B):
        def batch(dtype, **kw):
            return spoiled(Batch(ks, rng.integers(0, 60, B), 1, 64, 16, dtype, B + at, **kw), {at: bad})

        run_append(batch("bf16", Hq=2), "bf16")
        run_attend(batch("bf16", Hq=4), "bf16", 40, 2)
        run_attend(batch("fp32", Hq=8), "fp32")
        run_attend(batch("bf16", Hq=4, tree=True), "bf16")


def test_several_offsets_of_many():
    rng = np.random.default_rng(5)
    for B in (64, 65, 200):
        ks = rng.integers(0, 5, B)
        for step in range(6):
            bad = {int(at): int(rng.choice([-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])) for at in rng.integers(0, B + 1, 5)}
            run_append(spoiled(Batch(ks, rng.integers(0, 60, B), 1, 64, 16, "fp32", step, Hq=1), bad), "fp32")
            run_attend(spoiled(Batch(ks, rng.integers(0, 60, B), 2, 64, 16, "bf16", step, Hq=8), bad), "bf16")


@pytest.mark.parametrize("at,bad", [(1, -5), (1, 10 ** 6), (2, -5), (2, 2 ** 31 - 1), (3, -1), (0, -5)])
def test_prompts_beside_an_offset(at, bad):
    """Many columns per request: the prompts' kernel."""
    run_attend(spoiled(Batch([27, 31, 33], [20, 57, 84], 48, 64, 16, "bf16", at, Hq=192), {at: bad}), "bf16")
    ks = [(5 * i) % 40 + 8 for i in range(150)]
    run_attend(spoiled(Batch(ks, [(7 * i) % 90 for i in range(150)], 1, 64, 16, "bf16", 22, Hq=16), {at * 49: bad}), "bf16", 48, 2)
