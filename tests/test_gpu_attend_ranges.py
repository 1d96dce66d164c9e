"""Batches of more than 64 requests over long caches: their work is cut into ranges of equal length, and a lane holds the
lengths of several requests.  Against the binary64 oracle, with test_gpu_attend's tolerance."""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache_helpers import DEV, Batch
from test_gpu_attend import check

pytestmark = pytest.mark.gpu


def lengths(B, long, seed):
    """Mostly short and empty, some long; long ones next to each other too, and first and last."""
    rng = np.random.default_rng(seed)
    lens = rng.choice([0, 0, 1, 30, 31, 32, 200], B)
    lens[rng.choice(B, 6, replace=False)] = long
    lens[[0, B // 2, B // 2 + 1, B - 1]] = [long - 7, long, long - 1, long - 31]
    return lens


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B", [65, 130, 512])
def test_linear(B, dtype):
    rng = np.random.default_rng(B)
    check(Batch(rng.integers(0, 3, B), lengths(B, 2600, B), 1, 64, 16, dtype, B, Hq=4), dtype)


@pytest.mark.parametrize("B", [65, 300])
def test_window_pairs_of_column_tiles_and_wide_heads(B):
    rng = np.random.default_rng(B)
    check(Batch(rng.integers(0, 8, B), lengths(B, 2900, B), 1, 128, 32, "bf16", B, Hq=6), "bf16", 2300, 4)
    check(Batch([0] * B, lengths(B, 2600, B + 1), 2, 256, 16, "bf16", B, Hq=2), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_trees(dtype):
    rng = np.random.default_rng(9)
    ks = rng.integers(0, 20, 80)
    ks[33] = 6
    b = Batch(ks, lengths(80, 2500, 9), 1, 64, 16, dtype, 9, tree=True, Hq=4)
    b.parents[b.cu[33] + 2] = 2  # a parent that does not precede its node
    out = check(b, dtype)
    lo = int(b.cu[33]) + 33
    assert not out[lo:lo + 7].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_requests_that_are_passed_over(dtype):
    """Lengths and offsets that are not valid, inside a lane's group and at its ends, and pages that are missing."""
    B = 150
    rng = np.random.default_rng(10)
    b = Batch(rng.integers(0, 3, B), lengths(B, 2600, 10), 1, 64, 16, dtype, 10, Hq=4)
    over = (3, 4, 5, 30, 76, 149)
    b.len[list(over)] = [-1, -7, -2 ** 31, -9, -1, -1]
    b.table[75, 3:9] = -1
    out = check(b, dtype)
    for i in over:
        lo = int(b.cu[i]) + i
        assert not out[lo:lo + b.ks[i] + 1].any()
    b.len[list(over)] = [2 ** 31 - 1, 2 ** 31 - 1024 - b.ks[4], -1, 2 ** 31 - 2, 2 ** 31 - 1025, 2 ** 31 - 1024]
    table, length, cu = b.index_args()
    again = sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), table, length, cu)
    assert torch.equal(again, out)


@pytest.mark.parametrize("B", [65, 130, 512])
def test_no_request_is_valid(B):
    b = Batch([1] * B, [2600] + [3] * (B - 1), 1, 64, 16, "bf16", 11, Hq=4)
    table, length, cu = b.index_args()
    q, kc, vc = b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV)
    assert not sdv.attend(q, kc, vc, table, torch.full_like(length, -1), cu).any()
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=DEV)
    sdv.attend(q, kc, vc, table, length, torch.full_like(cu, -1), out=out)
    assert (out == 5.0).all()


def test_the_same_call_gives_the_same_bits_and_rows_behind_stay():
    rng = np.random.default_rng(12)
    b = Batch(rng.integers(0, 3, 130), lengths(130, 2600, 12), 1, 64, 16, "bf16", 12, Hq=4)
    table, length, cu = b.index_args()
    args = b.kc.to(DEV), b.vc.to(DEV), table, length, cu
    want = sdv.attend(b.q.to(DEV), *args)
    q = torch.cat([b.q, b.q[:9]]).to(DEV)
    for _ in range(3):
        assert torch.equal(sdv.attend(b.q.to(DEV), *args), want)
        out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=DEV)
        sdv.attend(q, *args, out=out)
        assert (out[b.rows:] == 5.0).all()
        assert (out[:b.rows].float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
