"""New lengths of sdv_kv_settle next to the arrays it reads."""
import ctypes

import numpy as np
import pytest
import torch

from cache_helpers import DEV, Batch, np64
from lossless_draft_verification_online_amd import _native
from oracle import cache as oracle
from test_gpu_kv_cache import accepted

pytestmark = pytest.mark.gpu


def test_neighbouring_arrays_and_the_same_one():
    b = Batch([5, 64, 0, 12], [9, 100, 3, 31], 2, 64, 16, "bf16", 3, tree=True)
    acc, nodes = accepted(np.random.default_rng(3), b)
    table, length, cu = b.index_args()
    kc, vc = b.kc.to(DEV), b.vc.to(DEV)
    room = torch.full((14,), -7, dtype=torch.int32, device=DEV)  # cache_len | new_len | accepted_len, without gaps
    room[1:5], room[9:13] = length, torch.from_numpy(acc).to(DEV)
    at = room.data_ptr()
    n = torch.from_numpy(nodes).to(DEV)
    c = _native.SdvCache(kc.data_ptr(), vc.data_ptr(), table.data_ptr(), at + 4, b.n_pages, table.shape[1], 16, 2, 64, 0)

    def settle(new):
        return _native.lib().sdv_kv_settle(ctypes.byref(c), 1, b.B, b.n_d, cu.data_ptr(), at + 36, n.data_ptr(), new,
                                           torch.cuda.current_stream().cuda_stream)

    for new in (at + 4, at + 8, at + 32, at + 36):
        assert settle(new) == -1
    torch.cuda.synchronize()
    assert torch.equal(kc.cpu(), b.kc) and torch.equal(vc.cpu(), b.vc)
    assert settle(at + 20) == 0
    rk, rv, rn = oracle.settle(np64(b.kc)[None], np64(b.vc)[None], b.table, b.len, b.cu, acc, nodes)
    assert np.array_equal(np64(kc), rk[0]) and np.array_equal(np64(vc), rv[0])
    assert room.tolist() == [-7, *b.lens, *rn.tolist(), *acc.tolist(), -7]
