"""The most rows that one launch takes."""
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from test_gpu_sample import DEV

pytestmark = pytest.mark.gpu


def test_sampling_of_many_short_rows():
    n = 2 ** 24 - 1
    z = torch.zeros((n + 1, 2), dtype=torch.bfloat16, device=DEV)
    z[:, 1] = -float("inf")
    z[n - 1] = torch.tensor([-float("inf"), 1.0])
    u = torch.full((n + 1,), 0.5, dtype=torch.float64, device=DEV)
    tok, prob, _ = sdv.sample(z[:n], u[:n], 1.0)
    assert tok[n - 1] == 1 and not tok[:n - 1].any() and (prob == 1).all()
    with pytest.raises(sdv.SdvError, match="LIMIT"):
        sdv.sample(z, u, 1.0)


def test_appending_many_rows():
    """One prompt of 2^24 - 1 rows behind a cache without pages; only the last rows have a place."""
    rows, D = 2 ** 24, 64
    k = torch.zeros((rows, 1, D), dtype=torch.bfloat16, device=DEV)
    k[-9:] = torch.randn((9, 1, D)).to(torch.bfloat16)
    kc = torch.zeros((2, 1, 1024, D), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    table = torch.full((1, 2 ** 14), -1, dtype=torch.int32, device=DEV)
    table[0, -1] = 1
    length = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(n):
        cu = torch.tensor([0, n - 1], dtype=torch.int32, device=DEV)
        sdv.kv_append(k[rows - n:], k[rows - n:], kc, vc, table, length, cu)

    run(rows - 1)
    assert torch.equal(kc[1, 0, :1023], k[-1023:, 0]) and torch.equal(vc, kc)
    assert not kc[0].any() and not kc[1, 0, 1023].any()
    with pytest.raises(sdv.SdvError, match="LIMIT"):
        run(rows)
