"""Numbers whose lower 32 bits say something else."""
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache_helpers import DEV, Batch

pytestmark = pytest.mark.gpu


def test_windows_and_sinks():
    b = Batch([3, 0], [50, 20], 2, 64, 16, "bf16", 9, Hq=4)
    args = (b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), *b.index_args())
    want = sdv.attend(*args)
    for window in (2 ** 31 - 1, 2 ** 31 + 7, 2 ** 32 + 5, 2 ** 40 + 1):
        assert torch.equal(sdv.attend(*args, window=window), want)
    for sinks in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1):
        assert (sdv.attend(*args, window=4, sinks=sinks).float() - want.float()).abs().max() <= 2.0 ** -7 * want.abs().max()
    for kw in (dict(window=-2 ** 32), dict(window=-2 ** 31), dict(sinks=-2 ** 32), dict(sinks=-2 ** 32 + 3)):
        with pytest.raises(sdv.SdvError):
            sdv.attend(*args, **kw)


def test_a_row_beyond_32_bits():
    z = torch.zeros((1, 2 ** 32 + 5), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sdv.SdvError, match="LIMIT"):
        sdv.sample(z, torch.full((1,), 0.5, dtype=torch.float64, device=DEV))


def test_a_table_beyond_32_bits():
    b = Batch([0], [9], 1, 64, 16, "bf16", 9, Hq=1)
    table, length, cu = b.index_args()
    wide = torch.full((1, 2 ** 32 + 2), -1, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        sdv.attend(b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), wide, length, cu)
    with pytest.raises(ValueError):
        sdv.kv_append(b.k.to(DEV), b.v.to(DEV), b.kc.to(DEV), b.vc.to(DEV), wide, length, cu)
