"""Temperatures given as a number, which is binary64: down to 5e-324 and up to 1.7e308, where binary32 holds neither T nor
the distance at which a weight vanishes, and 1 / T may not be finite in binary64.

At T <= 2^-160 a logit below the maximum lies at least 2^-149 below it and has the weight e^-2048 or less, 0 in binary64; at
T >= 2^200 every finite logit has the weight 1 to the last bit.  Tolerances as in test_gpu_sample.
"""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from test_gpu_sample import DEV, DT, check, logits_of, place, uniforms

pytestmark = pytest.mark.gpu

TEMPERATURES = [5e-324, 1e-310, 1e-307, 1e-160, 1e-50, 1e-48, 3e-47, 2.0 ** -149, 1e-40, 1e40, 1e200, 1e305, 1e306, 1.7e308]


def rows(V, dtype):
    z = logits_of(5, V, dtype, V)
    z[1, V // 3:V // 3 + 4] = 40.0  # copies of the maximum
    z[2] = -z[2].abs() - 1.0
    z[3, 3:] = -float("inf")
    z[4, ::3] = float("nan")
    return z


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [700, 40001])
@pytest.mark.parametrize("T", TEMPERATURES)
def test_numbers(T, V, dtype):
    z = rows(V, dtype)
    check(z, uniforms(5, 1), T)
    check(z, uniforms(5, 2), T, top_k=[7, 3, 0, 2, 650], top_p=[1000, 500, 900, 300, 1000])
    check(z, uniforms(5, 3), T, min_p=0.5)


@pytest.mark.parametrize("V", [700, 40001])
@pytest.mark.parametrize("T", [1e-45, 3e-45, 1e-48, 1e-47, 2.0 ** -155, 2.0 ** -160, 2.0 ** -170])
def test_logits_as_small_as_the_temperature(T, V):
    """Rows of binary32's smallest numbers: at these temperatures, weights between 0 and 1."""
    z = (torch.randint(-40, 41, (3, V), generator=torch.Generator().manual_seed(7)).double() * 2.0 ** -149).float()
    check(z, uniforms(3, 4), T)
    check(z, uniforms(3, 5), T, top_k=[50, 0, 600], top_p=[900, 500, 1000], min_p=[0.0, 0.2, 0.01])


@pytest.mark.parametrize("n", [5, 300])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_outputs_are_written(dtype, n):
    """Every row's outputs, over what the buffers held before."""
    z = place(logits_of(n, 40001, dtype, 8))
    u = torch.tensor(uniforms(n, 9), device=DEV)
    for T in (5e-324, 1e-50):
        out = (torch.full((n,), -7, dtype=torch.int32, device=DEV), torch.full((n,), -7.0, device=DEV))
        kept = torch.full((n,), -7, dtype=torch.int32, device=DEV)
        tok, prob, _ = sdv.sample(z, u, T, out=out, kept_tokens=kept)
        tok, prob, host = tok.cpu().numpy(), prob.cpu().numpy(), z.float().cpu().numpy()
        best = host.max(1)
        assert ((tok >= 0) & (tok < 40001)).all()
        assert np.array_equal(host[np.arange(n), tok], best)
        copies = (host == best[:, None]).sum(1)
        assert (np.abs(prob * copies - 1) <= 2.0 ** -23).all() and (kept == 40001).all()
