"""min-p where its border lies next to a logit of zero: m + T ln(min_p) is then much smaller than either term, and
neighbouring logits of the row's type are much closer together than the border is known.

Counts are exact (see test_gpu_sample).  The border is computed in binary64 here and in the oracle, from terms of at
most 5: off by at most 2^-53 (5 + 5 + T) each, so a logit 1e-13 or more from it is on one known side; rows hold none closer.
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_sample import DT, check, uniforms

pytestmark = pytest.mark.gpu


def row(m, T, min_p, V, dtype, seed):
    """A row of maximum m with logits on both sides of zero at every scale down to 1e-12, none within 1e-13 of the border."""
    scales = 10.0 ** -np.arange(1.0, 13.0)
    near = np.concatenate([scales, -scales, 3 * scales, -3 * scales, np.linspace(0.01, 0.9 * m, 40)])
    rest = np.random.default_rng(seed).normal(-2.0, 2.0, V - 1 - len(near)).clip(-9.0, 0.95 * m)
    z = torch.tensor(np.concatenate([near, rest]), dtype=torch.float32).to(DT[dtype])
    border = m + T * math.log(float(np.float32(min_p)))
    z = torch.where((z.double() - border).abs() < 1e-13, torch.tensor(-3.0, dtype=DT[dtype]), z)
    z = torch.cat([z, torch.tensor([m], dtype=torch.float32).to(DT[dtype])])
    return z[torch.from_numpy(np.random.default_rng(seed + 1).permutation(V))]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [600, 9000, 40001])
def test_a_border_next_to_zero(V, dtype):
    """Maxima of the row's type next to -T ln(min_p), at the scalar temperature that puts the border there."""
    for k, (min_p, T0) in enumerate([(0.01, 1.0), (0.02, 0.3), (0.5, 2.0), (0.1, 0.7)]):
        p = float(np.float32(min_p))
        m = float(torch.tensor(-T0 * math.log(p), dtype=torch.float32).to(DT[dtype]))
        for T in (m / -math.log(p), m / -math.log(p) * (1 + 1e-9), m / -math.log(p) * (1 - 1e-9)):
            z = torch.stack([row(m, T, min_p, V, dtype, 10 * k + r) for r in range(2)])
            check(z, uniforms(2, k), T, min_p=min_p)
            check(z, uniforms(2, k), T, min_p=min_p, top_k=[0, 300], top_p=[999, 950])


@pytest.mark.parametrize("V", [600, 9000, 40001])
@pytest.mark.parametrize("T", [0.1, 0.5, 1.0, 2.0])
def test_neighbouring_maxima(V, T):
    """The 33 binary32 maxima around -T ln(min_p), a row each."""
    for min_p in (0.01, 0.02):
        p = float(np.float32(min_p))
        m = np.float32(-T * math.log(p))
        near = (m.view(np.uint32) + np.arange(-16, 17, dtype=np.int64)).astype(np.uint32).view(np.float32)
        z = torch.stack([row(float(x), T, min_p, V, "fp32", r) for r, x in enumerate(near)])
        check(z, uniforms(len(near), 3), [T] * len(near), min_p=min_p, probs=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [600, 40001])
@pytest.mark.parametrize("T", [1e-45, 1e-30, 1e-3, 30.0, 1e4, 1e30, 3e38])
def test_borders_far_from_zero_and_beyond_the_type(T, V, dtype):
    """Borders at the maximum itself, below the lowest finite logit, and between."""
    z = torch.randn((3, V), generator=torch.Generator().manual_seed(V)).to(DT[dtype])
    z[1] = z[1].abs() + torch.finfo(DT[dtype]).tiny
    z[2] = -z[2].abs()
    z[:, 5] = torch.finfo(DT[dtype]).min
    z[:, 7] = -float("inf")
    z[:, 11] = float("nan")
    check(z, uniforms(3, 5), [T] * 3, min_p=0.5)
    check(z, uniforms(3, 6), [T] * 3, min_p=[1e-45, 1e-30, 0.999])
