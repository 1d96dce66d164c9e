"""Rows too long for one workgroup: their chunks' masses, maxima and frames, and how the rows' own pass puts them together.

A chunk of a few rows holds 4 x 64 vectors (1024 binary32 or 2048 bf16 logits), one of many rows 16 x 64.  Tolerances as in
test_gpu_sample.
"""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from test_gpu_sample import DEV, DT, check, logits_of, place, uniforms

pytestmark = pytest.mark.gpu
V = 40001
INF = float("inf")
# a row's kinds, of which [2, 3, 9, 11] have no draw
NONE = [2, 3, 9, 11]


def special_rows(dtype):
    z = logits_of(13, V, dtype, 3)
    z[1, :9000] = -INF  # whole chunks without a logit
    z[2, :] = -INF
    z[3, 39990] = INF  # in a later chunk than the rest
    z[4, 17000:17100] += 3000.0  # a chunk whose weights leave binary64 as they are
    z[5, 8192:24576] = float("nan")
    z[6, :] = torch.finfo(DT[dtype]).min
    z[6, 20000:20010] = -1.0
    z[7] = z[7].clamp(max=5.0)  # the maximum many times, over many chunks
    z[8, 16384:] -= 2000.0
    z[9, :] = float("nan")
    z[10, :32768] = -900.0  # chunks next to the borders of what a chunk's sum may be
    z[10, 32768:36000] = 690.0
    z[11, 0] = INF
    z[12, :] = -INF
    z[12, 40000] = -3.0
    return z


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1.0, 1e-3, 0.3, 1e3])
@pytest.mark.parametrize("profile", [{}, dict(top_k=60), dict(top_p=700), dict(min_p=0.01), dict(top_k=3000, top_p=950, min_p=1e-4)])
def test_chunks(profile, T, dtype, many):
    z = special_rows(dtype)
    if many:  # the special rows among enough others for long chunks
        at = torch.arange(13) * 20
        rest = logits_of(260, V, dtype, 4)
        rest[at] = z
        z = rest
    n = z.shape[0]
    if not many:
        tok, prob, cells = check(z, uniforms(n, 5), T, **profile)
        assert (tok[NONE] == -1).all() and not prob[NONE].any() and not cells[NONE].any()
        assert tok[12] == 40000 and tok[1] >= 9000
        return
    few = check(z[at], uniforms(13, 5), T, **profile)[0]
    u = np.random.default_rng(6).random(n)
    u[at.numpy()] = uniforms(13, 5)
    kw = {"top_k": torch.int32, "top_p": torch.int32, "min_p": torch.float32}
    given = {("top_p_milli" if k == "top_p" else k): torch.full((n,), v, dtype=kw[k], device=DEV) for k, v in profile.items()}
    logits = place(z)
    tok, prob, extra = sdv.sample(logits, torch.tensor(u, device=DEV), T, probs=True, **given)
    one = sdv.sample(logits[at].contiguous(), torch.tensor(uniforms(13, 5), device=DEV), T, probs=True,
                     **{k: v[:13] for k, v in given.items()})
    assert np.array_equal(tok[at].cpu().numpy(), few)
    assert torch.equal(extra["kept_tokens"][at], one[2]["kept_tokens"])
    # both ways are within 2^-22 of the oracle's cells
    a, b = extra["probs"][at], one[2]["probs"]
    assert ((a - b).abs() <= 2.0 ** -21 * b + 2.0 ** -125).all()


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_long_chunks_against_the_oracle(dtype, many):
    """Few profiles, but every row: temperatures from 0 to 50 in one batch."""
    z = special_rows(dtype)
    if many:
        z = torch.cat([z] * 17)
    n = z.shape[0]
    T = np.random.default_rng(7).choice([0.0, 1e-3, 0.05, 1.0, 50.0], n)
    tok, prob, cells = check(z, uniforms(n, 8), T)
    kind = np.arange(n) % 13
    assert (tok[np.isin(kind, NONE)] == -1).all()
    check(z, uniforms(n, 9), T, top_k=np.random.default_rng(10).choice([0, 1, 100, 30000], n), probs=False)


@pytest.mark.parametrize("n", [7, 230])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_argmax_over_chunks(dtype, n):
    """T = 0: the first of the copies of the maximum, wherever they are, and its one-hot row."""
    z = logits_of(n, V, dtype, 11).clamp(max=4.0)
    rng = np.random.default_rng(12)
    first = []
    for r in range(n):
        ids = np.sort(rng.choice(V, 3, replace=False))
        if r % 3 == 0:
            ids[0] = rng.choice([0, V - 1, 2048, 8191])
        z[r, torch.from_numpy(ids)] = 9.0
        first.append(int(ids.min()))
    tok, prob, extra = sdv.sample(place(z, pad=3, shift=1), torch.full((n,), 0.9, dtype=torch.float64, device=DEV), 0.0,
                                  probs=True, top_k=torch.full((n,), 50, dtype=torch.int32, device=DEV))
    assert tok.tolist() == first and (prob == 1).all() and (extra["kept_tokens"] == 1).all()
    want = torch.zeros((n, V), device=DEV)
    want[torch.arange(n), torch.tensor(first)] = 1.0
    assert torch.equal(extra["probs"], want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_uniforms_at_their_ends_of_long_rows(dtype):
    z = logits_of(4, V, dtype, 13)
    z[2, 30000:] = -INF
    z[3, :5000] = -INF
    u = [0.0, 1.0 - 2.0 ** -53, 1.0 - 2.0 ** -53, 0.0]
    for kw in ({}, dict(top_k=50), dict(top_p=700)):
        tok, _, cells = check(z, u, 1.0, **kw)
        assert (tok >= 0).all() and tok[2] < 30000 and tok[3] >= 5000
        kept = cells > 0
        assert tok[0] == kept[0].argmax() and tok[3] == kept[3].argmax()
        for r in (1, 2):
            assert tok[r] == V - 1 - kept[r][::-1].argmax()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [0.0, 1.0])
def test_slots_of_long_rows(T, dtype):
    z = place(special_rows(dtype)[:6])
    u = torch.tensor(uniforms(6, 14), device=DEV)
    k = torch.full((6,), 40, dtype=torch.int32, device=DEV)
    for kw in ({}, dict(top_k=k)):
        tok, prob, ex = sdv.sample(z, u, T, probs=True, **kw)
        out = (torch.full((9,), -7, dtype=torch.int32, device=DEV), torch.full((9,), -7.0, device=DEV))
        kept = torch.full((9,), -7, dtype=torch.int32, device=DEV)
        probs = torch.full((9, V), -7.0, device=DEV)
        slots = torch.tensor([8, -1, 0, 9, 3, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
        sdv.sample(z, u, T, probs=probs, slots=slots, out=out, kept_tokens=kept, **kw)
        for r, s in ((0, 8), (2, 0), (4, 3)):
            assert out[0][s] == tok[r] and out[1][s] == prob[r] and kept[s] == ex["kept_tokens"][r]
            assert torch.equal(probs[s], ex["probs"][r])
        for s in (1, 2, 4, 5, 6, 7):
            assert out[0][s] == -7 and out[1][s] == -7 and kept[s] == -7 and (probs[s] == -7).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_rows_that_describe_no_draw(dtype):
    z = logits_of(9, V, dtype, 15)
    nan = float("nan")
    T = [1.0, -1.0, nan, INF, 1.0, 1.0, 1.0, 1.0, 1.0]
    tok, prob, cells = check(z, [1.0, .5, .5, .5, -0.1, nan, .5, .5, .5], T, top_k=[0] * 6 + [-1, 0, 5],
                             top_p=[1000] * 7 + [1001, 900], min_p=[0.0] * 8 + [0.1])
    assert (tok[:8] == -1).all() and tok[8] >= 0 and not cells[:8].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_lowest_uniform_among_weights_that_vanish(dtype):
    """u = 0 takes the first token with a weight: logits 749 below the maximum have none in binary64, though the sum of a
    thousand of them would be above its smallest number."""
    z = torch.full((2, 40001), -7.0).to(DT[dtype])
    z[0, 30000:30003] = 742.0
    z[1, 39000:] = -float("inf")
    z[1, 20000] = 742.0
    tok, prob, extra = sdv.sample(place(z), torch.zeros(2, dtype=torch.float64, device=DEV), 1.0, probs=True, out=(
        torch.full((2,), -7, dtype=torch.int32, device=DEV), torch.full((2,), -7.0, device=DEV)))
    assert tok.tolist() == [30000, 20000]
    assert np.allclose(prob.cpu().numpy(), [1 / 3, 1.0], rtol=2.0 ** -23, atol=0)
    assert extra["kept_tokens"].tolist() == [40001] * 2
