"""Sampling on the GPU against the binary64 oracle.

Tolerances.  Tokens and kept counts are those of the definition: a kernel weight is within 2.2e-12 of
its value, so a draw whose uniform lies 1e-10 or more from every border of the oracle's distribution function
has one possible token.  prob is a binary64 quotient rounded once (2^-24, plus the weights' 5e-12).  A probs cell is a
binary32 product of 2^r (the hardware exponential, one step: 2^-23; its argument |r| <= 1/2 rounded by
2^-26), the rounded 1 / S (2^-24) and one rounding of the product (2^-24): under 2^-22 in all; below
2^-126 a subnormal's step of 2^-149 or a flush to zero replaces the relative bound.
"""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from oracle.sample import sample_row

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
PROB_REL, PROBS_REL = 2.0 ** -24 + 1e-11, 2.0 ** -22


def place(z, pad=0, shift=0):
    """z [n, V] on the device with rows V + pad apart, `shift` elements into a fresh buffer."""
    n, V = z.shape
    buf = torch.full((shift + n * (V + pad) + 8,), 77.0, dtype=z.dtype, device=DEV)
    view = buf[shift:shift + n * (V + pad)].view(n, V + pad)[:, :V]
    view.copy_(z)
    return view


def check(z, u, T, top_k=None, top_p=None, min_p=None, probs=True, **layout):
    """Runs the batch and compares every row.  T, top_k, ...: numbers or one value per row."""
    n, V = z.shape
    row = lambda v, d: np.broadcast_to(np.asarray(d if v is None else v), (n,))  # noqa: E731
    dev = lambda v, t: None if v is None else torch.tensor(np.array(row(v, 0)), dtype=t, device=DEV)  # noqa: E731
    u = np.array(row(u, 0.5), dtype=np.float64)
    logits = place(z, **layout)
    temp = float(T) if np.ndim(T) == 0 else dev(T, torch.float32)
    tok, prob, extra = sdv.sample(logits, torch.tensor(u, device=DEV), temp, top_k=dev(top_k, torch.int32),
                                  top_p_milli=dev(top_p, torch.int32), min_p=dev(min_p, torch.float32), probs=probs)
    tok, prob, kept = tok.cpu().numpy(), prob.cpu().numpy(), extra["kept_tokens"].cpu().numpy()
    cells = extra["probs"].cpu().numpy() if probs else None
    z64 = z.double().cpu().numpy()
    Ts = row(T, 1.0).astype(np.float32) if np.ndim(T) else row(T, 1.0).astype(np.float64)
    for r in range(n):
        ref = sample_row(z64[r], u[r], float(Ts[r]), int(row(top_k, 0)[r]), int(row(top_p, 1000)[r]),
                         float(row(min_p, 0.0)[r]))
        if ref["margin"] >= 1e-10:
            assert tok[r] == ref["token"], (r, tok[r], ref["token"], ref["margin"])
            assert abs(prob[r] - ref["prob"]) <= PROB_REL * ref["prob"]
        assert kept[r] == ref["kept"], r
        if probs:
            assert np.all(np.abs(cells[r] - ref["probs"]) <= PROBS_REL * ref["probs"] + 2.0 ** -125), r
    return tok, prob, cells


def logits_of(n, V, dtype, seed, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, V), generator=g) * sigma).to(DT[dtype])


def uniforms(n, seed):
    return np.random.default_rng(seed).random(n)


PROFILES = {
    "plain": {},
    "top_k": dict(top_k=[1, 2, 40, 0]),
    "top_p": dict(top_p=[0, 500, 900, 1000]),
    "min_p": dict(min_p=[0.0, 0.02, 0.5, 1.0]),
    "all": dict(top_k=[50, 7, 0, 300], top_p=[900, 1000, 950, 990], min_p=[0.01, 0.0, 0.05, 0.001]),
}


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [1, 2, 7, 64, 1000, 4099, 32000, 128256])
def test_profiles(V, dtype, profile):
    check(logits_of(4, V, dtype, V), uniforms(4, V + 1), [1.0, 0.7, 1.3, 2.5], **PROFILES[profile])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (7, 3), (64, 0), (5, 5)])
def test_strides_and_bases_off_the_16_byte_grid(dtype, pad, shift):
    for V in (1000, 8192, 20001):
        check(logits_of(3, V, dtype, V + pad), uniforms(3, pad), 0.9, top_k=[0, 30, 0], top_p=[1000, 900, 800],
              pad=pad, shift=shift)
        check(logits_of(3, V, dtype, V + pad), uniforms(3, pad + 1), 0.9, pad=pad, shift=shift)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_rows_take_long_chunks(dtype):
    n, V = 300, 33000
    rng = np.random.default_rng(5)
    check(logits_of(n, V, dtype, 6), uniforms(n, 7), rng.uniform(0.5, 1.5, n), probs=False,
          top_k=rng.choice([0, 1, 50, 500], n), top_p=rng.choice([1000, 900, 300], n), min_p=rng.choice([0, 0.1], n))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_vocabulary_of_more_chunks_than_threads(dtype):
    V = 2_500_000 if dtype == "bf16" else 1_300_000
    z = logits_of(2, V, dtype, 8)
    check(z, [0.37, 0.999], 1.0, probs=False)
    check(z, [0.37, 0.999], 1.0, top_k=[0, 900], top_p=[700, 999], probs=False)
    z = torch.zeros((2, V), dtype=DT[dtype])  # every copy of one key, cut in the middle
    check(z, [0.25, 0.75], 1.0, top_k=[V // 2 + 3, 0], top_p=[1000, 250], probs=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_equal_logits_rank_by_id(dtype):
    V = 5000
    z = torch.zeros((6, V), dtype=DT[dtype])
    z[3:, ::7] = 2.0
    z[5] = torch.tensor([0.0, -0.0], dtype=DT[dtype]).repeat(V // 2)  # the two zeros are one value
    check(z, uniforms(6, 9), 1.0, top_k=[10, 1, 4999, 715, 714, 33])
    check(z, uniforms(6, 10), 1.0, top_p=[500, 1, 999, 300, 0, 500])
    check(z, uniforms(6, 11), 1.0, top_k=[100, 100, 100, 1000, 1000, 1000], top_p=[500, 333, 10, 900, 999, 200])
    check(z, uniforms(6, 12), 1.0, min_p=[1.0, 0.5, 0.1, 1.0, 0.13, 0.14])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [3000, 90000])
def test_log_probabilities_and_narrow_rows(V, dtype):
    """Rows without a positive logit, rows whose logits lie close together, and cuts far below the maximum."""
    z = torch.log_softmax(logits_of(6, V, "fp32", 30), 1)
    z[1] = 5.0 + 0.01 * torch.randn(V, generator=torch.Generator().manual_seed(31))
    z[2] = -3.0 + 1e-4 * torch.randn(V, generator=torch.Generator().manual_seed(32))
    z[3] = 0.001 * z[3]
    z[4, 100:] -= 200.0
    z = z.to(DT[dtype])
    check(z, uniforms(6, 33), 1.0)
    check(z, uniforms(6, 34), 0.9, top_p=[900, 900, 500, 999, 990, 10])
    check(z, uniforms(6, 35), 0.9, top_k=[50, 2500, 2000, 2999, 700, 1], top_p=[950, 1000, 700, 1000, 400, 1000])
    check(z, uniforms(6, 36), 1.1, min_p=[0.001, 0.99, 0.9999, 0.9, 1e-30, 0.5])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masked_and_special_logits(dtype):
    V = 3001
    inf, nan = float("inf"), float("nan")
    lowest = torch.finfo(DT[dtype]).min
    z = logits_of(10, V, dtype, 13)
    z[0, 5:] = -inf
    z[1, :] = -inf
    z[2, 100] = inf
    z[3, ::2] = nan
    z[4, :] = nan
    z[5, 1:] = lowest
    z[6, :] = lowest
    z[7, :2999] = -inf
    z[8, 17] = -nan
    for kw in ({}, dict(top_k=20), dict(top_p=900), dict(min_p=0.05), dict(top_k=2000, top_p=990)):
        tok, prob, cells = check(z, uniforms(10, 14), 0.8, **kw)
        assert list(tok[[1, 2, 4]]) == [-1] * 3 and not cells[[1, 2, 4]].any() and not prob[[1, 2, 4]].any()
        assert tok[5] == 0 and tok[3] % 2 == 1 and tok[7] >= 2999
    tok, _, _ = check(z, 0.3, 0.0)
    assert list(tok[[1, 2, 4]]) == [-1] * 3


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1e-45, 1e-30, 1e-3, 0.02, 50.0, 1e6, 3e38])
def test_extreme_temperatures(dtype, T):
    z = logits_of(3, 2000, dtype, 15)
    check(z, uniforms(3, 16), [T] * 3)
    check(z, uniforms(3, 17), [T] * 3, top_k=[1999, 3, 0], top_p=[600, 1000, 900])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_uniforms_at_their_ends(dtype):
    z = logits_of(4, 9000, dtype, 18)
    z[2, 8990:] = -float("inf")
    u = [0.0, 1.0 - 2.0 ** -53, 1.0 - 2.0 ** -53, 2.0 ** -60]
    for kw in ({}, dict(top_k=50), dict(top_p=700)):
        tok, _, _ = check(z, u, 1.0, **kw)
        assert (tok >= 0).all() and tok[2] < 8990


def test_profiles_that_describe_no_draw():
    z = logits_of(9, 500, "bf16", 19)
    nan = float("nan")
    T = [1.0, -1.0, nan, float("inf"), 1.0, 1.0, 1.0, 1.0, 1.0]
    tok, prob, cells = check(z, [1.0, .5, .5, .5, -0.1, nan, .5, .5, .5], T, top_k=[0] * 6 + [-1, 0, 5],
                             top_p=[1000] * 7 + [1001, 900], min_p=[0.0] * 8 + [0.1])
    assert (tok[:8] == -1).all() and tok[8] >= 0 and not cells[:8].any()
    tok, _, _ = check(z, 0.5, 1.0, min_p=[-0.1, 1.5, nan] * 3)
    assert (tok == -1).all()
    tok, _, _ = check(z, 2.0, 0.0, top_k=[-5] * 9)  # T = 0 takes its argmax under any truncation and uniform
    assert (tok >= 0).all()


def test_slots_place_and_skip_rows():
    n, V = 6, 700
    z = place(logits_of(n, V, "bf16", 20))
    u = torch.tensor(uniforms(n, 21), device=DEV)
    tok, prob, ex = sdv.sample(z, u, 1.0, probs=True)
    out = (torch.full((9,), -7, dtype=torch.int32, device=DEV), torch.full((9,), -7.0, device=DEV))
    kept = torch.full((9,), -7, dtype=torch.int32, device=DEV)
    probs = torch.full((9, V), -7.0, device=DEV)
    slots = torch.tensor([8, -1, 0, 9, 3, -2 ** 31], dtype=torch.int32, device=DEV)
    t2, p2, e2 = sdv.sample(z, u, 1.0, probs=probs, slots=slots, out=out, kept_tokens=kept)
    assert t2 is out[0] and e2["probs"] is probs
    for r, s in ((0, 8), (2, 0), (4, 3)):
        assert t2[s] == tok[r] and p2[s] == prob[r] and kept[s] == V and torch.equal(probs[s], ex["probs"][r])
    for s in (1, 2, 4, 5, 6, 7):
        assert t2[s] == -7 and p2[s] == -7 and kept[s] == -7 and (probs[s] == -7).all()


def test_the_same_call_gives_the_same_bits():
    z = place(logits_of(64, 50000, "fp32", 22))
    u = torch.tensor(uniforms(64, 23), device=DEV)
    p = torch.full((64,), 900, dtype=torch.int32, device=DEV)
    first = sdv.sample(z, u, 1.0, top_p_milli=p, probs=True)
    for _ in range(3):
        again = sdv.sample(z, u, 1.0, top_p_milli=p, probs=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert torch.equal(first[2]["probs"], again[2]["probs"])


def test_graph_replays_and_another_stream():
    z = place(logits_of(8, 32000, "bf16", 24))
    u = torch.tensor(uniforms(8, 25), device=DEV)
    k = torch.full((8,), 50, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sdv.sample(z, u, 1.0, top_k=k, probs=True)
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                res = sdv.sample(z, u, 1.0, top_k=k, probs=True)
            graphs.append((g, res))
    torch.cuda.synchronize()
    for step in range(4):
        u.copy_(torch.tensor(uniforms(8, 26 + step)))
        z.copy_(logits_of(8, 32000, "bf16", 40 + step))
        want = sdv.sample(z, u, 1.0, top_k=k, probs=True)
        torch.cuda.synchronize()
        for g, res in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, res in graphs:
            assert torch.equal(res[0], want[0]) and torch.equal(res[2]["probs"], want[2]["probs"])


def test_draws_feed_the_verification():
    """Drafts and q rows go straight into verify_ex; a drafter that is the target is always accepted."""
    B, K, V = 5, 3, 4000
    z = place(logits_of(B * K, V, "fp32", 50))
    tok, prob, ex = sdv.sample(z, torch.tensor(uniforms(B * K, 51), device=DEV), 1.0, probs=True)
    cu = torch.arange(0, B * K + 1, K, dtype=torch.int32, device=DEV)
    target = torch.cat([torch.cat([z[i * K:(i + 1) * K], z[i * K:i * K + 1]]) for i in range(B)]).contiguous()
    r = torch.full((B * K,), 0.999, dtype=torch.float64, device=DEV)
    w = torch.full((B * K + B,), 0.5, dtype=torch.float64, device=DEV)
    acc, out, extra = sdv.verify_ex(target, None, tok, cu, 1.0, 1, draft_probs=ex["probs"], accept_uniform=r,
                                    draw_uniform=w, diag=("draft_logit",))
    assert (acc == K).all()
    assert torch.equal(extra["draft_logit"], ex["probs"].gather(1, tok[:, None].long())[:, 0])
    assert ((extra["draft_logit"] - prob).abs() <= 2.0 ** -21 * prob).all()


def test_refusals():
    z = place(logits_of(4, 100, "bf16", 60))
    u = torch.full((4,), 0.5, dtype=torch.float64, device=DEV)
    with pytest.raises(TypeError):
        sdv.sample(z.half(), u)
    with pytest.raises(ValueError):
        sdv.sample(z.t(), u)
    with pytest.raises(ValueError):
        sdv.sample(z, u.float())
    with pytest.raises(ValueError):
        sdv.sample(z, u[:3])
    with pytest.raises(ValueError):
        sdv.sample(z, u, top_k=torch.zeros(4, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        sdv.sample(z, u, probs=torch.zeros((4, 99), device=DEV))
    with pytest.raises(ValueError):
        sdv.sample(z, u, slots=torch.zeros(4, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        sdv.sample(z[:1].expand(4, 100), u)
    for T in (-1.0, float("nan"), float("inf")):
        with pytest.raises(sdv.SdvError):
            sdv.sample(z, u, T)
    with pytest.raises(sdv.SdvError):
        sdv.sample(z, u, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
