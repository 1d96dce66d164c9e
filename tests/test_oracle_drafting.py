"""The sampling and cache oracles against independent statements of the same definitions."""
import numpy as np
import pytest

from oracle import cache
from oracle.sample import sample_row


def test_the_draw_follows_the_truncated_distribution():
    """Uniforms on a fine even grid hit each token as often as its probability says."""
    z = np.array([1.0, -0.5, 2.0, 2.0, 0.0, -np.inf])
    for kw in ({}, dict(top_k=3), dict(top_p_milli=600), dict(min_p=0.2), dict(top_k=4, top_p_milli=900, min_p=0.1)):
        n = 4000
        got = np.bincount([sample_row(z, (i + 0.5) / n, 0.8, **kw)["token"] for i in range(n)], minlength=6) / n
        assert np.abs(got - sample_row(z, 0.5, 0.8, **kw)["probs"]).max() <= 1.0 / n


def test_truncations_by_enumeration():
    """The kept set is the smallest leading run that satisfies all three rules, found one rank at a time."""
    rng = np.random.default_rng(1)
    for _ in range(300):
        V = int(rng.integers(1, 9))
        z = np.round(rng.normal(size=V) * 2)
        k, p, mp = int(rng.integers(0, V + 2)), int(rng.choice([0, 300, 800, 1000])), float(rng.choice([0.0, 0.125, 1.0]))
        r = sample_row(z, rng.random(), 1.0, k, p, mp)
        ranks = sorted(range(V), key=lambda v: (-z[v], v))
        w = np.exp(z - z.max())
        top = ranks[:k] if 0 < k < V else ranks
        total, run, kept = sum(w[v] for v in top), 0.0, []
        for v in top:
            if p < 1000 and kept and run * 1000 >= p * total * (1 - 1e-12):
                break
            if w[v] < mp:
                break
            kept.append(v)
            run += w[v]
        assert r["kept"] == len(kept) and set(np.flatnonzero(r["probs"])) == set(kept)
        assert r["token"] in kept


def test_rows_that_describe_no_draw():
    z = np.array([0.0, 1.0])
    for bad in (dict(z=[-np.inf, np.nan]), dict(z=[np.inf, 0.0]), dict(T=-1.0), dict(T=np.nan), dict(u=1.0), dict(top_k=-1),
                dict(top_p_milli=1001), dict(min_p=1.5)):
        a = dict(z=z, u=0.5, T=1.0) | bad
        assert sample_row(np.array(a.pop("z")), a.pop("u"), a.pop("T"), **a)["token"] == -1
    assert sample_row(np.array([1.0, 3.0, 3.0]), 9.0, 0.0)["token"] == 1


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance_alone(interleaved):
    rng = np.random.default_rng(2)
    f = 10000.0 ** (-np.arange(4) / 4)
    q, k = rng.normal(size=(1, 12)), rng.normal(size=(1, 12))
    turn = lambda x, p: cache.rotate(x, p, f, interleaved)  # noqa: E731
    assert np.allclose(np.linalg.norm(turn(q, 77)), np.linalg.norm(q))
    assert np.array_equal(turn(q, 77)[:, 8:], q[:, 8:])
    assert np.allclose(turn(q, 1077) @ turn(k, 1000).T, turn(q, 77) @ turn(k, 0).T)


def test_attention_of_a_chain_is_that_of_a_linear_draft():
    rng = np.random.default_rng(3)
    kc, vc = rng.normal(size=(6, 2, 4, 8)), rng.normal(size=(6, 2, 4, 8))
    table, cu, length = np.array([[3, 1, 5], [0, 4, 2]]), np.array([0, 4, 6]), np.array([5, 7])
    q = rng.normal(size=(8, 4, 8))
    chain = [-1, 0, 1, 2, -1, 0]
    for window, sinks in ((0, 0), (3, 0), (3, 2)):
        a = cache.attend(q, kc, vc, table, length, cu, 0.5, window, sinks)[0]
        b = cache.attend(q, kc, vc, table, length, cu, 0.5, window, sinks, chain)[0]
        assert np.allclose(a, b)
    # one row by hand: request 1's row 0 (slot 7) in a window of 2, with one first token
    pick = [(0, 0), (4, 2), (4, 3)]  # slots 0, 6, 7
    k, v = (np.array([c[p, 1, s] for p, s in pick]) for c in (kc, vc))
    w = np.exp(k @ q[5, 3] * 0.5)
    got = cache.attend(q, kc, vc, table, length, cu, 0.5, 2, 1)[0][5, 3]
    assert np.allclose(got, (w / w.sum()) @ v)


def test_a_settled_tree_reads_as_the_linear_continuation():
    """Append a tree, settle a path: the cache holds what appending the path alone would have left."""
    rng = np.random.default_rng(4)
    parents, path, L = [-1, -1, 1, 0, 2, 4], [1, 2, 4, 5], 3
    f = 10000.0 ** (-np.arange(4) / 4)
    kc, vc = rng.normal(size=(5, 1, 4, 8)), rng.normal(size=(5, 1, 4, 8))
    table, keys, values = np.array([[4, 0, 2]]), rng.normal(size=(7, 1, 8)), rng.normal(size=(7, 1, 8))
    k1, v1, _ = cache.append(keys, values, kc, vc, table, [L], [0, 6], f, False, parents)
    nodes = np.array(path + [-1, -1])
    k2, v2, new = cache.settle(k1[None], v1[None], table, [L], [0, 6], [4], nodes)
    rows = [0] + [n + 1 for n in path]
    k3, v3, _ = cache.append(keys[rows], values[rows], kc, vc, table, [L], [0, 4], f)
    assert new[0] == L + 5
    for s in range(L + 5):
        pg, at = cache.place(table[0], 5, 4, s)
        assert np.allclose(k2[0, pg, :, at], k3[pg, :, at]) and np.array_equal(v2[0, pg, :, at], v3[pg, :, at])
