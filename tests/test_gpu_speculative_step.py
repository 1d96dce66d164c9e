"""Whole speculative rounds on a small two-layer model: draft with sample(), append the rows' keys and values,
attend, verify, settle.  At temperature 0 the tokens are those of decoding the target alone, which the test
computes without a cache in binary64 (its argmax margins are checked to exceed binary32's errors)."""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache_helpers import DEV

pytestmark = pytest.mark.gpu

V, H, HKV, D, LAYERS, PAGE, WINDOW, SINKS = 257, 4, 2, 64, 2, 16, 24, 2
E = H * D


class Model:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64) / s[0] ** 0.5  # noqa: E731
        self.embed = torch.randn((V, E), generator=g, dtype=torch.float64)
        self.qkv = [r(E, (H + 2 * HKV) * D) for _ in range(LAYERS)]
        self.o = [r(E, E) for _ in range(LAYERS)]
        self.head = r(E, V) * 4
        self.bigram = torch.randn((V, V), generator=g, dtype=torch.float64) * 2  # the drafter
        self.freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))

    def plain_logits(self, tokens):
        """Logits after the last token, no cache, binary64 on the host."""
        n = len(tokens)
        x, pos = self.embed[tokens], torch.arange(n, dtype=torch.float64)
        a = pos[:, None] * self.freq.float().double()
        c, s = a.cos()[:, None], a.sin()[:, None]
        turn = lambda t: torch.cat([t[..., :D // 2] * c - t[..., D // 2:] * s,  # noqa: E731
                                    t[..., D // 2:] * c + t[..., :D // 2] * s], -1)
        i = torch.arange(n)
        see = (i[None] <= i[:, None]) & ((i[:, None] - i[None] < WINDOW) | (i[None] < SINKS))
        for layer in range(LAYERS):
            y = (x @ self.qkv[layer]).view(n, H + 2 * HKV, D)
            q, k, v = turn(y[:, :H]), turn(y[:, H:H + HKV]), y[:, H + HKV:]
            k, v = (t.repeat_interleave(H // HKV, 1) for t in (k, v))
            w = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
            w = torch.softmax(w.masked_fill(~see, -torch.inf), -1)
            x = x + torch.einsum("hij,jhd->ihd", w, v).reshape(n, E) @ self.o[layer]
        return (x @ self.head)[-1]

    def decode(self, prompt, steps):
        tokens = list(prompt)
        for _ in range(steps):
            z = self.plain_logits(tokens)
            top = z.topk(2).values
            assert top[0] - top[1] > 1e-4 * z.abs().max()
            tokens.append(int(z.argmax()))
        return tokens

    def to_gpu(self):
        for name in ("embed", "head", "bigram", "freq"):
            setattr(self, name + "_g", getattr(self, name).float().to(DEV))
        self.qkv_g = [w.float().to(DEV) for w in self.qkv]
        self.o_g = [w.float().to(DEV) for w in self.o]


class Server:
    def __init__(self, model, B, max_len):
        self.m, self.B = model, B
        n = -(-max_len // PAGE)
        self.kc = torch.full((LAYERS, B * n, HKV, PAGE, D), float("nan"), device=DEV)
        self.vc = self.kc.clone()
        self.table = torch.randperm(B * n, generator=torch.Generator().manual_seed(0)).to(torch.int32).view(B, n).to(DEV)
        self.len = torch.zeros(B, dtype=torch.int32, device=DEV)

    def forward(self, tokens, cu, parents=None):
        x = self.m.embed_g[tokens.long()]
        at = (self.table, self.len, cu)
        for layer in range(LAYERS):
            y = (x @ self.m.qkv_g[layer]).view(-1, H + 2 * HKV, D)
            kc, vc = self.kc[layer], self.vc[layer]
            q = sdv.kv_append(y[:, H:H + HKV], y[:, H + HKV:], kc, vc, *at, parents=parents, inv_freq=self.m.freq_g,
                              queries=y[:, :H])
            o = sdv.attend(q, kc, vc, *at, parents=parents, window=WINDOW, sinks=SINKS)
            x = x + o.reshape(-1, E) @ self.m.o_g[layer]
        return x @ self.m.head_g


def offsets(ks):
    return torch.tensor(np.concatenate([[0], np.cumsum(ks)]), dtype=torch.int32, device=DEV)


def prompts(rng, B):
    return [list(rng.integers(0, V, size=n)) for n in [1, 5, 40][:B]]


def serve_prompts(s, ps):
    """All but the last token of each prompt enter the cache (in one call); the last is the frontier."""
    some = [i for i, p in enumerate(ps) if len(p) > 1]
    rows = torch.tensor([t for i in some for t in ps[i][:-1]], device=DEV)
    table, length = s.table, s.len
    s.table, s.len = table[some].contiguous(), length[some].contiguous()
    s.forward(rows, offsets([len(ps[i]) - 2 for i in some]))
    s.table, s.len = table, length
    s.len += torch.tensor([len(p) - 1 for p in ps], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("seed", [0, 1])
def test_linear_rounds_decode_the_target(seed):
    m = Model(seed)
    m.to_gpu()
    rng = np.random.default_rng(seed)
    ps = prompts(rng, 3)
    want = [m.decode(p, 24) for p in ps]
    s = Server(m, 3, 100)
    serve_prompts(s, ps)
    got, n_accepted = [list(p) for p in ps], 0
    for step in range(12):
        ks = rng.integers(0, 5, size=3)
        cu = offsets(ks)
        n_d = int(ks.sum())
        frontier = torch.tensor([g[-1] for g in got], device=DEV)
        drafts = torch.zeros(max(n_d, 1), dtype=torch.int32, device=DEV)
        prob = torch.zeros(max(n_d, 1), device=DEV)
        q_rows = torch.zeros((max(n_d, 1), V), device=DEV)
        last = frontier
        for j in range(int(ks.max())):  # the drafter's autoregressive steps; requests drop out at their K_i
            slots = torch.tensor([int(cu[i]) + j if j < ks[i] else -1 for i in range(3)], dtype=torch.int32, device=DEV)
            z = m.bigram_g[last.long()] if step % 2 else oracle_draft(m, got, j, want)
            sdv.sample(z, torch.tensor(rng.random(3), device=DEV), 0.7, top_k=torch.full((3,), 20, dtype=torch.int32, device=DEV),
                       slots=slots, out=(drafts, prob), probs=q_rows)
            last = torch.where(slots >= 0, drafts[slots.clamp(min=0).long()], last.int())
        drafts, q_rows = drafts[:n_d], q_rows[:n_d]
        tokens = torch.cat([torch.cat([frontier[i:i + 1].int(), drafts[int(cu[i]):int(cu[i + 1])]]) for i in range(3)])
        z = s.forward(tokens, cu)
        acc, out, _ = sdv.verify_ex(z, None, drafts, cu, 0.0, 1, draft_probs=q_rows)
        res = sdv.commit(cu, acc, out, s.len)
        s.len = s.len + 1 + acc
        off, new = res["offsets"].tolist(), res["tokens"].tolist()
        for i in range(3):
            got[i] += new[off[i]:off[i + 1]]
        n_accepted += int(acc.sum())
    assert n_accepted > 5
    for g, w in zip(got, want):
        n = min(len(g), len(w))
        assert n > 12 + 1 and g[:n] == w[:n]


def oracle_draft(m, got, j, want):
    """Draft logits that put most mass on the target's own continuation, so that drafts are accepted."""
    z = torch.zeros((3, V), device=DEV)
    for i in range(3):
        k = len(got[i]) + j
        if k < len(want[i]):
            z[i, want[i][k]] = 6.0
    return z


def test_tree_rounds_decode_the_target():
    m = Model(2)
    m.to_gpu()
    rng = np.random.default_rng(2)
    ps = prompts(rng, 3)
    want = [m.decode(p, 24) for p in ps]
    s = Server(m, 3, 120)
    serve_prompts(s, ps)
    got, depths = [list(p) for p in ps], []
    shape = [-1, -1, 1, 1, 3, 0]  # node 1's second child carries the target's own path: the path jumps
    parents = torch.tensor(shape * 3, dtype=torch.int32, device=DEV)
    cu = offsets([6, 6, 6])
    for step in range(8):
        nodes = []
        for g, w in zip(got, want):
            nxt = [w[len(g) + d] if len(g) + d < len(w) else 0 for d in range(3)]
            other = [(t + 1 + int(rng.integers(V - 1))) % V for t in nxt]
            nodes.append([other[0], nxt[0], other[1], nxt[1], nxt[2] if step % 2 else other[2], other[1]])
        drafts = torch.tensor([t for n in nodes for t in n], dtype=torch.int32, device=DEV)
        frontier = torch.tensor([g[-1] for g in got], dtype=torch.int32, device=DEV)
        tokens = torch.cat([torch.cat([frontier[i:i + 1], drafts[6 * i:6 * i + 6]]) for i in range(3)])
        z = s.forward(tokens, cu, parents)
        acc, out, path, _ = sdv.verify_tree(z, None, drafts, parents, cu, 0.0, 1)
        s.len = sdv.kv_settle(s.kc, s.vc, s.table, s.len, cu, acc, path)
        for i in range(3):
            a = int(acc[i])
            got[i] += out[int(cu[i]) + i:int(cu[i]) + i + a + 1].tolist()
            depths.append(a)
    assert max(depths) == 3
    for g, w in zip(got, want):
        n = min(len(g), len(w))
        assert n >= 24 and g[:n] == w[:n]
