"""Whole speculative rounds over a cache in 8 bits whose pages are managed on the GPU: the pages from the lengths, appending, attention
under a window, verification at temperature 0, settling, the next lengths, with no length read on the host.

The codes round keys and values to 2^-4, so the tokens are those of decoding with the same rounding: the test decodes with the
package's own calls one token at a time (every round K = 0), which rounds each row alike as long as a block's scale does not
depend on its rejected drafts: blocks of one token.
"""
import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache_helpers import DEV
from test_gpu_speculative_step import D, E, H, HKV, LAYERS, PAGE, SINKS, V, WINDOW, Model, offsets

pytestmark = pytest.mark.gpu
PAGES = 30


class Server8:
    def __init__(self, model, B, block):
        self.m, self.B = model, B
        shape = (LAYERS, PAGES, HKV, PAGE, D)
        self.kc = torch.full(shape, 0x7f, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # NaN
        self.vc = self.kc.clone()
        self.ks = torch.full((LAYERS, PAGES, HKV, PAGE // block), 255, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
        self.vs = self.ks.view(torch.uint8).clone().view(torch.float8_e8m0fnu)
        self.table = torch.full((B, 12), -1, dtype=torch.int32, device=DEV)
        self.ring = torch.randperm(PAGES, generator=torch.Generator().manual_seed(0)).to(torch.int32).to(DEV)
        self.state = torch.tensor([7, PAGES], dtype=torch.int32, device=DEV)
        self.len = torch.zeros(B, dtype=torch.int32, device=DEV)

    def forward(self, tokens, cu, n_d, parents=None):
        placed, slots = sdv.kv_pages(self.table, self.len, cu, n_d, self.ring, self.state, PAGE, window=WINDOW, sinks=SINKS)
        x = self.m.embed_g[tokens.long()]
        at = (self.table, self.len, cu)
        for layer in range(LAYERS):
            y = (x @ self.m.qkv_g[layer]).view(-1, H + 2 * HKV, D)
            kc, vc = self.kc[layer], self.vc[layer]
            scales = dict(key_scales=self.ks[layer], value_scales=self.vs[layer])
            q = sdv.kv_append(y[:, H:H + HKV], y[:, H + HKV:], kc, vc, *at, parents=parents, inv_freq=self.m.freq_g,
                              queries=y[:, :H], **scales)
            o = sdv.attend(q, kc, vc, *at, parents=parents, window=WINDOW, sinks=SINKS, **scales)
            x = x + o.reshape(-1, E) @ self.m.o_g[layer]
        return x @ self.m.head_g, placed, slots


def decode(m, first, steps, block):
    """Tokens of B requests decoded one at a time, and the least margin of an argmax."""
    s = Server8(m, len(first), block)
    got, margin = [list(f) for f in first], np.inf
    cu = offsets([0] * len(first))
    longest = max(len(f) for f in first)
    for step in range(longest - 1 + steps):
        z, placed, _ = s.forward(torch.tensor([g[step] for g in got], dtype=torch.int32, device=DEV), cu, 0)
        assert placed.tolist() == [1] * len(first)
        s.len = s.len + 1
        top = z.topk(2, dim=1).values
        for i, g in enumerate(got):
            if len(g) == step + 1:
                g.append(int(z[i].argmax()))
                margin = min(margin, float((top[i, 0] - top[i, 1]) / z[i].abs().max()))
    return got, margin


@pytest.mark.parametrize("tree", [False, True])
def test_rounds_decode_as_one_token_at_a_time(tree):
    m = Model(3)
    m.to_gpu()
    rng = np.random.default_rng(3)
    first = [list(rng.integers(0, V, size=1)) for _ in range(3)]
    want, margin = decode(m, first, 60, 1)
    assert margin > 1e-4  # binary32's errors do not change a token
    s = Server8(m, 3, 1)
    got = [list(f) for f in first]
    shape = [-1, -1, 1, 1, 3, 0] if tree else None  # node 1's second child carries the target's own path
    depths = []
    for step in range(14):
        nodes, ks = [], []
        for i, (g, w) in enumerate(zip(got, want)):
            nxt = [w[len(g) + d] if len(g) + d < len(w) else 0 for d in range(4)]
            other = [(t + 1 + int(rng.integers(V - 1))) % V for t in nxt]
            if tree:
                nodes.append([other[0], nxt[0], other[1], nxt[1], nxt[2] if step % 2 else other[2], other[1]])
            else:
                good = int(rng.integers(0, 5))
                nodes.append((nxt[:good] + other[good:])[:int(rng.integers(0, 5))])
            ks.append(len(nodes[-1]))
        cu, n_d = offsets(ks), sum(ks)
        drafts = torch.tensor([t for n in nodes for t in n], dtype=torch.int32, device=DEV)
        tokens = torch.tensor([t for g, n in zip(got, nodes) for t in [g[-1]] + n], dtype=torch.int32, device=DEV)
        parents = torch.tensor(shape * 3, dtype=torch.int32, device=DEV) if tree else None
        z, placed, slots = s.forward(tokens, cu, n_d, parents)
        assert placed.tolist() == [1, 1, 1] and (slots >= 0).all()
        if tree:
            acc, out, path, _ = sdv.verify_tree(z, None, drafts, parents, cu, 0.0, 1)
            s.len = sdv.kv_settle(s.kc, s.vc, s.table, s.len, cu, acc, path, key_scales=s.ks, value_scales=s.vs)
        else:
            q_rows = torch.zeros((n_d, V), device=DEV)
            q_rows[torch.arange(n_d, device=DEV), drafts.long()] = 1.0
            acc, out, _ = sdv.verify_ex(z, None, drafts, cu, 0.0, 1, draft_probs=q_rows)
            s.len = s.len + 1 + acc
        for i in range(3):
            a = int(acc[i])
            got[i] += out[int(cu[i]) + i:int(cu[i]) + i + a + 1].tolist()
            depths.append(a)
    assert max(depths) >= 3
    for g, w in zip(got, want):
        n = min(len(g), len(w))
        assert n >= 20 and g[:n] == w[:n]
    held = s.table[s.table >= 0].tolist()
    first_free, free = s.state.tolist()
    assert sorted(held + [int(s.ring[(first_free + x) % PAGES]) for x in range(free)]) == list(range(PAGES))


def test_a_round_in_a_graph():
    """Pages, append, attention and settling captured once: each replay goes on from the lengths that the one before left."""
    m = Model(4)
    m.to_gpu()
    B, K = 3, 6
    shape = [-1, -1, 1, 1, 3, 0]
    parents = torch.tensor(shape * B, dtype=torch.int32, device=DEV)
    cu = offsets([K] * B)
    rounds = [torch.randint(0, V, ((K + 1) * B,), generator=torch.Generator().manual_seed(r)).to(DEV) for r in range(5)]
    paths = [[1, 3, 4, -1, -1, -1], [0, 5, -1, -1, -1, -1], [1, 2, -1, -1, -1, -1]]
    acc = torch.tensor([3, 2, 0], dtype=torch.int32, device=DEV)
    nodes = torch.tensor(sum(paths, []), dtype=torch.int32, device=DEV)
    tokens = torch.zeros((K + 1) * B, dtype=torch.int64, device=DEV)

    def step(s):
        z, placed, slots = s.forward(tokens, cu, K * B, parents)
        new = sdv.kv_settle(s.kc, s.vc, s.table, s.len, cu, acc, nodes, key_scales=s.ks, value_scales=s.vs)
        s.len.copy_(new)
        return z, placed, slots

    eager, replayed = Server8(m, B, 16), Server8(m, B, 16)
    want = []
    for r in rounds:
        tokens.copy_(r)
        want.append([x.clone() for x in step(eager)] + [eager.len.clone()])
    start = [x.clone() for x in (replayed.table, replayed.ring, replayed.state, replayed.len)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(replayed)  # libraries set themselves up
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = step(replayed)
    torch.cuda.synchronize()
    for x, y in zip((replayed.table, replayed.ring, replayed.state, replayed.len), start):
        x.copy_(y)
    for r, w in zip(rounds, want):
        tokens.copy_(r)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[1], w[1]) and torch.equal(out[2], w[2]) and torch.equal(replayed.len, w[3])
        assert (out[0] - w[0]).abs().max() <= 2.0 ** -16 * w[0].abs().max()
