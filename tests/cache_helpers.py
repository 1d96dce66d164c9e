"""Seeded paged caches for the cache tests: layouts, trees, pages in random order."""
import numpy as np
import torch

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def random_tree(rng, K):
    return [int(rng.choice([n - 1, rng.integers(-1, n)])) for n in range(K)]


class Batch:
    """ks: K_i of each request, lens: L_i; the tables hold spare pages, in random order."""

    def __init__(self, ks, lens, Hkv, D, page, dtype, seed, tree=False, Hq=0, layers=0, spare=2):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.ks, self.lens, self.B = list(ks), list(lens), len(ks)
        self.cu = np.concatenate([[0], np.cumsum(ks)]).astype(np.int32)
        self.n_d = int(self.cu[-1])
        self.rows = self.n_d + self.B
        need = [-(-(n + k + 1) // page) for n, k in zip(lens, ks)]
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.full((self.B, max(need) + 1), -1, dtype=np.int32)
        at = 0
        for i, m in enumerate(need):
            self.table[i, :m] = order[at:at + m]
            at += m
        self.trees = [random_tree(rng, k) for k in ks] if tree else None
        self.parents = np.array([p for t in self.trees for p in t], dtype=np.int32) if tree else None
        shape = (self.n_pages, Hkv, page, D)
        if layers:
            shape = (layers,) + shape
        t = lambda *s: torch.randn(s, generator=g).to(DT[dtype])  # noqa: E731
        self.kc, self.vc = t(*shape), t(*shape)
        self.k, self.v = t(self.rows, Hkv, D), t(self.rows, Hkv, D)
        self.q = t(self.rows, Hq, D) if Hq else None
        self.len = np.array(lens, dtype=np.int32)

    def index_args(self):
        return [torch.from_numpy(x).to(DEV) for x in (self.table, self.len, self.cu)]

    def tree_arg(self):
        return None if self.parents is None else torch.from_numpy(self.parents).to(DEV)


def np64(t):
    return t.detach().double().cpu().numpy()
