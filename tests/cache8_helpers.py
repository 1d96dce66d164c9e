"""Seeded paged caches in 8 bits for the cache tests."""
import numpy as np
import torch

import lossless_draft_verification_online_amd as sdv
from cache_helpers import DEV, DT, Batch
from oracle import cache8 as oracle

CODES, SCALES = torch.float8_e4m3fn, torch.float8_e8m0fnu


class Batch8(Batch):
    """A Batch whose caches are codes of about 100 (values of about 1) under scales of 2^-9 to 2^-5 per block; rows in dtype."""

    def __init__(self, ks, lens, Hkv, D, page, block, dtype, seed, **kw):
        super().__init__(ks, lens, Hkv, D, page, "fp32", seed, **kw)
        rng = np.random.default_rng(seed + 1)
        self.block, self.page, self.dtype = block, page, dtype
        self.kc, self.vc = (oracle.encode(x.double().numpy() * 100) for x in (self.kc, self.vc))
        shape = self.kc.shape[:-2] + (page // block,)
        self.ks8, self.vs8 = (rng.integers(118, 123, shape).astype(np.uint8) for _ in range(2))
        self.k, self.v = self.k.to(DT[dtype]), self.v.to(DT[dtype])
        self.q = None if self.q is None else self.q.to(DT[dtype])

    def caches(self):
        """Device tensors: key codes, value codes, key scales, value scales."""
        t = [torch.from_numpy(x).to(DEV) for x in (self.kc, self.vc, self.ks8, self.vs8)]
        return [t[0].view(CODES), t[1].view(CODES), t[2].view(SCALES), t[3].view(SCALES)]

    def values(self):
        return oracle.values(self.kc, self.ks8, self.block), oracle.values(self.vc, self.vs8, self.block)

    def attend(self, q=None, caches=None, **kw):
        kc, vc, ks, vs = caches or self.caches()
        table, length, cu = self.index_args()
        return sdv.attend(self.q.to(DEV) if q is None else q, kc, vc, table, length, cu, key_scales=ks, value_scales=vs,
                          parents=self.tree_arg(), **kw)

    def append(self, caches, f=None, **kw):
        kc, vc, ks, vs = caches
        table, length, cu = self.index_args()
        return sdv.kv_append(kw.pop("k", self.k.to(DEV)), kw.pop("v", self.v.to(DEV)), kc, vc, table, length, cu, key_scales=ks,
                             value_scales=vs, parents=self.tree_arg(), inv_freq=f, **kw)


def host(t):
    """Codes or scales as bytes on the host."""
    return t.view(torch.uint8).cpu().numpy()
