"""The paged cache in 8 bits, and its pages from the requests' lengths, as cases that can be timed.

Four operators: appending rotated keys and values to a cache of e4m3 codes with a power-of-two scale for
each block of tokens and head ("append8"), attention of a ragged batch's rows over that cache
("attend8"), moving a verified tree's accepted path in it ("settle8"), and page tables and slot maps
made on the GPU from the requests' lengths ("pages").

run() computes an operator in elementary torch operations, or through the package's entry points
when `own` is true.  exact() computes the same from the definition in 64 bits.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CODES = torch.float8_e4m3fn
SCALES = torch.float8_e8m0fnu


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one request's drafts enter a small model's cache: latency counts
        dict(name="append8_b1", op="append8", B=1, K=4, ragged=False, tree=False, ctx=1000, Hq=16, Hkv=2, D=128, page=16,
             block=16, dtype="bf16", style="half", rotary=128),
        # a verification round of 256 requests, K in 0..8: rotate queries and keys, append both
        dict(name="append8_b256_k8", op="append8", B=256, K=8, ragged=True, tree=False, ctx=2048, Hq=32, Hkv=8, D=128,
             page=16, block=16, dtype="bf16", style="half", rotary=128),
        # prompts of four requests entering the cache in one call, odd lengths, far positions
        dict(name="append8_prompt", op="append8", B=4, K=4096, ragged=True, tree=False, ctx=65536, Hq=16, Hkv=2, D=128,
             page=64, block=32, dtype="bf16", style="interleaved", rotary=64),
        # one request, one token, short cache: latency
        dict(name="attend8_b1", op="attend8", B=1, K=0, ragged=False, tree=False, ctx=1000, Hq=16, Hkv=2, D=128, page=16,
             block=16, dtype="bf16", window=512, sinks=4),
        # the verification forward of 64 requests with long caches, K in 0..8, window and sinks
        dict(name="attend8_b64_k8", op="attend8", B=64, K=8, ragged=True, tree=False, ctx=8192, Hq=32, Hkv=8, D=128,
             page=16, block=16, dtype="bf16", window=4096, sinks=4),
        # few requests with very long caches, each token read
        dict(name="attend8_long", op="attend8", B=3, K=3, ragged=True, tree=False, ctx=131072, Hq=32, Hkv=8, D=128,
             page=128, block=64, dtype="bf16", window=0, sinks=0),
        # token trees with binary32 rows
        dict(name="attend8_tree_fp32", op="attend8", B=16, K=24, ragged=True, tree=True, ctx=2048, Hq=8, Hkv=2, D=64,
             page=32, block=8, dtype="fp32", window=1024, sinks=8),
        # prompts: many rows per request, products bound the call
        dict(name="attend8_prompt", op="attend8", B=2, K=2500, ragged=True, tree=False, ctx=700, Hq=32, Hkv=8, D=128,
             page=64, block=32, dtype="bf16", window=1024, sinks=4),
        # accepted paths of 64 token trees settle in four layers' caches
        dict(name="settle8_b64", op="settle8", B=64, K=24, ragged=True, tree=True, ctx=2048, Hkv=8, D=128, page=16,
             block=16, dtype="bf16", layers=4),
        # one request's tree in one layer: latency
        dict(name="settle8_b1", op="settle8", B=1, K=12, ragged=False, tree=True, ctx=500, Hkv=2, D=64, page=16, block=4,
             dtype="bf16", layers=1),
        # one request's pages for a round, then for the next: latency
        dict(name="pages_b1", op="pages", B=1, K=4, ragged=False, ctx=1000, page=16, window=0, sinks=0, closing=False),
        # 512 requests with long tables under a window, some of them ending
        dict(name="pages_b512", op="pages", B=512, K=64, ragged=True, ctx=65536, page=16, window=4096, sinks=4,
             closing=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append8", "append8", "attend8", "attend8", "attend8", "settle8", "pages"])
    page = rng.choice([1, 16, 16, 32, 64, 128])
    if op == "pages":
        return dict(op=op, B=_log_int(rng, 1, 512), K=_log_int(rng, 1, 64) if rng.random() < 0.7 else _log_int(rng, 64, 2000),
                    ragged=rng.random() < 0.7, ctx=_log_int(rng, 1, 65536 if page >= 16 else 4096), page=page,
                    window=rng.choice([0, 64, 1000, 4096]), sinks=rng.choice([0, 1, 4, 30]), closing=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    block = 2 ** rng.randint(0, int(math.log2(min(page, 64))))
    case = dict(op=op, Hkv=Hkv, D=D, page=page, block=block, dtype=dtype)
    if op == "settle8":
        return dict(case, B=_log_int(rng, 1, 64), K=_log_int(rng, 1, 64), ragged=rng.random() < 0.7, tree=True,
                    ctx=_log_int(rng, 1, 2048), layers=rng.choice([1, 2, 4]))
    case["Hq"] = Hkv * rng.choice([1, 2, 4, 5, 7, 8])
    tree = rng.random() < 0.3
    if not tree and rng.random() < 0.3:  # prompts
        case.update(B=_log_int(rng, 1, 4), K=_log_int(rng, 100, 1500), ctx=_log_int(rng, 1, 1024))
    else:
        case.update(B=_log_int(rng, 1, 64), K=rng.randint(0, 24) if tree else rng.randint(0, 12),
                    ctx=_log_int(rng, 1, 4096))
    case.update(ragged=rng.random() < 0.7, tree=tree)
    if op == "append8":
        case.update(style=rng.choice(["half", "interleaved"]), rotary=rng.choice([D, D // 2]))
    else:
        case.update(window=rng.choice([0, 64, 1000, 4096]), sinks=rng.choice([0, 1, 4, 30]))
    return case


def _layout(case):
    """Depths K_i and cached lengths of a case's requests: fixed by the case, so that its work is."""
    rng = random.Random(case["B"] * 1000003 + case["K"] * 1009 + case["ctx"])
    ks, lens = [], []
    for i in range(case["B"]):
        k = case["K"]
        if case["ragged"]:
            k = rng.randint(k // 2, k) if k > 64 else rng.randint(0, k)
        ks.append(k)
        lens.append(rng.randint((case["ctx"] + 1) // 2, case["ctx"]) if case["ragged"] else case["ctx"])
    if case["ragged"] and case["ctx"] >= 1 and case["B"] > 2 and case["op"] != "settle8":
        lens[1] = 0  # a request whose cache is still empty
    return ks, lens


# ------------------------------------------------------------------------------------------ inputs

def _random_tree(rng, K):
    parents = []
    for n in range(K):
        parents.append(rng.choice([n - 1, rng.randint(-1, n - 1)]))
    return parents


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _sums(ks):
    offsets = [0]
    for k in ks:
        offsets.append(offsets[-1] + k)
    return offsets


def _cache_state(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    ks, lens = _layout(case)
    B, ps, Hkv, D = case["B"], case["page"], case["Hkv"], case["D"]
    need = [-(-(n + k + 1) // ps) for n, k in zip(lens, ks)]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((B, max(need) + 1), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    window, sinks = case.get("window", 0), case.get("sinks", 0)
    if window:  # pages that left the window are free again, as in a serving engine
        for i, n in enumerate(lens):
            lo, hi = -(-sinks // ps), (n - window + 1) // ps
            if hi > lo:
                table[i, lo:hi] = -1
    offsets = _sums(ks)
    layers = (case["layers"],) if case["op"] == "settle8" else ()

    def codes():  # values of about 1 under the scales below
        x = torch.randn(layers + (n_pages, Hkv, ps, D), generator=g, device=DEVICE, dtype=torch.bfloat16)
        return x.mul_(120.0).clamp_(-448.0, 448.0).to(CODES)

    def scales():  # 2^-8 to 2^-6
        shape = layers + (n_pages, Hkv, ps // case["block"])
        return torch.randint(119, 122, shape, generator=g, device=DEVICE, dtype=torch.uint8).view(SCALES)

    s = dict(case=case, ks=ks, lens=lens, key_cache=codes(), value_cache=codes(), key_scales=scales(),
             value_scales=scales(), page_table=table, cache_len=_int32(lens), offsets=_int32(offsets), parents=None)
    if case["tree"]:
        trees = [_random_tree(rng, k) for k in ks]
        s["parents"] = _int32([p for t in trees for p in t])
        if case["op"] == "settle8":
            acc, nodes = [], []
            for t in trees:
                path, here = [], -1
                while True:
                    kids = [n for n, p in enumerate(t) if p == here]
                    if not kids or (path and rng.random() < 0.15):
                        break
                    here = rng.choice(kids)
                    path.append(here)
                acc.append(len(path))
                nodes += path + [-1] * (len(t) - len(path))
            s["accepted_len"], s["accepted_nodes"] = _int32(acc), _int32(nodes)
    rows = offsets[-1] + B
    if case["op"] == "append8":
        # one fused projection's output, as a model's layer leaves it; tokens of different size
        Hq = case["Hq"]
        size = torch.exp2(torch.randn((rows, 1, 1), generator=g, device=DEVICE))
        qkv = (torch.randn((rows, Hq + 2 * Hkv, D), generator=g, device=DEVICE) * size).to(dt)
        s["queries"], s["keys"], s["values"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        half = case["rotary"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, device=DEVICE, dtype=torch.float64) / half)).float()
    if case["op"] == "attend8":
        s["queries"] = torch.randn((rows, case["Hq"], D), generator=g, device=DEVICE, dtype=dt)
    return s


def _pages_state(case, seed):
    """Tables that hold what the cached tokens need; a round's lengths, and those of the round after it."""
    rng = random.Random(seed)
    ks, lens = _layout(case)
    B, ps, window = case["B"], case["page"], case["window"]
    acc = [rng.randint(0, k) for k in ks]
    next_lens = [n + 1 + a for n, a in zip(lens, acc)]
    if case["closing"]:
        for i in range(B):
            if rng.random() < 0.1 or i == 0:
                next_lens[i] = -1  # this request ends
    wide = max(n + 2 * k + 2 for n, k in zip(lens, ks))
    width = -(-wide // ps) + 1
    held = []
    for n in lens:
        lo = max(0, n - window + 1) // ps if window else 0
        near = -(-min(case["sinks"], n) // ps) if window else 0
        held.append([k for k in range(-(-n // ps)) if k >= lo or k < near])
    spare = sum(k // ps + 2 for k in ks)
    n_pages = sum(len(h) for h in held) + spare + 5
    order = list(range(n_pages))
    rng.shuffle(order)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for i, h in enumerate(held):
        table[i, h] = torch.tensor(order[at:at + len(h)], dtype=torch.int32)
        at += len(h)
    rest = order[at:]
    first = rng.randrange(n_pages)
    ring = [0] * n_pages
    for x, p in enumerate(rest):
        ring[(first + x) % n_pages] = p
    n_d = sum(ks)
    return dict(case=case, n_d=n_d, page_table=table.to(DEVICE), free_pages=_int32(ring),
                free_state=_int32([first, len(rest)]), offsets=_int32(_sums(ks)),
                cache_len=_int32(lens), next_len=_int32(next_lens))


def prepare(case, seed):
    return _pages_state(case, seed) if case["op"] == "pages" else _cache_state(case, seed)


# ------------------------------------------------------------------------------------ plain forms

def _rows_of(s, rows):
    """Each row's request and its index j within it."""
    B = s["cache_len"].shape[0]
    starts = s["offsets"].long() + torch.arange(B + 1, device=DEVICE)
    req = torch.searchsorted(starts, torch.arange(rows, device=DEVICE), right=True) - 1
    return req, torch.arange(rows, device=DEVICE) - starts[req]


def _twice(a):
    return ((a @ a) > 0).float()


def _ancestors(s, R):
    """[B, R, R]: row a's token is row b's, or one of its ancestors' (row 0 the last committed token)."""
    B = s["cache_len"].shape[0]
    if s["parents"] is None:
        return torch.ones(R, R, device=DEVICE).tril().bool().expand(B, R, R)
    n = s["parents"].shape[0]
    starts = s["offsets"].long()
    req = torch.searchsorted(starts, torch.arange(n, device=DEVICE), right=True) - 1
    j = torch.arange(n, device=DEVICE) - starts[req] + 1
    a = torch.eye(R, device=DEVICE).repeat(B, 1, 1)
    a[req, j, s["parents"].long() + 1] = 1.0
    return _twice(_twice(_twice(_twice(_twice(_twice(_twice(a))))))).bool()


def _places(s, req, slot):
    ps = s["case"]["page"]
    return s["page_table"][req, slot // ps].long(), slot % ps


def _exponents(scales):
    return scales.view(torch.uint8).int() - 127


def _rotate(x, angle, style, rotary):
    """x [rows, H, D] in 32 bits, turned by angle [rows, rotary / 2] (64 bits) in its first values."""
    c, n = angle.cos().float()[:, None], angle.sin().float()[:, None]
    turn, rest = x[..., :rotary], x[..., rotary:]
    if style == "half":
        a, b = turn[..., : rotary // 2], turn[..., rotary // 2:]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = turn[..., ::2], turn[..., 1::2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _least_exponent(top, limit):
    """The least e in [-117, 119] with top <= limit 2^e."""
    m, x = torch.frexp(top.double() / limit)  # m in [0.5, 1)
    e = torch.where(m > 0.5, x, x - 1)
    return torch.where(top > 0, e, -117).clamp(-117, 119)


def _put8(s, name, x, limit, top, req, j):
    """Rows x [rows, H, D] (32 bits) into a cache of codes: `top` [rows, H] the largest of each before rotation."""
    case, cache, scales = s["case"], s[name + "_cache"], s[name + "_scales"]
    n_pages, H, ps, D = cache.shape
    block = case["block"]
    bytes_, sbytes = cache.view(torch.uint8), scales.view(torch.uint8)
    n = s["cache_len"].long()[req]
    slot = n + j
    page, at = _places(s, req, slot)
    heads = torch.arange(H, device=DEVICE)
    # the largest of the new rows in each block, at the block's place among all
    which = ((page * (ps // block) + at // block)[:, None] * H + heads).flatten()
    largest = torch.zeros(n_pages * (ps // block) * H, device=DEVICE).scatter_reduce_(0, which, top.flatten(), "amax")
    e = _least_exponent(largest[which].view(-1, H), limit)
    old = _exponents(scales)[page[:, None], heads, (at // block)[:, None]]
    first = slot // block * block  # the block's first slot
    e = torch.where((first < n)[:, None], torch.maximum(e, old), e)
    # cached tokens of the blocks that were begun before
    lead = torch.nonzero((j == 0) & (first < n))[:, 0]
    if lead.numel():
        r, f = req[lead], first[lead]
        p, a = _places(s, r, f)
        span = a[:, None] + torch.arange(block, device=DEVICE)
        held = cache[p].float().gather(2, span[:, None, :, None].expand(-1, H, -1, D))
        held = torch.ldexp(held, (old[lead] - e[lead])[:, :, None, None]).to(CODES).view(torch.uint8)
        live = (f[:, None] + torch.arange(block, device=DEVICE)) < n[lead][:, None]
        who, which_token = torch.nonzero(live, as_tuple=True)
        bytes_[p[who], :, span[who, which_token]] = held[who, :, which_token]
    codes = torch.ldexp(x, -e[:, :, None]).clamp(-448.0, 448.0).to(CODES)
    bytes_[page, :, at] = codes.view(torch.uint8)
    sbytes[page[:, None], heads, (at // block)[:, None]] = (e + 127).to(torch.uint8)


def _plain_append8(s):
    case, rows = s["case"], s["keys"].shape[0]
    req, j = _rows_of(s, rows)
    depth = j
    if s["parents"] is not None:
        depth = (_ancestors(s, case["K"] + 1).sum(-1) - 1)[req, j]
    n = s["cache_len"].long()[req]
    angle = (n + depth).double()[:, None] * s["inv_freq"].double()  # far positions need 64 bits
    k, v = s["keys"].float(), s["values"].float()
    _put8(s, "key", _rotate(k, angle, case["style"], case["rotary"]), 316.0, k.abs().amax(-1), req, j)
    _put8(s, "value", v, 448.0, v.abs().amax(-1), req, j)
    q = _rotate(s["queries"].float(), angle, case["style"], case["rotary"]).to(s["queries"].dtype)
    return [q, s["key_cache"], s["value_cache"], s["key_scales"], s["value_scales"]]


def _plain_attend8(s):
    case = s["case"]
    rows, Hq, D = s["queries"].shape
    B, Hkv, ps, R = case["B"], case["Hkv"], case["page"], case["K"] + 1
    G = Hq // Hkv
    req, j = _rows_of(s, rows)
    q = torch.zeros(B, R, Hq, D, device=DEVICE)
    q[req, j] = s["queries"].float()
    q = q.view(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    table = s["page_table"].long()
    S = table.shape[1] * ps

    def values(cache, scales):
        x = cache.view(torch.uint8)[table.clamp(min=0)].view(CODES).float()  # [B, pages, H, ps, D]
        f = scales.view(torch.uint8)[table.clamp(min=0)].view(SCALES).float()
        x = x.view(*x.shape[:3], -1, case["block"], D) * f[..., None, None]
        return x.view(B, -1, Hkv, ps, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, S, D)

    k, v = values(s["key_cache"], s["key_scales"]), values(s["value_cache"], s["value_scales"])
    n = s["cache_len"].long()[:, None]
    slot = torch.arange(S, device=DEVICE)[None]
    node = slot - n  # row index of a slot behind the cached ones
    anc = _ancestors(s, R)
    depth = anc.sum(-1) - 1
    inside = (node >= 0) & (node < R)
    at = node.clamp(0, R - 1)
    pos = torch.where(inside, n + depth.gather(1, at), slot)
    see = torch.where(inside[:, None], anc.gather(2, at[:, None].expand(B, R, S)), (slot < n)[:, None])
    if case["window"]:
        near = (n + depth)[:, :, None] - pos[:, None] < case["window"]
        see = see & (near | (slot < case["sinks"])[:, None])
    see = see & (table >= 0).repeat_interleave(ps, 1)[:, None]
    x = (q @ k.transpose(2, 3).contiguous()).view(B, Hkv, R, G, S) / math.sqrt(D)
    x = x.masked_fill(~see[:, None, :, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    p = (p / p.sum(-1, keepdim=True)).nan_to_num(0.0).view(B, Hkv, R * G, S)
    o = (p @ v).view(B, Hkv, R, G, D).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D)
    return [o[req, j].to(s["queries"].dtype)]


def _settle8(s, name, req, d, src, dst):
    """Accepted tokens (request, number d, slots from and to) of all layers of one cache of codes."""
    cache, scales = s[name + "_cache"], s[name + "_scales"]
    layers, n_pages, H, ps, D = cache.shape
    block = s["case"]["block"]
    bytes_, sbytes = cache.view(torch.uint8), scales.view(torch.uint8)
    n = s["cache_len"].long()[req]
    sp, so = _places(s, req, src)
    dp, do = _places(s, req, dst)
    e = _exponents(scales)
    mine = e[:, sp, :, so // block]  # [tokens, layers, H]
    old = e[:, dp, :, do // block]
    first = dst // block * block
    begun = first <= n  # the block holds tokens that were there before
    where = dp * (ps // block) + do // block
    most = torch.full((n_pages * (ps // block), layers, H), -128, dtype=torch.int32, device=DEVICE)
    most.scatter_reduce_(0, where[:, None, None].expand_as(mine), mine, "amax")
    new = torch.where(begun[:, None, None], torch.maximum(most[where], old), most[where])
    moved = torch.ldexp(cache.view(torch.uint8)[:, sp, :, so].view(CODES).float(), (mine - new)[..., None])
    moved = moved.to(CODES).view(torch.uint8)
    lead = torch.nonzero((d == 0) & begun)[:, 0]  # cached tokens, row 0's among them
    p, a = dp[lead], first[lead] % ps
    span = a[:, None] + torch.arange(block, device=DEVICE)
    live = first[lead][:, None] + torch.arange(block, device=DEVICE) <= n[lead][:, None]
    who, t = torch.nonzero(live, as_tuple=True)
    held = bytes_[:, p[who], :, span[who, t]].view(CODES).float()
    held = torch.ldexp(held, (old - new)[lead][who][..., None]).to(CODES).view(torch.uint8)
    bytes_[:, p[who], :, span[who, t]] = held
    bytes_[:, dp, :, do] = moved
    sbytes[:, dp, :, do // block] = (new + 127).to(torch.uint8)


def _plain_settle8(s):
    nodes = s["accepted_nodes"].long()
    starts = s["offsets"].long()
    i = torch.arange(nodes.shape[0], device=DEVICE)
    req = torch.searchsorted(starts, i, right=True) - 1
    kept = nodes >= 0
    n = s["cache_len"].long()[req] + 1
    d = i - starts[req]
    for name in ("key", "value"):
        _settle8(s, name, req[kept], d[kept], (n + nodes)[kept], (n + d)[kept])
    return [s["cache_len"] + 1 + s["accepted_len"], s["key_cache"], s["value_cache"], s["key_scales"], s["value_scales"]]


def _plain_round(s, cache_len):
    """One call's pages: the table, the ring of free pages and its state in place; (placed, slots)."""
    case, table, ring, state = s["case"], s["page_table"], s["free_pages"], s["free_state"]
    ps, (B, width), n_pages = case["page"], table.shape, ring.shape[0]
    L = cache_len.long()
    K = (s["offsets"][1:] - s["offsets"][:-1]).long()
    k = torch.arange(width, device=DEVICE)[None]
    last = ((L + K) // ps)[:, None]
    keep = k <= last
    if case["window"]:
        low = (L - case["window"] + 1).clamp(min=0) // ps
        keep &= (k >= low[:, None]) | (k * ps < case["sinks"])
    opened = L >= 0
    keep &= opened[:, None]
    have = (table >= 0) & (table < n_pages)
    freed = have & ~keep
    fits = opened & (last[:, 0] < width)
    want = (k >= (L // ps)[:, None]) & (k <= last) & ~have & fits[:, None]
    d = want.sum(1)
    first, count = state[0].long(), state[1].long()
    placed = fits & ((d == 0) | (d.cumsum(0) <= count))
    want &= placed[:, None]
    rank = want.flatten().long().cumsum(0).view(B, width) - 1
    taken = ring[(first + rank.clamp(min=0)) % n_pages]
    back = table[freed]
    ring[(first + count + torch.arange(back.shape[0], device=DEVICE)) % n_pages] = back
    table.copy_(torch.where(want, taken, torch.where(freed, -1, table)))
    used = want.sum()
    state.copy_(torch.stack([(first + used) % n_pages, count - used + back.shape[0]]))
    req, j = _rows_of(s, s["n_d"] + B)
    slot = (L[req] + j).clamp(min=0)
    page = table[req, (slot // ps).clamp(max=width - 1)].long()
    return placed.int(), torch.where(placed[req], page * ps + slot % ps, -1)


def _plain_pages(s):
    placed, slots = _plain_round(s, s["cache_len"])
    placed_next, slots_next = _plain_round(s, s["next_len"])
    return [placed, slots, placed_next, slots_next, s["page_table"], s["free_pages"], s["free_state"]]


# --------------------------------------------------------------------------- the package's calls

def _own_append8(s):
    import lossless_draft_verification_online_amd as sdv

    q = sdv.kv_append(s["keys"], s["values"], s["key_cache"], s["value_cache"], s["page_table"], s["cache_len"],
                      s["offsets"], key_scales=s["key_scales"], value_scales=s["value_scales"], parents=s["parents"],
                      inv_freq=s["inv_freq"], interleaved=s["case"]["style"] == "interleaved", queries=s["queries"])
    return [q, s["key_cache"], s["value_cache"], s["key_scales"], s["value_scales"]]


def _own_attend8(s):
    import lossless_draft_verification_online_amd as sdv

    return [sdv.attend(s["queries"], s["key_cache"], s["value_cache"], s["page_table"], s["cache_len"], s["offsets"],
                       key_scales=s["key_scales"], value_scales=s["value_scales"], parents=s["parents"],
                       window=s["case"]["window"], sinks=s["case"]["sinks"])]


def _own_settle8(s):
    import lossless_draft_verification_online_amd as sdv

    length = sdv.kv_settle(s["key_cache"], s["value_cache"], s["page_table"], s["cache_len"], s["offsets"],
                           s["accepted_len"], s["accepted_nodes"], key_scales=s["key_scales"],
                           value_scales=s["value_scales"])
    return [length, s["key_cache"], s["value_cache"], s["key_scales"], s["value_scales"]]


def _own_pages(s):
    import lossless_draft_verification_online_amd as sdv

    got = []
    for length in (s["cache_len"], s["next_len"]):
        got += sdv.kv_pages(s["page_table"], length, s["offsets"], s["n_d"], s["free_pages"], s["free_state"],
                            s["case"]["page"], window=s["case"]["window"], sinks=s["case"]["sinks"])
    return got + [s["page_table"], s["free_pages"], s["free_state"]]


PLAIN = {"append8": _plain_append8, "attend8": _plain_attend8, "settle8": _plain_settle8, "pages": _plain_pages}
OWN = {"append8": _own_append8, "attend8": _own_attend8, "settle8": _own_settle8, "pages": _own_pages}


def run(state):
    if own:
        return OWN[state["case"]["op"]](state)
    return PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------------------------------- work

def _visible(case):
    """(query-slot pairs of one head, slots any row of a request sees) summed over the requests of a
    linear batch; a tree's rows are counted as a chain of half their number."""
    pairs = slots = 0
    window, sinks = case["window"], case["sinks"]
    ks, lens = _layout(case)
    for k, n in zip(ks, lens):
        chain = k // 2 if case["tree"] else k
        for j in range(k + 1):
            at = n + min(j, chain)
            pairs += at + 1 if not window else min(at + 1, window) + min(sinks, max(0, at + 1 - window))
        low = max(0, n + 1 - window) if window else 0
        slots += n + k + 1 - low + min(sinks, low)
    return pairs, slots


def work(case):
    ks, lens = _layout(case)
    rows = sum(ks) + case["B"]
    if case["op"] == "pages":
        wide = max(n + 2 * k + 2 for n, k in zip(lens, ks))
        entries = case["B"] * -(-wide // case["page"])
        return {"bytes": 2 * (4 * entries + 8 * rows), "flops": 0}  # two calls
    size = DTYPES[case["dtype"]].itemsize
    line = case["Hkv"] * case["D"]  # bytes of a token's keys, or values, in the cache
    if case["op"] == "append8":
        qline = case["Hq"] * case["D"] * size
        return {"bytes": rows * (2 * line * (size + 1) + 2 * qline),
                "flops": 3 * rows * (case["Hq"] + case["Hkv"]) * case["rotary"]}
    if case["op"] == "settle8":
        moved = sum(k / 3 for k in ks)  # about a third of a tree's nodes lie on the accepted path
        return {"bytes": max(1, moved) * case["layers"] * 4 * line, "flops": 0}
    pairs, slots = _visible(case)
    return {"bytes": 2 * slots * (line + case["Hkv"] / case["block"]) + 2 * rows * case["Hq"] * case["D"] * size,
            "flops": 4 * pairs * case["Hq"] * case["D"]}


# ------------------------------------------------------------------------------------------- exact

def _depths(parents):
    depth = []
    for p in parents:
        depth.append(1 if p < 0 else depth[p] + 1)
    return [0] + depth


def _exact_requests(s):
    """Per request: its first row, cached length, row depths and per-row lists of visible rows."""
    parents = None if s["parents"] is None else s["parents"].tolist()
    row = at = 0
    for i, (k, n) in enumerate(zip(s["ks"], s["lens"])):
        if parents is None:
            yield i, row, n, list(range(k + 1)), None
        else:
            tree = parents[at:at + k]
            see = [[0]]
            for m, p in enumerate(tree):
                see.append(see[p + 1] + [m + 1])
            yield i, row, n, _depths(tree), see
        row, at = row + k + 1, at + k


def _exact_turn(x, pos, freq, case):
    """Complex multiplication of the pairs by e^(i pos f)."""
    x, half = x.double().clone(), case["rotary"] // 2
    first, second = (slice(0, half), slice(half, 2 * half)) if case["style"] == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    turn = torch.polar(torch.ones_like(freq)[None].expand(len(pos), half), torch.tensor(pos, device=DEVICE, dtype=torch.float64)[:, None] * freq)
    w = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn[:, None]
    x[..., first], x[..., second] = w.real, w.imag
    return x


def _nearest_code(x):
    """The e4m3 number next to x (ties to the even one), as a 64-bit number."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * torch.minimum(torch.round(a / step) * step, torch.full_like(a, 448.0))


def _exact_append8(s):
    case, ps, block = s["case"], s["case"]["page"], s["case"]["block"]
    freq = s["inv_freq"].double()
    q = torch.empty(s["queries"].shape, dtype=torch.float64, device=DEVICE)
    out = {}
    for name in ("key", "value"):
        out[name] = s[name + "_cache"].double(), s[name + "_scales"].double()
    table = s["page_table"].tolist()
    for i, row, n, depth, _ in _exact_requests(s):
        R = len(depth)
        pos = [n + d for d in depth]
        q[row:row + R] = _exact_turn(s["queries"][row:row + R], pos, freq, case)
        turned = {"key": _exact_turn(s["keys"][row:row + R], pos, freq, case), "value": s["values"][row:row + R].double()}
        raw = {"key": s["keys"][row:row + R].double(), "value": turned["value"]}
        for first in range(n // block * block, n + R, block):
            page, at = table[i][first // ps], first % ps
            lo, hi = max(n, first), min(n + R, first + block)
            for name, limit in (("key", 316.0), ("value", 448.0)):
                cache, scales = out[name]
                top = raw[name][lo - n:hi - n].abs().amax((0, 2))  # [H]
                scale = torch.exp2(torch.ceil(torch.log2(top / limit))).clamp(2.0 ** -117, 2.0 ** 119)
                scale = torch.where(top <= limit * scale / 2, scale / 2, scale).clamp(min=2.0 ** -117)
                if first < n:
                    was = scales[page, :, at // block]
                    scale = torch.maximum(scale, was)
                    held = cache[page, :, at:at + n - first]
                    cache[page, :, at:at + n - first] = _nearest_code(held * (was / scale)[:, None, None])
                new = turned[name][lo - n:hi - n].transpose(0, 1) / scale[:, None, None]
                cache[page, :, lo % ps:lo % ps + hi - lo] = _nearest_code(new)
                scales[page, :, at // block] = scale
    return [q, out["key"][0], out["value"][0], out["key"][1], out["value"][1]]


def _exact_attend8(s):
    case, ps, block = s["case"], s["case"]["page"], s["case"]["block"]
    rows, Hq, D = s["queries"].shape
    G = Hq // case["Hkv"]
    out = torch.zeros((rows, Hq, D), dtype=torch.float64, device=DEVICE)
    for i, row, n, depth, see in _exact_requests(s):
        R = len(depth)
        slots = torch.arange(n + R, device=DEVICE)
        pages = s["page_table"][i].long()[torch.div(slots, ps, rounding_mode="floor")]
        d = torch.tensor(depth, device=DEVICE)
        pos = torch.cat([slots[:n], n + d])
        ok = torch.zeros((R, n + R), dtype=torch.bool, device=DEVICE)
        ok[:, :n] = True
        if see is None:
            ok[:, n:] = torch.arange(R, device=DEVICE)[None] <= torch.arange(R, device=DEVICE)[:, None]
        else:
            for r, list_ in enumerate(see):
                ok[r, [n + a for a in list_]] = True
        if case["window"]:
            ok &= ((n + d)[:, None] - pos[None] < case["window"]) | (slots < case["sinks"])[None]
        ok &= (pages >= 0)[None]
        p, o, b = pages.clamp(min=0), slots % ps, slots % ps // block
        for h in range(case["Hkv"]):
            k = s["key_cache"].view(torch.uint8)[p, h, o].view(CODES).double() * s["key_scales"].view(torch.uint8)[p, h, b].view(SCALES).double()[:, None]
            v = s["value_cache"].view(torch.uint8)[p, h, o].view(CODES).double() * s["value_scales"].view(torch.uint8)[p, h, b].view(SCALES).double()[:, None]
            for g in range(h * G, h * G + G):
                x = (s["queries"][row:row + R, g].double() @ k.T) * D ** -0.5
                out[row:row + R, g] = torch.softmax(x.masked_fill(~ok, -math.inf), -1) @ v
    return [out]


def _exact_settle8(s):
    ps, block = s["case"]["page"], s["case"]["block"]
    acc, nodes = s["accepted_len"].tolist(), s["accepted_nodes"].tolist()
    table = s["page_table"].tolist()
    out = []
    for name in ("key", "value"):
        cache, scales = s[name + "_cache"].double(), s[name + "_scales"].double()
        start = 0
        for i, (k, n) in enumerate(zip(s["ks"], s["lens"])):
            path = nodes[start:start + acc[i]]
            start += k

            def slot(x, i=i):
                return table[i][x // ps], x % ps

            took = []  # each accepted token's codes and scale, before any of them moves
            for node in path:
                p, o = slot(n + 1 + node)
                took.append((cache[:, p, :, o].clone(), scales[:, p, :, o // block].clone()))
            for first in range((n + 1) // block * block, n + 1 + len(path), block):
                p, o = slot(first)
                inside = [d for d in range(len(path)) if first <= n + 1 + d < first + block]
                if not inside:
                    continue
                old = scales[:, p, :, o // block].clone()
                new = torch.stack([took[d][1] for d in inside] + ([old] if first <= n else [])).amax(0)
                for x in range(first, min(n + 1, first + block)):
                    cache[:, p, :, x % ps] = _nearest_code(cache[:, p, :, x % ps] * (old / new)[..., None])
                for d in inside:
                    cache[:, p, :, (n + 1 + d) % ps] = _nearest_code(took[d][0] * (took[d][1] / new)[..., None])
                scales[:, p, :, o // block] = new
        out.append((cache, scales))
    return [None, out[0][0], out[1][0], out[0][1], out[1][1]]


def exact(case, seed):
    if case["op"] == "pages":  # whole numbers
        return None
    s = prepare(case, seed)
    return {"append8": _exact_append8, "attend8": _exact_attend8, "settle8": _exact_settle8}[case["op"]](s)
