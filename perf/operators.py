"""The drafting and cache operators around the verification step, as cases that can be timed.

Four operators: sampling a drafter's tokens from its logits ("sample"), appending rotated keys and
values of a ragged batch to a paged cache ("append"), attention of the batch's rows over that cache
under a sliding window with visible first tokens ("attend"), and moving the accepted path of a
verified token tree to its contiguous place in the cache ("settle").

run() computes an operator in elementary torch operations, or through the package's entry points
when `own` is true.  exact() computes the same from the definition in 64 bits.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the repository's smallest workload's vocabulary: one request drafts one token; latency counts
        dict(name="sample_b1_v1000", op="sample", n=1, V=1000, dtype="fp32", profile="plain", probs=True),
        # a serving batch under full sampling profiles, q rows published for the verifier; padded rows
        dict(name="sample_b64_v32000", op="sample", n=64, V=32000, dtype="bf16", profile="mixed", probs=True, pad=64),
        # the headline batch's requests, plain temperature: the whole row counts
        dict(name="sample_b256_v128256", op="sample", n=256, V=128256, dtype="bf16", profile="plain", probs=False),
        # the widest vocabulary, nucleus sampling without top-k, q rows published
        dict(name="sample_b512_v151936", op="sample", n=512, V=151936, dtype="bf16", profile="nucleus", probs=True),
        # a verification round of 256 requests, K in 0..8: rotate queries and keys, append both
        dict(name="append_b256_k8", op="append", B=256, K=8, ragged=True, tree=False, ctx=8192, Hq=32, Hkv=8, D=128,
             page=16, dtype="bf16", style="half", rotary=128),
        # prompts of four requests entering the cache in one call, odd lengths, far positions
        dict(name="append_prompt", op="append", B=4, K=4096, ragged=True, tree=False, ctx=131072, Hq=16, Hkv=2, D=128,
             page=64, dtype="bf16", style="interleaved", rotary=64),
        # one request, one token, short cache: latency
        dict(name="attend_b1", op="attend", B=1, K=0, ragged=False, tree=False, ctx=1000, Hq=16, Hkv=2, D=128, page=16,
             dtype="bf16", window=512, sinks=4),
        # the verification forward of 64 requests with long caches, K in 0..8, window and sinks
        dict(name="attend_b64_k8", op="attend", B=64, K=8, ragged=True, tree=False, ctx=8192, Hq=32, Hkv=8, D=128,
             page=16, dtype="bf16", window=4096, sinks=4),
        # token trees in binary32
        dict(name="attend_tree_fp32", op="attend", B=16, K=24, ragged=True, tree=True, ctx=2048, Hq=8, Hkv=2, D=64,
             page=32, dtype="fp32", window=1024, sinks=8),
        # prompts: many rows per request, products bound the call
        dict(name="attend_prompt", op="attend", B=2, K=2500, ragged=True, tree=False, ctx=700, Hq=32, Hkv=8, D=128,
             page=64, dtype="bf16", window=1024, sinks=4),
        # accepted paths of 64 token trees settle in four layers' caches
        dict(name="settle_b64", op="settle", B=64, K=24, ragged=True, tree=True, ctx=2048, Hkv=8, D=128, page=16,
             dtype="bf16", layers=4),
        # one request's tree in one layer: latency
        dict(name="settle_b1", op="settle", B=1, K=12, ragged=False, tree=True, ctx=500, Hkv=2, D=64, page=16,
             dtype="fp32", layers=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "append", "attend", "attend", "settle"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "sample":
        V = _log_int(rng, 1000, 151936)
        n = _log_int(rng, 1, max(1, min(512, 40_000_000 // V)))
        return dict(op=op, n=n, V=V, dtype=dtype, profile=rng.choice(["plain", "mixed", "nucleus", "top_k"]),
                    probs=rng.random() < 0.5, pad=rng.choice([0, 0, 1, 7, 64]))
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([1, 16, 16, 32, 64, 128])
    case = dict(op=op, Hkv=Hkv, D=D, page=page, dtype=dtype)
    if op == "settle":
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
    if op == "append":
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
    if case["ragged"] and case["ctx"] >= 1 and case["B"] > 2 and case["op"] != "settle":
        lens[1] = 0  # a request whose cache is still empty
    return ks, lens


# ------------------------------------------------------------------------------------------ inputs

def _random_tree(rng, K):
    parents = []
    for n in range(K):
        parents.append(rng.choice([n - 1, rng.randint(-1, n - 1)]))
    return parents


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
    offsets = [0]
    for k in ks:
        offsets.append(offsets[-1] + k)
    shape = (n_pages, Hkv, ps, D)
    if case["op"] == "settle":
        shape = (case["layers"],) + shape
    s = dict(case=case, ks=ks, lens=lens,
             key_cache=torch.randn(shape, generator=g, device=DEVICE, dtype=dt),
             value_cache=torch.randn(shape, generator=g, device=DEVICE, dtype=dt),
             page_table=table, cache_len=torch.tensor(lens, dtype=torch.int32, device=DEVICE),
             offsets=torch.tensor(offsets, dtype=torch.int32, device=DEVICE), parents=None)
    if case["tree"]:
        trees = [_random_tree(rng, k) for k in ks]
        s["parents"] = torch.tensor([p for t in trees for p in t], dtype=torch.int32, device=DEVICE)
        if case["op"] == "settle":
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
            s["accepted_len"] = torch.tensor(acc, dtype=torch.int32, device=DEVICE)
            s["accepted_nodes"] = torch.tensor(nodes, dtype=torch.int32, device=DEVICE)
    rows = offsets[-1] + B
    if case["op"] == "append":
        # one fused projection's output, as a model's layer leaves it
        Hq = case["Hq"]
        qkv = torch.randn((rows, Hq + 2 * Hkv, D), generator=g, device=DEVICE, dtype=dt)
        s["queries"], s["keys"], s["values"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        half = case["rotary"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, device=DEVICE, dtype=torch.float64) / half)).float()
    if case["op"] == "attend":
        s["queries"] = torch.randn((rows, case["Hq"], D), generator=g, device=DEVICE, dtype=dt)
    return s


def _sample_state(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    n, V = case["n"], case["V"]
    rows = torch.randn((n, V + case.get("pad", 0)), generator=g, device=DEVICE) * 3.0
    logits = rows.to(DTYPES[case["dtype"]])[:, :V]
    f = lambda lo, hi: lo + (hi - lo) * torch.rand(n, generator=g, device=DEVICE)  # noqa: E731
    pick = lambda *v: torch.tensor(v, device=DEVICE)[torch.randint(len(v), (n,), generator=g, device=DEVICE)]  # noqa: E731
    s = dict(case=case, logits=logits, uniform=torch.rand(n, generator=g, device=DEVICE, dtype=torch.float64),
             temperature=f(0.6, 1.2), top_k=None, top_p_milli=None, min_p=None)
    kind = case["profile"]
    if kind in ("mixed", "top_k"):
        s["top_k"] = pick(0, 20, 50, 200).to(torch.int32) if kind == "mixed" else pick(1, 40, 64, 100).to(torch.int32)
    if kind in ("mixed", "nucleus"):
        s["top_p_milli"] = pick(800, 900, 950, 1000).to(torch.int32)
    if kind == "mixed":
        s["min_p"] = pick(0.0, 0.02, 0.1).to(torch.float32)
        s["temperature"] = torch.where(torch.rand(n, generator=g, device=DEVICE) < 0.1, 0.0, s["temperature"])
    return s


def prepare(case, seed):
    return _sample_state(case, seed) if case["op"] == "sample" else _cache_state(case, seed)


# ------------------------------------------------------------------------------------ plain forms

def _plain_sample(s):
    z, V = s["logits"].double(), s["logits"].shape[1]  # 64 bits: draws and cuts lie next to borders
    T = s["temperature"].double()[:, None]
    greedy = T == 0
    top, best = z.max(1, keepdim=True)
    first = (z == top).int().argmax(1, keepdim=True)  # ties go to the lowest index
    w = torch.exp((z - top) / torch.where(greedy, 1.0, T))
    ids = torch.arange(V, device=z.device)[None]
    if s["top_k"] is not None or s["top_p_milli"] is not None or s["min_p"] is not None:
        order = torch.sort(z, dim=1, descending=True, stable=True).indices
        ranked = w.gather(1, order)
        keep = torch.full_like(first, V)
        if s["top_k"] is not None:
            k = s["top_k"].long()[:, None]
            keep = torch.where((k == 0) | (k >= V), V, k)
        ranked = torch.where(ids < keep, ranked, 0.0)
        if s["top_p_milli"] is not None:
            p = s["top_p_milli"].double()[:, None]
            run_mass = ranked.cumsum(1)
            total = run_mass[:, -1:]
            short = (run_mass * 1000 < p * total).sum(1, keepdim=True) + 1
            keep = torch.where(p < 1000, torch.minimum(keep, short), keep)
        if s["min_p"] is not None:
            high = (ranked >= s["min_p"].double()[:, None]).sum(1, keepdim=True)
            keep = torch.minimum(keep, high)
        kept = torch.zeros_like(w, dtype=torch.bool).scatter_(1, order, ids < keep)
        w = torch.where(kept, w, 0.0)
        count = keep
    else:
        count = torch.full_like(first, V)
    w = torch.where(greedy, (ids == first).double(), w)
    count = torch.where(greedy, 1, count)
    c = w.cumsum(1)
    total = c[:, -1:]
    y = (c <= s["uniform"][:, None] * total).sum(1, keepdim=True)
    last = (ids * (w > 0)).amax(1, keepdim=True)
    y = torch.minimum(y, last)
    out = [y[:, 0].int(), (w.gather(1, y) / total)[:, 0].float(), count[:, 0].int()]
    if s["case"]["probs"]:
        out.append((w / total).float())
    return out


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


def _plain_append(s):
    case, rows = s["case"], s["keys"].shape[0]
    req, j = _rows_of(s, rows)
    depth = j
    if s["parents"] is not None:
        depth = (_ancestors(s, case["K"] + 1).sum(-1) - 1)[req, j]
    n = s["cache_len"].long()[req]
    angle = (n + depth).double()[:, None] * s["inv_freq"].double()  # far positions need 64 bits
    page, at = _places(s, req, n + j)
    k = _rotate(s["keys"].float(), angle, case["style"], case["rotary"])
    s["key_cache"][page, :, at] = k.to(s["key_cache"].dtype)
    s["value_cache"][page, :, at] = s["values"]
    q = _rotate(s["queries"].float(), angle, case["style"], case["rotary"]).to(s["queries"].dtype)
    return [q, s["key_cache"], s["value_cache"]]


def _plain_attend(s):
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
    k = s["key_cache"][table.clamp(min=0)].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, S, D)
    v = s["value_cache"][table.clamp(min=0)].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, S, D)
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
    x = (q @ k.transpose(2, 3)).view(B, Hkv, R, G, S) / math.sqrt(D)
    x = x.masked_fill(~see[:, None, :, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    p = (p / p.sum(-1, keepdim=True)).nan_to_num(0.0).view(B, Hkv, R * G, S)
    o = (p @ v).view(B, Hkv, R, G, D).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D)
    return [o[req, j].to(s["queries"].dtype)]


def _plain_settle(s):
    nodes = s["accepted_nodes"].long()
    starts = s["offsets"].long()
    e = torch.arange(nodes.shape[0], device=DEVICE)
    req = torch.searchsorted(starts, e, right=True) - 1
    n = s["cache_len"].long()[req] + 1
    moves = nodes >= 0
    req, src, dst = req[moves], (n + nodes)[moves], (n + e - starts[req])[moves]
    sp, so = _places(s, req, src)
    dp, do = _places(s, req, dst)
    s["key_cache"][:, dp, :, do] = s["key_cache"][:, sp, :, so]
    s["value_cache"][:, dp, :, do] = s["value_cache"][:, sp, :, so]
    return [s["cache_len"] + 1 + s["accepted_len"], s["key_cache"], s["value_cache"]]


# --------------------------------------------------------------------------- the package's calls

def _own_sample(s):
    import lossless_draft_verification_online_amd as sdv

    tokens, prob, extra = sdv.sample(s["logits"], s["uniform"], s["temperature"], top_k=s["top_k"],
                                     top_p_milli=s["top_p_milli"], min_p=s["min_p"], probs=s["case"]["probs"])
    return [tokens, prob, extra["kept_tokens"]] + ([extra["probs"]] if s["case"]["probs"] else [])


def _own_append(s):
    import lossless_draft_verification_online_amd as sdv

    q = sdv.kv_append(s["keys"], s["values"], s["key_cache"], s["value_cache"], s["page_table"], s["cache_len"],
                      s["offsets"], parents=s["parents"], inv_freq=s["inv_freq"],
                      interleaved=s["case"]["style"] == "interleaved", queries=s["queries"])
    return [q, s["key_cache"], s["value_cache"]]


def _own_attend(s):
    import lossless_draft_verification_online_amd as sdv

    return [sdv.attend(s["queries"], s["key_cache"], s["value_cache"], s["page_table"], s["cache_len"], s["offsets"],
                       parents=s["parents"], window=s["case"]["window"], sinks=s["case"]["sinks"])]


def _own_settle(s):
    import lossless_draft_verification_online_amd as sdv

    length = sdv.kv_settle(s["key_cache"], s["value_cache"], s["page_table"], s["cache_len"], s["offsets"],
                           s["accepted_len"], s["accepted_nodes"])
    return [length, s["key_cache"], s["value_cache"]]


PLAIN = {"sample": _plain_sample, "append": _plain_append, "attend": _plain_attend, "settle": _plain_settle}
OWN = {"sample": _own_sample, "append": _own_append, "attend": _own_attend, "settle": _own_settle}


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
    size = DTYPES[case["dtype"]].itemsize
    if case["op"] == "sample":
        cells = case["n"] * case["V"]
        return {"bytes": cells * (size + (4 if case["probs"] else 0)), "flops": 4 * cells}
    ks, lens = _layout(case)
    rows = sum(ks) + case["B"]
    line = case["Hkv"] * case["D"] * size
    if case["op"] == "append":
        qline = case["Hq"] * case["D"] * size
        return {"bytes": rows * (4 * line + 2 * qline), "flops": 3 * rows * (case["Hq"] + case["Hkv"]) * case["rotary"]}
    if case["op"] == "settle":
        moved = sum(k / 3 for k in ks)  # about a third of a tree's nodes lie on the accepted path
        return {"bytes": max(1, moved) * case["layers"] * 4 * line, "flops": 0}
    pairs, slots = _visible(case)
    return {"bytes": 2 * slots * line + 2 * rows * case["Hq"] * case["D"] * size,
            "flops": 4 * pairs * case["Hq"] * case["D"]}


# ------------------------------------------------------------------------------------------- exact

def _exact_sample(s):
    n, V = s["logits"].shape
    prob = torch.zeros(n, dtype=torch.float64, device=DEVICE)
    probs = torch.zeros((n, V), dtype=torch.float64, device=DEVICE) if s["case"]["probs"] else None
    host = {k: (None if s[k] is None else s[k].tolist()) for k in ("temperature", "top_k", "top_p_milli", "min_p", "uniform")}
    for r in range(n):
        z = s["logits"][r].double()
        T = host["temperature"][r]
        if T == 0:
            y = int(torch.nonzero(z == z.max())[0])
            prob[r] = 1.0
            if probs is not None:
                probs[r, y] = 1.0
            continue
        e = (z - z.max()) / T
        value, index = torch.sort(e, descending=True, stable=True)
        end = V
        if host["top_k"] is not None and 0 < host["top_k"][r] < V:
            end = host["top_k"][r]
        if host["top_p_milli"] is not None and host["top_p_milli"][r] < 1000:
            m = torch.softmax(value[:end], 0).cumsum(0)
            end = int(torch.searchsorted(m, torch.tensor([host["top_p_milli"][r] / 1000.0], device=DEVICE,
                                                         dtype=torch.float64))[0].clamp(max=end - 1)) + 1
        if host["min_p"] is not None and host["min_p"][r] > 0:
            end = min(end, int((value >= math.log(host["min_p"][r])).sum()))
        p = torch.zeros(V, dtype=torch.float64, device=DEVICE)
        p[index[:end]] = torch.softmax(value[:end], 0)
        c = p.cumsum(0)
        y = int((c <= host["uniform"][r]).sum().clamp(max=V - 1))
        prob[r] = p[y]
        if probs is not None:
            probs[r] = p
    return [None, prob, None] + ([probs] if probs is not None else [])


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


def _exact_append(s):
    case, ps = s["case"], s["case"]["page"]
    key, value = s["key_cache"].double(), s["value_cache"].double()
    q = torch.empty(s["queries"].shape, dtype=torch.float64, device=DEVICE)
    freq = s["inv_freq"].double()
    for i, row, n, depth, _ in _exact_requests(s):
        rows = slice(row, row + len(depth))
        pos = [n + d for d in depth]
        q[rows] = _exact_turn(s["queries"][rows], pos, freq, case)
        slots = torch.arange(n, n + len(depth), device=DEVICE)
        pages = s["page_table"][i].long()[torch.div(slots, ps, rounding_mode="floor")]
        key[pages, :, slots % ps] = _exact_turn(s["keys"][rows], pos, freq, case)
        value[pages, :, slots % ps] = s["values"][rows].double()
    return [q, key, value]


def _exact_attend(s):
    case, ps = s["case"], s["case"]["page"]
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
        for h in range(case["Hkv"]):
            k = s["key_cache"][pages.clamp(min=0), h, slots % ps].double()
            v = s["value_cache"][pages.clamp(min=0), h, slots % ps].double()
            for g in range(h * G, h * G + G):
                x = (s["queries"][row:row + R, g].double() @ k.T) * D ** -0.5
                out[row:row + R, g] = torch.softmax(x.masked_fill(~ok, -math.inf), -1) @ v
    return [out]


def _exact_settle(s):
    ps = s["case"]["page"]
    key, value = s["key_cache"].double(), s["value_cache"].double()
    acc, nodes = s["accepted_len"].tolist(), s["accepted_nodes"].tolist()
    table = s["page_table"].tolist()
    at = 0
    for i, (k, n) in enumerate(zip(s["ks"], s["lens"])):
        for d, node in enumerate(nodes[at:at + acc[i]]):  # ascending: a source is never overwritten early
            to, frm = n + 1 + d, n + 1 + node
            for cache in (key, value):
                cache[:, table[i][to // ps], :, to % ps] = cache[:, table[i][frm // ps], :, frm % ps]
        at += k
    return [None, key, value]


def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _exact_sample, "append": _exact_append, "attend": _exact_attend, "settle": _exact_settle}[case["op"]](s)
