"""Operators for long and shared KV caches, as they are measured: tree attention of a batch whose
requests share long prefixes, and sparse attention over pages that a cheap score selects, with the
steps that lead to it (bounds of a page's keys, scores of pages against queries, selection).

Each case runs one call of one operator.  ``run`` computes it in plain torch operations, or, with
``own`` set, through this repository's entry points; ``exact`` is the definition in 64 bits, written
apart from the plain form.  Sizes are those of this repository's workloads (heads 32:8, 64:8 and 32:32,
head dim 128, prefixes up to 32768, pages of 16, up to 64 nodes) or around them.
"""
import math

import numpy as np
import torch

own = False

# ------------------------------------------------------------------------- trees

EXAMPLE7 = [-1, 0, 0, 1, 1, 2, 2]
T26 = [-1, 0, 0, 0, 0, 1, 1, 1, 2, 2, 3, 4, 5, 5, 6, 6, 7, 8, 8, 10, 12, 13, 14, 16, 17, 19]
T64 = [-1, 0, 0, 0, 0, 1, 1, 1, 2, 2, 2, 3, 3, 3, 4, 4, 4, 5, 5, 6, 6, 7, 7, 8, 8,
       9, 9, 10, 10, 11, 11, 12, 12, 13, 13, 14, 14, 15, 15, 16, 16, 17, 18, 19, 20,
       21, 22, 23, 24, 25, 26, 27, 28, 29, 30, 31, 32, 33, 34, 35, 36, 37, 38, 39]


def tree_of(name):
    """The parent array of a tree: "chainG" (G drafts after the root) or a named tree."""
    if name.startswith("chain"):
        return list(range(-1, int(name[5:])))
    return {"example7": EXAMPLE7, "t26": T26, "t64": T64}[name]


def nodes_of(case):
    return len(tree_of(case["tree"]))


def ancestors_of(parent):
    a = torch.zeros(len(parent), len(parent), dtype=torch.bool)
    for n, p in enumerate(parent):
        if p >= 0:
            a[n] = a[p]
        a[n, n] = True
    return a


# ------------------------------------------------------------------------- cases

def listed():
    shared = dict(op="shared", dtype="bf16", D=128)
    sparse = dict(op="sparse", dtype="bf16", D=128)
    scores = dict(op="scores", D=128)
    return [
        # one token each for a few requests behind one system prompt
        dict(shared, name="shared-decode", B=8, groups=1, tree="chain0", Hq=32, Hkv=8, lo=8192, hi=8192, own_lo=1, own_hi=300, page=16),
        # a full server: four applications with prompts of their own, chains of drafts, ragged own parts
        dict(shared, name="shared-groups", B=256, groups=4, tree="chain4", Hq=32, Hkv=8, lo=2048, hi=8192, own_lo=16, own_hi=512, page=16),
        # many samples of one prompt with Medusa's tree, no grouped heads, odd lengths
        dict(shared, name="shared-medusa-t64", B=32, groups=1, tree="t64", Hq=32, Hkv=32, lo=4099, hi=4099, own_lo=0, own_hi=77, page=0),
        # one decoded token of one long request, an eighth of a 32k prefix
        dict(sparse, name="sparse-decode-1", B=1, tree="chain0", Hq=32, Hkv=8, lo=32001, hi=32001, page=16, pages=256, per_node=False),
        # long contexts with a candidate tree whose nodes look at the same pages
        dict(sparse, name="sparse-long-tree", B=16, tree="t26", Hq=64, Hkv=8, lo=30000, hi=32768, page=16, pages=256, per_node=False),
        # each draft of a chain with pages of its own, as plain decoding would choose them
        dict(sparse, name="sparse-chain-nodes", B=64, tree="chain4", Hq=32, Hkv=8, lo=700, hi=8192, page=32, pages=32, per_node=True),
        # scores of all pages for the two long cases
        dict(scores, name="scores-decode", dtype="bf16", B=16, tree="chain0", Hq=32, Hkv=8, lo=30000, hi=32768, page=16, paged=True, per_node=False),
        dict(scores, name="scores-long-tree", dtype="bf16", B=16, tree="t26", Hq=64, Hkv=8, lo=30000, hi=32768, page=16, paged=True, per_node=False),
        # pages of one request, and of every node of a batch
        dict(op="select", name="select-decode-1", B=1, sets=1, Hkv=8, lo=32001, hi=32001, page=16, pages=256, first=1, last=4, levels=0),
        dict(op="select", name="select-chain-nodes", B=64, sets=5, Hkv=8, lo=700, hi=32768, page=16, pages=128, first=1, last=2, levels=0),
        # bounds of a batch of prompts, and after a verify step's commit
        dict(op="bounds", name="bounds-prompts", dtype="bf16", D=128, B=16, Hkv=8, lo=20000, hi=32768, page=16, paged=True, new_lo=32768, new_hi=32768),
        dict(op="bounds", name="bounds-step", dtype="bf16", D=128, B=256, Hkv=8, lo=512, hi=8192, page=16, paged=True, new_lo=1, new_hi=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


TREES = ["chain0", "chain0", "chain1", "chain3", "chain4", "chain7", "example7", "t26", "t64"]


def draw(rng):
    op = rng.choice(["shared", "shared", "sparse", "sparse", "scores", "select", "bounds"])
    while True:
        f32 = rng.random() < 0.2
        dtype = "f32" if f32 else "bf16"
        Hq, Hkv = rng.choice([(8, 8), (4, 4), (8, 2)] if f32 else [(32, 8), (32, 32), (64, 8), (28, 4), (16, 2), (8, 1)])
        D, tree, B = rng.choice([64, 128]), rng.choice(TREES), _log(rng, 1, 16 if f32 else 256)
        hi = _log(rng, 1, 4000 if f32 else 32768)
        lo = max(1, int(hi * rng.choice([0.1, 0.5, 1.0])))
        rows = B * len(tree_of(tree)) * Hq
        if op == "shared":
            own_hi = _log(rng, 1, 1000)
            c = dict(op=op, dtype=dtype, B=B, groups=rng.choice([1, 1, 2, 5]), tree=tree, Hq=Hq, Hkv=Hkv, D=D, lo=lo, hi=hi,
                     own_lo=rng.choice([0, 1, own_hi // 2]), own_hi=own_hi, page=rng.choice([0, 16, 16, 32, 64, 128]))
            c["groups"] = min(c["groups"], B)
            keys = hi + own_hi + 64
            if rows * keys <= (6e6 if f32 else 2.4e8) and B * keys * Hkv * D <= 2.4e9 and (c["page"] or B * keys * Hkv * D <= 8e8):
                return c
        if op == "sparse":
            page = rng.choice([16, 16, 32, 64, 128])
            per_node = rng.random() < 0.4
            pages = _log(rng, 1, max(1, 4096 // page))
            c = dict(op=op, dtype=dtype, B=B, tree=tree, Hq=Hq, Hkv=Hkv, D=D, lo=lo, hi=hi, page=page, pages=pages, per_node=per_node)
            units = B * (len(tree_of(tree)) if per_node else 1) * Hkv
            if rows * (pages * page + 64) <= (6e6 if f32 else 1.2e8) and units * (pages * page) * D <= 6e8 and B * (hi + 64) * Hkv * D <= 1.2e9:
                return c
        if op == "scores":
            c = dict(op=op, dtype=dtype, B=B, tree=tree, Hq=Hq, Hkv=Hkv, D=D, lo=lo, hi=hi, page=rng.choice([16, 32, 64, 128, 48]),
                     paged=rng.random() < 0.7, per_node=rng.random() < 0.5)
            if rows * (hi // c["page"] + 1) <= (3e6 if f32 else 1e8):
                return c
        if op == "select":
            c = dict(op=op, B=B, sets=rng.choice([1, 1, 5, 26]), Hkv=Hkv, hi=_log(rng, 600, 131072), page=rng.choice([16, 32, 64, 128]),
                     pages=_log(rng, 1, 512), first=rng.choice([0, 1, 4]), last=rng.choice([0, 1, 4]), levels=rng.choice([0, 0, 3, 40]))
            c["lo"] = max(c["hi"] // 8, 4 * c["page"])
            c["pages"] = min(c["pages"], c["lo"] // c["page"] // 2)
            c["first"], c["last"] = min(c["first"], c["pages"] // 2), min(c["last"], c["pages"] // 4)
            if B * c["sets"] * Hkv * (c["hi"] // c["page"] + 1) <= 6e6:
                return c
        if op == "bounds":
            c = dict(op=op, dtype=dtype, D=D, B=B, Hkv=Hkv, lo=lo, hi=hi, page=rng.choice([16, 32, 64, 128, 48]), paged=rng.random() < 0.7,
                     new_lo=1, new_hi=rng.choice([1, 5, 40, hi]))
            if B * (hi + 128) * Hkv * D <= 6e8:
                return c


# ------------------------------------------------------------------------- inputs

def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _tables(gc, count, most=0):
    """Block tables of requests that hold `count` pages each, ids in random order, and the pool's size:
    rows for `most` pages each, or for those that are there."""
    total = len(count) * most or int(count.sum())
    order = torch.randperm(total, generator=gc)[:int(count.sum())].to(torch.int32)
    held = torch.arange(max(most, int(count.max())))[None, :] < count[:, None]
    table = torch.full(held.shape, -1, dtype=torch.int32)
    table[held] = order
    return table, total


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    dtype = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    gc = torch.Generator().manual_seed(int(seed))
    g = torch.Generator(device=dev).manual_seed(int(seed) + 1)

    def randn(*shape, dtype=dtype):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    def ints(t):
        return t.to(torch.int32).to(dev)

    op, B, Hkv, page = c["op"], c["B"], c["Hkv"], c["page"]
    if op == "select":
        length = _ints(gc, c["lo"], c["hi"], B)
        P = -(-c["hi"] // page)
        # what the nodes of a request have in common, and their own part; few levels make ties
        base, mine = randn(B, 1, Hkv, P, dtype=torch.float32), randn(B, c["sets"], Hkv, P, dtype=torch.float32)
        x = 40 + 8 * base + 3 * mine
        if c["levels"]:
            x = torch.round(x / 30 * c["levels"])
        there = torch.arange(P) < ((length + page - 1) // page)[:, None]
        x = torch.where(there.to(dev)[:, None, None, :], x, -math.inf)
        return dict(case=c, scores=x, length=ints(length))
    D = c["D"]
    if op == "bounds":
        length = _ints(gc, c["lo"], c["hi"], B)
        start = (length - _ints(gc, c["new_lo"], c["new_hi"], B)).clamp(min=0)
        count = (length + page - 1) // page
        s = dict(case=c, length=ints(length), start=ints(start), block_table=None)
        if c["paged"]:
            table, total = _tables(gc, count, -(-c["hi"] // page))
            s["block_table"], s["k"] = table.to(dev), randn(total, page, Hkv, D)
            rows = (total,)
        else:
            s["k"] = randn(B, c["hi"], Hkv, D)
            rows = (B, -(-c["hi"] // page))
        s["v"] = s["k"]  # (not read)
        s["bounds"] = randn(*rows, Hkv, 2, D)
        return s
    parent = tree_of(c["tree"])
    N, Hq = len(parent), c["Hq"]
    if op == "scores":
        length = _ints(gc, c["lo"], c["hi"], B)
        count = (length + page - 1) // page
        s = dict(case=c, length=ints(length), block_table=None, q=randn(B, N, Hq, D), max_prefix=c["hi"])
        if c["paged"]:
            table, total = _tables(gc, count, -(-c["hi"] // page))
            s["block_table"] = table.to(dev)
            rows = (total,)
        else:
            rows = (B, -(-c["hi"] // page))
        # the largest and smallest of a page's 16 or more keys lie about 1.8 around their mean
        middle, half = 0.5 * randn(*rows, Hkv, D, dtype=torch.float32), 1.8 + 0.4 * randn(*rows, Hkv, D, dtype=torch.float32)
        s["bounds"] = torch.stack([middle - half.abs(), middle + half.abs()], -2).to(dtype)
        return s
    s = dict(case=c, parent=parent, ancestor=ancestors_of(parent).to(dev), scale=D ** -0.5, q=randn(B, N, Hq, D),
             k_tree=randn(B, N, Hkv, D), v_tree=randn(B, N, Hkv, D), block_table=None)
    if op == "shared":
        n = c["groups"]
        bounds = torch.sort(torch.randperm(B - 1, generator=gc)[:n - 1] + 1).values if n > 1 else torch.zeros(0, dtype=torch.long)
        starts = torch.cat([torch.zeros(1, dtype=torch.long), bounds, torch.tensor([B])])
        group = torch.bucketize(torch.arange(B), starts[1:], right=True)
        shared = _ints(gc, c["lo"], c["hi"], n)
        length = shared[group] + _ints(gc, c["own_lo"], c["own_hi"], B)
        s.update(group_start=ints(starts), shared_len=ints(shared), length=ints(length))
        if page:
            count = (length + N + page - 1) // page
            table, total = _tables(gc, count)
            whole = (shared // page)[group]  # pages that the members of a group have in common
            col = torch.arange(table.shape[1])
            table = torch.where(col[None, :] < whole[:, None], table[starts[group]], table)
            s["block_table"] = table.to(dev)
            s["k"], s["v"] = randn(total, page, Hkv, D), randn(total, page, Hkv, D)
        else:
            s["k"], s["v"] = randn(B, int(length.max()) + N, Hkv, D), randn(B, int(length.max()) + N, Hkv, D)
        for b in range(B):  # the rest of the shared prefix is a copy of the first member's
            first, n = int(starts[group[b]]), int(shared[group[b]])
            for t in (s["k"], s["v"]):
                if first == b:
                    continue
                if not page:
                    t[b, :n] = t[first, :n]
                elif n % page:
                    t[int(table[b, n // page]), :n % page] = t[int(table[first, n // page]), :n % page]
        return s
    # sparse
    length = _ints(gc, c["lo"], c["hi"], B)
    count = (length + page - 1) // page
    table, total = _tables(gc, (length + N + page - 1) // page)
    s.update(block_table=table.to(dev), length=ints(length), k=randn(total, page, Hkv, D), v=randn(total, page, Hkv, D))
    sets, K, P = N if c["per_node"] else 1, c["pages"], int(count.max())
    x = randn(B, 1, Hkv, P, dtype=torch.float32) + 0.4 * randn(B, sets, Hkv, P, dtype=torch.float32)
    col = torch.arange(P, device=dev)
    n = count.to(dev)[:, None, None, None]
    x = torch.where((col == 0) | (col == n - 1), math.inf, x).masked_fill(col >= n, -math.inf)
    top, at = x.topk(min(K, P), -1)
    at = torch.where(top > -math.inf, at, P).sort(-1).values
    pages = torch.full((B, sets, Hkv, K), -1, dtype=torch.int32, device=dev)
    pages[..., :at.shape[-1]] = torch.where(at < P, at, -1).to(torch.int32)
    s["pages"] = pages
    return s


# -------------------------------------------------------------------- plain forms

def _attend(q, k, v, see, scale):
    """q [U,R,D], k and v [U,K,D], see [U,R,K] -> [U,R,D] in 32 bits."""
    x = (q @ k.transpose(1, 2) * scale).masked_fill(~see, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return (e / e.sum(-1, keepdim=True)) @ v


def _plain_shared(s):
    c = s["case"]
    B, N, Hq, D = s["q"].shape
    Hkv, page = c["Hkv"], c["page"]
    L = s["length"].long()[:, None]
    pos = torch.arange(c["hi"] + c["own_hi"], device=L.device).expand(B, -1)
    there = pos < L
    seq = torch.arange(B, device=L.device)[:, None]
    at = torch.where(there, pos, 0)
    if page:
        row = s["block_table"][seq, at // page].long() * page + at % page
    else:
        row = seq * s["k"].shape[1] + at
    k = torch.cat([s["k"].view(-1, Hkv, D)[row].float(), s["k_tree"].float()], 1).transpose(1, 2).reshape(B * Hkv, -1, D)
    v = torch.cat([s["v"].view(-1, Hkv, D)[row].float(), s["v_tree"].float()], 1).transpose(1, 2).reshape(B * Hkv, -1, D)
    see = torch.cat([there[:, None, :].expand(B, N, -1), s["ancestor"].expand(B, N, N)], 2)
    see = see[:, None, :, None, :].expand(B, Hkv, N, Hq // Hkv, -1).reshape(B * Hkv, N * (Hq // Hkv), -1)
    q = s["q"].float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B * Hkv, -1, D)
    o = _attend(q, k, v, see, s["scale"])
    return o.view(B, Hkv, N, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(s["q"].dtype)


def _plain_sparse(s):
    c = s["case"]
    B, N, Hq, D = s["q"].shape
    Hkv, page, G = c["Hkv"], c["page"], c["Hq"] // c["Hkv"]
    S, K = s["pages"].shape[1], s["pages"].shape[3]
    dev = s["q"].device
    pages = s["pages"].long()
    pos = (pages[..., None] * page + torch.arange(page, device=dev)).view(B, S, Hkv, K * page)
    there = (pages >= 0)[..., None].expand(-1, -1, -1, -1, page).reshape(pos.shape) & (pos < s["length"].long()[:, None, None, None])
    at = torch.where(there, pos, 0)
    row = s["block_table"][torch.arange(B, device=dev)[:, None, None, None], at // page].long() * page + at % page
    head = torch.arange(Hkv, device=dev)[None, None, :, None]
    tree = lambda t: t.float().transpose(1, 2)[:, None].expand(B, S, Hkv, N, D)  # noqa: E731
    k = torch.cat([s["k"].view(-1, Hkv, D)[row, head].float(), tree(s["k_tree"])], 3).view(B * S * Hkv, -1, D)
    v = torch.cat([s["v"].view(-1, Hkv, D)[row, head].float(), tree(s["v_tree"])], 3).view(B * S * Hkv, -1, D)
    # the rows of a set: all nodes, or one
    anc = s["ancestor"].view(1, S, 1, N // S, 1, N).expand(B, S, Hkv, N // S, G, N).reshape(B, S, Hkv, -1, N)
    see = torch.cat([there[:, :, :, None, :].expand(-1, -1, -1, N // S * G, -1), anc], 4).view(B * S * Hkv, N // S * G, -1)
    q = s["q"].float().view(B, S, N // S, Hkv, G, D).permute(0, 1, 3, 2, 4, 5).reshape(B * S * Hkv, -1, D)
    o = _attend(q, k, v, see, s["scale"])
    return o.view(B, S, Hkv, N // S, G, D).permute(0, 1, 3, 2, 4, 5).reshape(B, N, Hq, D).to(s["q"].dtype)


def _plain_scores(s):
    c = s["case"]
    B, N, Hq, D = s["q"].shape
    Hkv, page = c["Hkv"], c["page"]
    S = N if c["per_node"] else 1
    P = s["block_table"].shape[1] if c["paged"] else -(-s["max_prefix"] // page)
    n = (s["length"].long() + page - 1) // page
    there = torch.arange(P, device=n.device) < n[:, None]
    if c["paged"]:
        b = s["bounds"][s["block_table"].long().clamp(min=0)].float()  # [B, P, Hkv, 2, D]
    else:
        b = s["bounds"].float()
    q = s["q"].float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    x = q.clamp(min=0) @ b[..., 1, :].permute(0, 2, 3, 1) + q.clamp(max=0) @ b[..., 0, :].permute(0, 2, 3, 1)
    x = x.view(B, Hkv, S, -1, P).amax(3).transpose(1, 2)  # the largest of a set's rows
    return torch.where(there[:, None, None, :], x, -math.inf)


def _plain_select(s):
    c = s["case"]
    x = s["scores"]
    P = x.shape[-1]
    n = ((s["length"].long() + c["page"] - 1) // c["page"])[:, None, None, None]
    col = torch.arange(P, device=x.device)
    kept = ((col < c["first"]) | (col >= n - c["last"])) & (col < n)
    # kept pages, then the others by score, then what is not there; equal ones in order of their index
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    rank = torch.gather(torch.where(col >= n, 2, torch.where(kept, 0, 1)).expand(x.shape), -1, order)
    order = torch.gather(order, -1, torch.sort(rank, dim=-1, stable=True).indices)[..., :c["pages"]]
    order = torch.where(order < n, order, P).sort(-1).values
    out = torch.full((*x.shape[:-1], c["pages"]), -1, dtype=torch.int32, device=x.device)
    out[..., :order.shape[-1]] = torch.where(order < P, order, -1).to(torch.int32)
    return out


def _plain_bounds(s):
    c = s["case"]
    page, Hkv, D = c["page"], c["Hkv"], c["D"]
    L, start = s["length"].long(), s["start"].long()
    n, first = (L + page - 1) // page, start // page
    P = int(c["hi"] + page - 1) // page
    col = torch.arange(P, device=L.device)
    b, p = torch.nonzero((col >= first[:, None]) & (col < n[:, None]) & (start < L)[:, None], as_tuple=True)
    pos = p[:, None] * page + torch.arange(page, device=L.device)
    there = pos < L[b][:, None]
    if c["paged"]:
        at = s["block_table"][b, p].long()
        k = s["k"][at]
    else:
        at = b * s["bounds"].shape[1] + p
        k = s["k"][b[:, None], pos.clamp(max=s["k"].shape[1] - 1)]
    there = there[:, :, None, None]
    low = torch.where(there, k, math.inf).amin(1)
    high = torch.where(there, k, -math.inf).amax(1)
    s["bounds"].view(-1, Hkv, 2, D)[at] = torch.stack([low, high], 2)
    return s["bounds"]


# ------------------------------------------------------------- this repository's calls

def _cache(s):
    """What a program keeps between steps: the cache's handle, the output and the workspace."""
    import speculative_decoding_verify_sv_gb300 as sv
    if "cache" not in s:
        k = s.get("k")
        s["cache"] = sv.KVCache(k, s.get("v"), s["length"], s["block_table"], s["case"]["page"] or 16)
    return sv, s["cache"]


def _own_shared(s):
    sv, cache = _cache(s)
    c = s["case"]
    if "out" not in s:
        B, N, Hq, D = s["q"].shape
        size = sv.sv_shared_attention_workspace_size(s["q"].dtype, B, N, Hq, c["Hkv"], D, cache.max_prefix, c["groups"])
        s["workspace"] = torch.zeros(max(size, 16), dtype=torch.uint8, device=s["q"].device)
        s["out"] = torch.empty_like(s["q"])
    return sv.sv_shared_attention(s["q"], s["k_tree"], s["v_tree"], cache, s["parent"], s["scale"], s["group_start"], s["shared_len"],
                                  out=s["out"], workspace=s["workspace"])


def _own_sparse(s):
    sv, cache = _cache(s)
    c = s["case"]
    if "out" not in s:
        B, N, Hq, D = s["q"].shape
        size = sv.sv_sparse_attention_workspace_size(s["q"].dtype, B, N, Hq, c["Hkv"], D, c["page"], c["pages"], s["pages"].shape[1])
        s["workspace"] = torch.zeros(max(size, 16), dtype=torch.uint8, device=s["q"].device)
        s["out"] = torch.empty_like(s["q"])
    return sv.sv_sparse_attention(s["q"], s["k_tree"], s["v_tree"], cache, s["parent"], s["scale"], s["pages"], out=s["out"],
                                  workspace=s["workspace"])


def _own_scores(s):
    import speculative_decoding_verify_sv_gb300 as sv
    c = s["case"]
    return sv.sv_page_scores(s["q"], s["bounds"], s["length"], c["page"], block_table=s["block_table"], per_node=c["per_node"])


def _own_select(s):
    import speculative_decoding_verify_sv_gb300 as sv
    c = s["case"]
    return sv.sv_select_pages(s["scores"], s["length"], c["page"], c["pages"], first=c["first"], last=c["last"])


def _own_bounds(s):
    sv, cache = _cache(s)
    return sv.sv_page_bounds(cache, s["bounds"], start=s["start"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"shared": _own_shared, "sparse": _own_sparse, "scores": _own_scores, "select": _own_select, "bounds": _own_bounds}[op](state)
    return {"shared": _plain_shared, "sparse": _plain_sparse, "scores": _plain_scores, "select": _plain_select, "bounds": _plain_bounds}[op](state)


# ---------------------------------------------------------------------------- work

def work(case):
    c = case
    e = 2 if c.get("dtype") == "bf16" else 4
    mean, most = (c["lo"] + c["hi"]) / 2, c["hi"]
    if c["op"] == "select":
        return {"bytes": c["B"] * c["sets"] * c["Hkv"] * 4.0 * (mean / c["page"] + c["pages"]), "flops": 0.0}
    row = c["Hkv"] * c["D"] * e
    if c["op"] == "bounds":
        new = min(mean, (c["new_lo"] + c["new_hi"]) / 2)
        # (a new token's page is read from its start)
        keys = min(mean, new + (c["page"] - 1) / 2) if new < mean else mean
        return {"bytes": c["B"] * row * (keys + 2 * max(1.0, keys / c["page"])), "flops": 2.0 * c["B"] * keys * c["Hkv"] * c["D"]}
    N = nodes_of(c)
    qo = c["B"] * N * c["Hq"] * c["D"]
    if c["op"] == "scores":
        pages = c["B"] * (mean / c["page"])
        sets = N if c["per_node"] else 1
        return {"bytes": qo * e + 2 * pages * row + 4.0 * c["B"] * sets * c["Hkv"] * most / c["page"],
                "flops": 4.0 * pages * N * c["Hq"] * c["D"]}
    if c["op"] == "shared":
        own_part = c["B"] * ((c["own_lo"] + c["own_hi"]) / 2 + N)
        keys = mean + (c["own_lo"] + c["own_hi"]) / 2 + N
        return {"bytes": 2 * row * (c["groups"] * mean + own_part) + 2 * qo * e, "flops": 4.0 * qo * keys}
    # sparse: a page that several nodes of a request have listed is counted once
    P = max(1, int(mean / c["page"]))
    K = min(c["pages"], P)
    seen = float(K)
    if c["per_node"] and N > 1:
        r = np.random.RandomState(0)
        x = r.randn(8, 1, P) + 0.4 * r.randn(8, N, P)
        at = np.argsort(-x, -1)[..., :K]
        seen = float(np.mean([len(np.unique(a)) for a in at]))
    return {"bytes": 2 * row * c["B"] * (seen * c["page"] + N) + 2 * qo * e + 4.0 * c["B"] * (N if c["per_node"] else 1) * c["Hkv"] * c["pages"],
            "flops": 4.0 * qo * (min(K * c["page"], mean) + N)}


# --------------------------------------------------------------- the definition, 64 bits

def _rows_of(s, b, pos):
    """Keys and values at these positions of sequence b."""
    page = s["case"]["page"]
    if s["block_table"] is None:
        return s["k"][b, pos], s["v"][b, pos]
    at = s["block_table"][b, pos // page].long()
    return s["k"][at, pos % page], s["v"][at, pos % page]


def _softmax_sum(q, k, v, see, scale):
    """q [R, D], k and v [K, D], see [R, K]"""
    x = torch.einsum("rd,kd->rk", q.double(), k.double()) * scale
    return torch.einsum("rk,kd->rd", torch.softmax(torch.where(see, x, torch.full_like(x, -math.inf)), -1), v.double())


def _exact_shared(s):
    c = s["case"]
    B, N, Hq, D = s["q"].shape
    Hkv, G = c["Hkv"], Hq // c["Hkv"]
    out = torch.empty(B, N, Hq, D, dtype=torch.float64, device=s["q"].device)
    starts, lens = s["group_start"].tolist(), s["length"].tolist()
    for i, shared in enumerate(s["shared_len"].tolist()):
        ks, vs = _rows_of(s, starts[i], torch.arange(shared, device=out.device))
        for b in range(starts[i], starts[i + 1]):
            ko, vo = _rows_of(s, b, torch.arange(shared, lens[b], device=out.device))
            k, v = torch.cat([ks, ko, s["k_tree"][b]]), torch.cat([vs, vo, s["v_tree"][b]])
            see = torch.ones(N, k.shape[0], dtype=torch.bool, device=out.device)
            see[:, lens[b]:] = s["ancestor"]
            see = see.repeat_interleave(G, 0)
            for h in range(Hkv):
                q = s["q"][b, :, h * G:(h + 1) * G].reshape(-1, D)
                out[b, :, h * G:(h + 1) * G] = _softmax_sum(q, k[:, h], v[:, h], see, s["scale"]).view(N, G, D)
    return out


def _exact_sparse(s):
    c = s["case"]
    B, N, Hq, D = s["q"].shape
    Hkv, G, page = c["Hkv"], Hq // c["Hkv"], c["page"]
    out = torch.empty(B, N, Hq, D, dtype=torch.float64, device=s["q"].device)
    S = s["pages"].shape[1]
    pages = s["pages"].cpu()
    for b, L in enumerate(s["length"].tolist()):
        for i in range(S):
            nodes = slice(0, N) if S == 1 else slice(i, i + 1)
            for h in range(Hkv):
                pos = [p for j in pages[b, i, h].tolist() if j >= 0 for p in range(j * page, min(L, (j + 1) * page))]
                kp, vp = _rows_of(s, b, torch.tensor(pos, dtype=torch.long, device=out.device))
                k, v = torch.cat([kp[:, h], s["k_tree"][b, :, h]]), torch.cat([vp[:, h], s["v_tree"][b, :, h]])
                anc = s["ancestor"][nodes]
                see = torch.cat([torch.ones(len(anc), len(pos), dtype=torch.bool, device=out.device), anc], 1).repeat_interleave(G, 0)
                q = s["q"][b, nodes, h * G:(h + 1) * G]
                out[b, nodes, h * G:(h + 1) * G] = _softmax_sum(q.reshape(-1, D), k, v, see, s["scale"]).view(q.shape)
    return out


def _exact_scores(s):
    c = s["case"]
    B, N, Hq, D = s["q"].shape
    Hkv, page = c["Hkv"], c["page"]
    G, S = Hq // Hkv, N if c["per_node"] else 1
    P = s["block_table"].shape[1] if c["paged"] else -(-s["max_prefix"] // page)
    out = torch.full((B, S, Hkv, P), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, L in enumerate(s["length"].tolist()):
        n = -(-L // page)
        x = s["bounds"][s["block_table"][b, :n].long()] if c["paged"] else s["bounds"][b, :n]
        for h in range(Hkv):
            best = torch.full((S, n), -math.inf, dtype=torch.float64, device=out.device)
            for j in range(G):
                q = s["q"][b, :, h * G + j].double()
                # the largest product that a key between the bounds can have, channel by channel
                up = torch.where(q[:, None, :] > 0, x[None, :, h, 1].double(), x[None, :, h, 0].double())
                y = torch.einsum("nd,npd->np", q, up)
                best = torch.maximum(best, y if S == N else y.amax(0, keepdim=True))
            out[b, :, h, :n] = best
    return out


def _exact_select(s):
    c = s["case"]
    x, out = s["scores"].cpu().numpy(), None
    out = np.full((*x.shape[:-1], c["pages"]), -1, np.int32)
    for b, L in enumerate(s["length"].tolist()):
        n = -(-L // c["page"])
        keep = sorted(set(range(min(c["first"], n))) | set(range(max(0, n - c["last"]), n)))
        rest = np.setdiff1d(np.arange(n), keep)
        for i in np.ndindex(x.shape[1:-1]):
            by = rest[np.argsort(-x[(b, *i)][rest], kind="stable")][:c["pages"] - len(keep)]
            got = np.sort(np.concatenate([np.array(keep, np.int64), by]))
            out[(b, *i)][:len(got)] = got
    return out


def _exact_bounds(s):
    c = s["case"]
    page = c["page"]
    out = s["bounds"].double()
    for b, (L, start) in enumerate(zip(s["length"].tolist(), s["start"].tolist())):
        for p in range(start // page, -(-L // page) if start < L else 0):
            if c["paged"]:
                at = int(s["block_table"][b, p])
                k, to = s["k"][at, :min(page, L - p * page)], out[at]
            else:
                k, to = s["k"][b, p * page:min(L, (p + 1) * page)], out[b, p]
            to[:, 0], to[:, 1] = k.amin(0).double(), k.amax(0).double()
    return out


def exact(case, seed):
    c = case
    if c["op"] == "sparse" and c["B"] * (nodes_of(c) if c["per_node"] else 1) * c["Hkv"] * (c["pages"] * c["page"] + 400) > 3e7:
        return None
    if c["op"] == "scores" and c["B"] * nodes_of(c) * c["Hq"] * (c["hi"] / c["page"] + 1) * c["D"] > 3e10:
        return None
    if c["op"] == "bounds" and c["B"] * min(c["hi"], c["new_hi"]) / c["page"] > 60000:
        return None
    if c["op"] == "select" and c["B"] * c["sets"] * c["Hkv"] > 40000:
        return None
    s = prepare(case, seed)
    return {"shared": _exact_shared, "sparse": _exact_sparse, "scores": _exact_scores, "select": _exact_select, "bounds": _exact_bounds}[c["op"]](s)
