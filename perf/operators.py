"""Three operators around the KV cache, as they are measured: block tables and slot maps from
request lengths, the per-head norms of queries and keys with the position rotation, and tree
attention with a sliding window and sinks.

Each case runs one call of one operator.  ``run`` computes it in plain torch operations, or,
with ``own`` set, through this repository's entry points; ``exact`` is the definition in 64
bits, written apart from the plain form.  Sizes are those of this repository's workloads
(heads 32:8, 64:8 and 32:32, head dim 128, prefixes up to 32768, pages of 16, up to 64 nodes)
or around them.
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


def depth_of(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


# ------------------------------------------------------------------------- cases

def listed():
    att = dict(op="window", dtype="bf16", D=128)
    rope = dict(op="rope", dtype="bf16", D=128, rot=128, interleaved=False)
    return [
        # plain decoding of one request (no drafts): one token, a windowed layer
        dict(att, name="window-decode-1", B=1, tree="chain0", Hq=32, Hkv=8, lo=4097, hi=4097, W=1024, S=4, page=0),
        # a full server's verify step on a windowed layer: many ragged requests, paged cache
        dict(att, name="window-ragged-paged", B=256, tree="chain4", Hq=32, Hkv=8, lo=512, hi=8192, W=1024, S=4, page=16),
        # Medusa's 64-node tree without grouped heads, short odd window and no sinks
        dict(att, name="window-medusa-t64", B=8, tree="t64", Hq=32, Hkv=32, lo=2048, hi=2048, W=513, S=0, page=0),
        # long contexts with a wide window and many sinks
        dict(att, name="window-long-tree", B=16, tree="t26", Hq=64, Hkv=8, lo=30000, hi=32768, W=8192, S=64, page=0),
        # the 32-bit form on a small model: odd lengths
        dict(op="window", name="window-f32", dtype="f32", B=5, tree="chain4", Hq=4, Hkv=4, D=64, lo=100, hi=777, W=129, S=3, page=0),
        # one decoded token: where latency counts
        dict(rope, name="rope-token-1", form="slots", T=1, Hq=32, Hkv=8, pad=0),
        # the tree rows of a verify step: positions from the prefix lengths and the tree
        dict(rope, name="rope-verify-tree", form="tree", B=64, tree="chain5", Hq=32, Hkv=8, pad=0),
        # prompts of a batch written straight into the paged cache
        dict(rope, name="rope-prompt-32k", form="slots", T=32768, Hq=32, Hkv=8, pad=0),
        # partial rotation of neighbouring pairs, 32 bits, rows inside a wider projection
        dict(op="rope", name="rope-partial-f32", dtype="f32", form="slots", T=777, Hq=12, Hkv=4, D=64, rot=32, interleaved=True, pad=64),
        # the new slots of one verify step: a chain of 4 drafts each
        dict(op="tables", name="tables-verify", B=256, lo=512, hi=8192, new_lo=5, new_hi=5, page=16),
        # a batch of fresh prompts: every page of the ragged-paged workload
        dict(op="tables", name="tables-prompts", B=256, lo=0, hi=0, new_lo=512, new_hi=8192, page=16),
        # many requests with a few tokens each, some with none
        dict(op="tables", name="tables-many", B=4096, lo=0, hi=2000, new_lo=0, new_hi=64, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "rope", "tables"])
    if op == "window":
        while True:
            f32 = rng.random() < 0.2
            heads = rng.choice([(8, 8), (4, 4), (8, 2)] if f32 else
                               [(32, 8), (32, 32), (64, 8), (28, 4), (16, 2), (8, 1)])
            hi = _log(rng, 1, 2000 if f32 else 32768)
            c = dict(op=op, dtype="f32" if f32 else "bf16", B=_log(rng, 1, 16 if f32 else 256),
                     tree=rng.choice(["chain0", "chain1", "chain3", "chain4", "chain7", "example7", "t26", "t64"]),
                     Hq=heads[0], Hkv=heads[1], D=rng.choice([64, 128]), lo=max(1, int(hi * rng.choice([0.1, 0.5, 1.0]))),
                     hi=hi, W=_log(rng, 1, 500 if f32 else 8192), S=rng.choice([0, 1, 4, 17, 64]),
                     page=rng.choice([0, 16, 16, 32, 64, 128]))
            rows = c["B"] * len(tree_of(c["tree"])) * c["Hq"]
            seen = min(c["hi"], c["W"]) + c["S"] + 64
            cache = c["B"] * (c["hi"] + 64) * c["Hkv"] * c["D"]
            if cache <= 1.2e9 and rows * seen <= (3e6 if f32 else 2e8) and c["B"] * seen * c["Hkv"] * c["D"] <= 3e8:
                return c
    if op == "rope":
        D = rng.choice([64, 128])
        heads = rng.choice([(32, 8), (32, 32), (64, 8), (12, 4), (28, 4), (5, 1)])
        f32 = rng.random() < 0.3
        c = dict(op=op, dtype="f32" if f32 else "bf16", D=D, rot=rng.choice([D, D // 2, 16]),
                 interleaved=rng.random() < 0.4, Hq=heads[0], Hkv=heads[1], pad=rng.choice([0, 0, 8, 64]))
        most = int(32768 * 48 * 128 / ((heads[0] + 2 * heads[1]) * D * (2 if f32 else 1)))
        if rng.random() < 0.5:
            return dict(c, form="slots", T=_log(rng, 1, min(32768, most)))
        return dict(c, form="tree", B=_log(rng, 1, 128), tree=rng.choice(["chain0", "chain4", "example7", "t26", "t64"]))
    lo = rng.choice([0, 1, 700])
    new = _log(rng, 1, 8192)
    return dict(op=op, B=_log(rng, 1, min(8192, max(1, 1100000 // new))), lo=lo, hi=lo + _log(rng, 1, 2000),
                new_lo=rng.choice([0, new]), new_hi=new, page=rng.choice([16, 32, 64, 1, 48]))


# ------------------------------------------------------------------------- inputs

def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gc = torch.Generator().manual_seed(int(seed))
    g = torch.Generator(device=dev).manual_seed(int(seed) + 1)

    def randn(*shape, dtype=None):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype or _dtype(c))

    if c["op"] == "window":
        parent = tree_of(c["tree"])
        B, N, Hq, Hkv, D = c["B"], len(parent), c["Hq"], c["Hkv"], c["D"]
        lens = _ints(gc, c["lo"], c["hi"], B)
        s = dict(case=c, parent=parent, depth=torch.tensor(depth_of(parent), device=dev), scale=D ** -0.5,
                 q=randn(B, N, Hq, D), k_tree=randn(B, N, Hkv, D), v_tree=randn(B, N, Hkv, D),
                 length=lens.to(torch.int32).to(dev))
        anc = torch.zeros(N, N, dtype=torch.bool)
        for n in range(N):
            a = n
            while a >= 0:
                anc[n, a] = True
                a = parent[a]
        s["ancestor"] = anc.to(dev)
        if c["page"]:
            pages = [(int(x) + N + c["page"] - 1) // c["page"] for x in lens.tolist()]
            order = torch.randperm(sum(pages), generator=gc).to(torch.int32)
            table = torch.full((B, max(pages)), -1, dtype=torch.int32)
            at = 0
            for b, n in enumerate(pages):
                table[b, :n] = order[at:at + n]
                at += n
            s["block_table"] = table.to(dev)
            shape = (sum(pages), c["page"], Hkv, D)
        else:
            s["block_table"] = None
            shape = (B, int(lens.max()) + N, Hkv, D)
        s["k"], s["v"] = randn(*shape), randn(*shape)
        return s

    if c["op"] == "rope":
        Hq, Hkv, D, rot = c["Hq"], c["Hkv"], c["D"], c["rot"]
        width = (Hq + 2 * Hkv) * D
        s = dict(case=c, eps=1e-6,
                 q_weight=1 + 0.2 * randn(D, dtype=torch.float32), k_weight=1 + 0.2 * randn(D, dtype=torch.float32),
                 inv_freq=torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=dev))
        if c["form"] == "tree":
            s["parent"] = tree_of(c["tree"])
            s["depth"] = torch.tensor(depth_of(s["parent"]), device=dev)
            s["length"] = _ints(gc, 1, 32768, c["B"]).to(torch.int32).to(dev)
            lead = (c["B"], len(s["parent"]))
        else:
            T = c["T"]
            lead = (T,)
            # prompts one after another, each counted from a start of its own
            s["positions"] = ((torch.arange(T) + int(_ints(gc, 0, 4096, 1))) % 32768).to(torch.int32).to(dev)
            rows = T + T // 4 + 8
            s["slots"] = torch.randperm(rows, generator=gc)[:T].to(torch.int32).to(dev)
            s["k"], s["v"] = randn(rows, Hkv, D), randn(rows, Hkv, D)
        wide = randn(*lead, width + c["pad"])
        s["qkv"] = wide[..., c["pad"]:]
        return s

    B, bs = c["B"], c["page"]
    length = _ints(gc, c["lo"], c["hi"], B)
    new = _ints(gc, c["new_lo"], c["new_hi"], B)
    have = (length + bs - 1) // bs
    need = (length + new + bs - 1) // bs - have
    num_blocks = int(have.sum() + need.sum()) + 64
    order = torch.randperm(num_blocks, generator=gc).to(torch.int32)
    table = torch.full((B, c["hi"] // bs + c["new_hi"] // bs + 2), -1, dtype=torch.int32)
    col = torch.arange(table.shape[1])
    held = col[None, :] < have[:, None]
    table[held] = order[:int(have.sum())]
    return dict(case=c, length=length.to(torch.int32).to(dev), new=new.to(torch.int32).to(dev), block_table=table.to(dev),
                free=order[int(have.sum()):].to(dev), head=torch.tensor([17], dtype=torch.int32, device=dev),
                num_blocks=num_blocks, slots=B * c["new_hi"] + 16)


# -------------------------------------------------------------------- plain forms

def _plain_window(s):
    c = s["case"]
    B, N, Hq, D = s["q"].shape
    Hkv, W, S = c["Hkv"], c["W"], c["S"]
    L = s["length"].long()
    first = (L - W + 1).clamp(min=0)
    span = min(c["hi"], W - 1)
    pos = torch.cat([torch.arange(S, device=L.device).expand(B, S),
                     first[:, None] + torch.arange(span, device=L.device)], 1)
    there = pos < L[:, None]
    there[:, :S] &= pos[:, :S] < first[:, None]
    at = torch.where(there, pos, 0)
    if c["page"]:
        row = torch.gather(s["block_table"], 1, at // c["page"]).long().clamp(min=0) * c["page"] + at % c["page"]
    else:
        row = torch.arange(B, device=L.device)[:, None] * s["k"].shape[1] + at
    k = torch.cat([s["k"].view(-1, Hkv, D)[row].float(), s["k_tree"].float()], 1)
    v = torch.cat([s["v"].view(-1, Hkv, D)[row].float(), s["v_tree"].float()], 1)
    me = L[:, None] + s["depth"]  # [B, N]
    near = (me[:, :, None] - pos[:, None, :] < W) | (pos < S)[:, None, :]
    near_tree = (me[:, :, None] - me[:, None, :] < W) | (me < S)[:, None, :]
    see = torch.cat([near & there[:, None, :], near_tree & s["ancestor"]], 2)
    q = s["q"].float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    score = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
    score = score.view(B, Hkv, N, Hq // Hkv, -1).masked_fill(~see[:, None, :, None, :], -math.inf)
    e = torch.exp(score - score.amax(-1, keepdim=True))
    o = (e / e.sum(-1, keepdim=True)).view(B, Hkv, -1, e.shape[-1]) @ v.permute(0, 2, 1, 3)
    return o.view(B, Hkv, N, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(s["q"].dtype)


def _plain_rope(s):
    c = s["case"]
    Hq, Hkv, D, rot = c["Hq"], c["Hkv"], c["D"], c["rot"]
    if c["form"] == "tree":
        position = s["length"].double()[:, None] + s["depth"].double()
    else:
        position = s["positions"].double()
    angle = position[..., None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float()[..., None, :], torch.sin(angle).float()[..., None, :]
    x = s["qkv"].unflatten(-1, (Hq + 2 * Hkv, D))

    def turn(y, weight):
        y = y.float()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * weight
        if c["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([r, y[..., rot:]], -1).to(x.dtype)

    q, k, v = turn(x[..., :Hq, :], s["q_weight"]), turn(x[..., Hq:Hq + Hkv, :], s["k_weight"]), x[..., Hq + Hkv:, :]
    if c["form"] == "tree":
        return q, k, v.contiguous()
    s["k"][s["slots"].long()] = k
    s["v"][s["slots"].long()] = v
    return q, s["k"], s["v"]


def _plain_tables(s):
    bs, table = s["case"]["page"], s["block_table"]
    length, new = s["length"].long(), s["new"].long()
    have = (length + bs - 1) // bs
    need = (length + new + bs - 1) // bs - have
    base = torch.cumsum(need, 0) - need + s["head"].long()
    col = torch.arange(table.shape[1], device=table.device)[None, :] - have[:, None]
    fresh = (col >= 0) & (col < need[:, None])
    given = s["free"][torch.where(fresh, base[:, None] + col, 0)]
    table.copy_(torch.where(fresh, given, table))
    start = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    t = torch.arange(s["slots"], device=table.device)
    b = torch.searchsorted(start, t, right=True) - 1
    used = b < len(new)
    b = torch.where(used, b, 0)
    position = length[b] + t - start[b]
    position = torch.where(used, position, -1)
    slot = table[b, torch.where(used, position // bs, 0)].long() * bs + position % bs
    slot = torch.where(used, slot, -1)
    return dict(block_table=table, token_start=start.int(), slots=slot.int(), positions=position.int(),
                free_head=s["head"] + need.sum().int())


# ------------------------------------------------------------- this repository's calls

def _own_window(s):
    import speculative_decoding_verify_sv_gb300 as sv
    c = s["case"]
    if "cache" not in s:  # what a program keeps between steps: the cache's handle, the workspace and the output
        s["cache"] = sv.KVCache(s["k"], s["v"], s["length"], s["block_table"], c["page"] or 16)
        B, N, Hq, D = s["q"].shape
        size = sv.sv_window_attention_workspace_size(s["q"].dtype, B, N, Hq, c["Hkv"], D, s["cache"].max_prefix, c["W"])
        s["workspace"] = torch.zeros(max(size, 16), dtype=torch.uint8, device=s["q"].device)
        s["out"] = torch.empty_like(s["q"])
    return sv.sv_window_attention(s["q"], s["k_tree"], s["v_tree"], s["cache"], s["parent"], s["scale"], c["W"],
                                  sinks=c["S"], out=s["out"], workspace=s["workspace"])


def _own_rope(s):
    import speculative_decoding_verify_sv_gb300 as sv
    c = s["case"]
    if c["form"] == "tree":
        return sv.sv_tree_qk_norm_rope(s["qkv"], c["Hq"], c["Hkv"], s["q_weight"], s["k_weight"], s["inv_freq"], s["length"],
                                       s["parent"], eps=s["eps"], interleaved=c["interleaved"])
    q, k, v = sv.sv_qk_norm_rope(s["qkv"], c["Hq"], c["Hkv"], s["q_weight"], s["k_weight"], s["inv_freq"], s["positions"],
                                 eps=s["eps"], interleaved=c["interleaved"], slots=s["slots"], k_out=s["k"], v_out=s["v"])
    return q, k, v


def _own_tables(s):
    import speculative_decoding_verify_sv_gb300 as sv
    r = sv.sv_block_tables(s["length"], s["new"], s["block_table"], s["free"], s["case"]["page"], s["num_blocks"], s["slots"],
                           free_head=s["head"])
    return dict(block_table=s["block_table"], token_start=r["token_start"], slots=r["slots"], positions=r["positions"],
                free_head=r["free_head"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"window": _own_window, "rope": _own_rope, "tables": _own_tables}[op](state)
    return {"window": _plain_window, "rope": _plain_rope, "tables": _plain_tables}[op](state)


# ---------------------------------------------------------------------------- work

def work(case):
    c = case
    e = 2 if c.get("dtype") == "bf16" else 4
    if c["op"] == "window":
        N, row = len(tree_of(c["tree"])), c["Hkv"] * c["D"] * e
        n = c["hi"] - c["lo"] + 1
        lens = np.arange(c["lo"], c["hi"] + 1, max(1, n // 4096))
        keys = np.minimum(lens, c["W"] - 1) + np.minimum(c["S"], np.maximum(0, lens - c["W"] + 1))
        keys = float(keys.mean()) + N
        return {"bytes": c["B"] * (2 * keys * row + 2 * N * c["Hq"] * c["D"] * e),
                "flops": 4.0 * c["B"] * N * c["Hq"] * c["D"] * keys}
    if c["op"] == "rope":
        T = c["T"] if c["form"] == "slots" else c["B"] * len(tree_of(c["tree"]))
        n = T * (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": 2 * n * e + 8 * T, "flops": 10.0 * n}
    new = c["B"] * (c["new_lo"] + c["new_hi"]) / 2
    pages = new / c["page"]
    return {"bytes": 12.0 * c["B"] + 8 * (c["B"] * c["new_hi"] + 16) + 8 * pages, "flops": 0.0}


# --------------------------------------------------------------- the definition, 64 bits

def _exact_window(s):
    """Row by row of the definition: per sequence, every key of prefix and tree with its mask."""
    c = s["case"]
    B, N, Hq, D = s["q"].shape
    Hkv, W, S = c["Hkv"], c["W"], c["S"]
    out = torch.empty(B, N, Hq, D, dtype=torch.float64, device=s["q"].device)
    for b, L in enumerate(s["length"].tolist()):
        keep = [p for p in range(min(S, L)) if p <= L - W] + list(range(max(0, L - W + 1), L))
        pos = torch.tensor(keep, dtype=torch.long, device=out.device)
        if c["page"]:
            page = s["block_table"][b, pos // c["page"]].long()
            kp, vp = s["k"][page, pos % c["page"]], s["v"][page, pos % c["page"]]
        else:
            kp, vp = s["k"][b, pos], s["v"][b, pos]
        k, v = torch.cat([kp, s["k_tree"][b]]).double(), torch.cat([vp, s["v_tree"][b]]).double()
        where = torch.cat([pos, L + s["depth"]])
        mine = (L + s["depth"])[:, None]
        visible = (where[None, :] > mine - W) | (where[None, :] < S)
        visible[:, len(keep):] &= s["ancestor"]
        head = torch.arange(Hq, device=out.device) // (Hq // Hkv)
        for h in range(Hkv):
            qs = s["q"][b][:, head == h].double()  # [N, G, D]
            x = torch.einsum("ngd,kd->ngk", qs, k[:, h]) * s["scale"]
            x = torch.where(visible[:, None, :], x, torch.full_like(x, -math.inf))
            out[b][:, head == h] = torch.einsum("ngk,kd->ngd", torch.softmax(x, -1), v[:, h])
    return out


def _exact_rope(s):
    c = s["case"]
    Hq, Hkv, D, half = c["Hq"], c["Hkv"], c["D"], c["rot"] // 2
    lead = s["qkv"].shape[:-1]
    x = s["qkv"].reshape(-1, Hq + 2 * Hkv, D).double()
    if c["form"] == "tree":
        position = (s["length"][:, None] + s["depth"][None, :]).reshape(-1)
    else:
        position = s["positions"]
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device), torch.outer(position.double(), s["inv_freq"]))
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    parts = []
    for lo, hi, weight in ((0, Hq, s["q_weight"]), (Hq, Hq + Hkv, s["k_weight"])):
        y = x[:, lo:hi]
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * weight.double()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        parts.append(y)
    q, k, v = parts[0], parts[1], x[:, Hq + Hkv:]
    if c["form"] == "tree":
        return q.reshape(*lead, Hq, D), k.reshape(*lead, Hkv, D), v.reshape(*lead, Hkv, D)
    kc, vc = s["k"].double(), s["v"].double()
    kc[s["slots"].long()], vc[s["slots"].long()] = k, v
    return q, kc, vc


def _exact_tables(s):
    bs = s["case"]["page"]
    table, free = s["block_table"].cpu().numpy().copy(), s["free"].cpu().numpy()
    head, at, start = int(s["head"]), 0, [0]
    slots, positions = np.full(s["slots"], -1, np.int32), np.full(s["slots"], -1, np.int32)
    for b, (length, new) in enumerate(zip(s["length"].tolist(), s["new"].tolist())):
        pages, total = -(-length // bs), -(-(length + new) // bs)
        table[b, pages:total] = free[head:head + max(0, total - pages)]
        head += max(0, total - pages)
        p = np.arange(length, length + new)
        slots[at:at + new], positions[at:at + new] = table[b, p // bs] * bs + p % bs, p
        at += new
        start.append(at)
    return dict(block_table=table, token_start=np.array(start, np.int32), slots=slots, positions=positions,
                free_head=np.array([head], np.int32))


def exact(case, seed):
    s = prepare(case, seed)
    return {"window": _exact_window, "rope": _exact_rope, "tables": _exact_tables}[case["op"]](s)
