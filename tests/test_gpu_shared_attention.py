"""Tree attention of sequences that share prefixes against its definition in 64 bits."""
import math

import pytest
import torch

import plain_ops
import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def shared_inputs(sizes, shared, own, N, Hq, Hkv, D, dtype=BF, page=16, seed=0, extra=8):
    """Groups of `sizes` sequences that share `shared` positions, with `own` further ones each; `page` 0: a
    contiguous cache.  The whole pages of a shared prefix are the group's first sequence's."""
    B = sum(sizes)
    group = [g for g, n in enumerate(sizes) for _ in range(n)]
    lens = [shared[g] + own[b] for b, g in enumerate(group)]
    inp = wl.attention_inputs(B, N, Hq, Hkv, D, lens, dtype=dtype, paged=page > 0, block_size=page or 16, extra=extra, seed=seed)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + n)
    for b, g in enumerate(group):
        a, n = starts[g], shared[g]
        if a == b:
            continue
        if page:
            whole = n // page
            inp["block_table"][b, :whole] = inp["block_table"][a, :whole]
            if n % page:
                for t in ("cache_k", "cache_v"):
                    inp[t][int(inp["block_table"][b, whole]), :n % page] = inp[t][int(inp["block_table"][a, whole]), :n % page]
        else:
            for t in ("cache_k", "cache_v"):
                inp[t][b, :n] = inp[t][a, :n]
    inp["group_start"] = torch.tensor(starts, dtype=torch.int32)
    inp["shared_len"] = torch.tensor(shared, dtype=torch.int32)
    return inp


def roomy(inp, page):
    """The same sequences in a cache with room for so many positions that bf16 calls go through the stacked kernel."""
    B, N, Hq, D = inp["q"].shape
    Hkv = inp["k_tree"].shape[2]
    most = 2000 * torch.cuda.get_device_properties(0).multi_processor_count
    cap = max(256, -(-most // (B * Hkv * ((N * Hq // Hkv + 63) // 64))))
    out = dict(inp)
    if page:
        have = inp["block_table"].shape[1]
        out["block_table"] = torch.cat([inp["block_table"], torch.full((B, max(0, -(-cap // page) - have)), -1, dtype=torch.int32)], 1)
        cap = out["block_table"].shape[1] * page
    else:
        more = max(0, cap - inp["cache_k"].shape[1])
        for t in ("cache_k", "cache_v"):
            out[t] = torch.cat([inp[t], torch.full((B, more, Hkv, D), math.nan, dtype=inp[t].dtype)], 1)
        cap = out["cache_k"].shape[1]
    assert sv.sv_shared_attention_workspace_size(BF, B, N, Hq, Hkv, D, cap, inp["shared_len"].numel()) > 0
    return out


def call(inp, parent, page=16, **kw):
    g = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
    cache = sv.KVCache(g["cache_k"], g["cache_v"], g["prefix_len"], g["block_table"], page or 16)
    par = parent if not isinstance(parent[0], list) else torch.tensor(parent, dtype=torch.int32, device="cuda")
    return sv.sv_shared_attention(g["q"], g["k_tree"], g["v_tree"], cache, par, g["q"].shape[-1] ** -0.5, g["group_start"],
                                  g["shared_len"], **kw)


def check(inp, parent, page=16, status=0):
    """The call, and in bf16 the same through the stacked kernel, whose result is returned."""
    outs = []
    for x in ([inp, roomy(inp, page)] if inp["q"].dtype == BF else [inp]):
        outs.append(call(x, parent, page))
        torch.cuda.synchronize()
        assert sv.sv_read_device_status() == status
    D = inp["q"].shape[-1]
    ref, spread = plain_ops.window_attention(inp["q"], inp["k_tree"], inp["v_tree"], inp["cache_k"], inp["cache_v"],
                                             inp["prefix_len"], parent, D ** -0.5, 2 ** 31, 0, inp["block_table"], page or 16)
    size = D ** -0.5 * inp["q"].float().norm(dim=-1).max().item() * max(
        inp["k_tree"].float().norm(dim=-1).max().item(), inp["cache_k"].float().norm(dim=-1).max().item())
    bound = plain_ops.attention_bound(ref, spread, inp["q"].dtype, D, size, int(inp["prefix_len"].max()) + 64)
    for out in outs:
        err = (out.double().cpu() - ref).abs()
        worst = (err - bound).max().item()
        assert bool(torch.isfinite(out).all()) and worst <= 0, (worst, err.max().item())
    return out


@pytest.mark.parametrize("shared", [0, 1, 15, 16, 17, 127, 128, 130, 255, 256, 257, 400])
@pytest.mark.parametrize("page", [0, 16])
def test_shared_lengths(cuda_ok, shared, page):
    own = [0, 1, 2, 15, 16, 17, 40]
    check(shared_inputs([7], [shared], own, 5, 8, 2, 64, page=page, seed=shared), wl.chain_parent(4), page)


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (32, 4), (8, 1), (14, 2), (6, 2), (80, 2)])
@pytest.mark.parametrize("tree", ["root", "chain4", "t26", "t64"])
def test_trees_and_head_groups(cuda_ok, Hq, Hkv, tree):
    """One to many row tiles, groups of heads that fill a tile and that do not."""
    par = {"root": [-1], "chain4": wl.chain_parent(4), "t26": wl.TREE_T26, "t64": wl.TREE_T64}[tree]
    check(shared_inputs([3, 1], [200, 131], [0, 9, 33, 70], len(par), Hq, Hkv, 128, seed=3), par)


@pytest.mark.parametrize("page", [0, 16, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(cuda_ok, page, D):
    check(shared_inputs([4, 2], [300, 77], [1, 0, 20, 61, 5, 130], 5, 8, 2, D, page=page, seed=4), wl.chain_parent(4), page)


def test_many_groups(cuda_ok):
    """Empty groups, groups of one, groups without a shared prefix, sequences outside any group."""
    sizes, shared = [2, 1, 3, 1, 5, 2], [160, 300, 0, 16, 144, 513]
    own = [(7 * i) % 50 for i in range(sum(sizes))]
    inp = shared_inputs(sizes, shared, own, 3, 8, 4, 128, seed=5)
    check(inp, wl.chain_parent(2))
    # an empty group in the middle, and only some of the sequences in groups
    inp["group_start"] = torch.tensor([2, 3, 3, 6, 7], dtype=torch.int32)
    inp["shared_len"] = torch.tensor([300, 199, 0, 16], dtype=torch.int32)
    check(inp, wl.chain_parent(2))


def test_the_most_groups(cuda_ok):
    sizes, shared = [1] * 128, [(37 * i) % 90 for i in range(128)]
    check(shared_inputs(sizes, shared, [3] * 128, 1, 4, 2, 64, seed=6), [-1])


@pytest.mark.parametrize("page", [0, 16])
def test_units_cut_over_many_ctas(cuda_ok, page):
    """One KV head with a long shared prefix: its key tiles are split and joined again."""
    check(shared_inputs([3], [9001], [0, 12, 300], 5, 8, 1, 128, page=page, seed=8), wl.chain_parent(4), page)
    check(shared_inputs([40], [2500], list(range(40)), 26, 8, 2, 128, page=page, seed=9), wl.TREE_T26, page)


def test_trees_of_each_sequence(cuda_ok):
    g = torch.Generator().manual_seed(6)
    parents = [[-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, 13)] for _ in range(5)]
    check(shared_inputs([5], [150], [0, 3, 20, 90, 17], 13, 8, 2, 128, seed=7), parents)


def test_float32(cuda_ok):
    inp = shared_inputs([3, 2], [130, 64], [0, 9, 33, 70, 1], 5, 8, 2, 64, dtype=F32, seed=10)
    check(inp, wl.chain_parent(4))


def test_large_scores(cuda_ok):
    """Scores that grow along the prefix, so that the running maximum moves at every tile."""
    inp = shared_inputs([4], [1000], [5, 6, 7, 8], 5, 8, 2, 128, page=0, seed=11)
    q = inp["q"].float()
    q[:] = q[:1, :1, :1]
    k = inp["cache_k"].float()
    k[:, :1000] = k[:1, :1000] + q[0, 0, 0] * torch.linspace(-3, 9, 1000)[None, :, None, None]
    inp["q"], inp["cache_k"] = q.to(BF), k.to(BF)
    check(inp, wl.chain_parent(4), 0)


def test_what_no_row_sees_may_hold_anything(cuda_ok):
    """NaN behind the ends of the prefixes, which the last tiles of the shared part read past."""
    for page in (0, 16):
        inp = shared_inputs([3], [200], [0, 5, 33], 5, 8, 2, 128, page=page, seed=12)
        clean = check(inp, wl.chain_parent(4), page)
        for b, L in enumerate(inp["prefix_len"].tolist()):
            if page:
                for p in range(L, inp["block_table"].shape[1] * 16):
                    blk = int(inp["block_table"][b, p // 16])
                    if blk >= 0:
                        inp["cache_k"][blk, p % 16], inp["cache_v"][blk, p % 16] = math.nan, math.inf
            else:
                inp["cache_k"][b, L:], inp["cache_v"][b, L:] = math.inf, math.nan
        out = call(roomy(inp, page), wl.chain_parent(4), page)
        assert torch.equal(out, clean) and sv.sv_read_device_status() == 0
        assert bool(call(inp, wl.chain_parent(4), page).isfinite().all()) and sv.sv_read_device_status() == 0


def test_bad_groups_share_nothing(cuda_ok):
    inp = shared_inputs([3, 2], [200, 100], [0, 5, 33, 8, 9], 5, 8, 2, 128, seed=13)
    for starts in ([0, 3, 2], [-1, 3, 5], [0, 3, 6], [4, 3, 5], [0, 2 ** 31 - 1, 5]):
        inp["group_start"] = torch.tensor(starts, dtype=torch.int32)
        check(inp, wl.chain_parent(4), status=sv.SV_DEV_BAD_GROUP)


def test_shared_lengths_outside_the_cache(cuda_ok):
    inp = shared_inputs([3, 2], [200, 100], [0, 5, 33, 8, 9], 5, 8, 2, 128, seed=14)
    inp["shared_len"] = torch.tensor([200, -5], dtype=torch.int32)  # (as 0)
    check(inp, wl.chain_parent(4), status=sv.SV_DEV_BAD_PREFIX)
    # beyond a member's prefix: that sequence alone is off
    for room in (False, True):
        inp["shared_len"] = torch.tensor([200, 112], dtype=torch.int32)
        inp["prefix_len"][3] = 100
        out = call(roomy(inp, 16) if room else inp, wl.chain_parent(4))
        assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
        inp["shared_len"] = torch.tensor([200, 0], dtype=torch.int32)
        want = call(roomy(inp, 16) if room else inp, wl.chain_parent(4))
        assert sv.sv_read_device_status() == 0
        assert torch.equal(out[:3], want[:3])


@pytest.mark.parametrize("room", [True, False])
def test_bad_pages_of_the_shared_part_are_left_out(cuda_ok, room):
    """Reported; the keys of the page are no keys of the group's sequences."""
    inp = shared_inputs([3], [192], [0, 5, 33], 5, 8, 2, 128, seed=15)
    inp["block_table"][:, 4] = inp["num_blocks"] + 7
    out = call(roomy(inp, 16) if room else inp, wl.chain_parent(4))
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
    keep = [j for j in range(inp["block_table"].shape[1]) if j != 4]
    inp["block_table"] = inp["block_table"][:, keep].contiguous()
    inp["prefix_len"] -= 16
    inp["shared_len"] -= 16
    want = check(inp, wl.chain_parent(4))
    # the same keys in other tiles: weights rounded against another maximum, 2^-8 of sum(p |v|) <= 4 each
    # way, and the results to bf16
    assert (out.float() - want.float()).abs().max() <= 4 * 2 * 2 ** -8 + 4 * 2 ** -8
