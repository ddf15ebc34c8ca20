"""Tree attention over listed pages against its definition in 64 bits."""
import math

import pytest
import torch

import plain_ops
import plain_pages
import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TREES = {"root": [-1], "chain4": wl.chain_parent(4), "t26": wl.TREE_T26, "t64": wl.TREE_T64}


def lists_of(lens, sets, Hkv, K, page, seed, holes=True):
    """Random lists of different pages: ascending, shuffled, with holes, empty."""
    g = torch.Generator().manual_seed(seed)
    out = torch.full((len(lens), sets, Hkv, K), -1, dtype=torch.int32)
    for b, L in enumerate(lens):
        n = -(-L // page)
        for s in range(sets):
            for h in range(Hkv):
                k = min(n, K) if not holes else int(torch.randint(0, min(n, K) + 1, (1,), generator=g))
                at = torch.randperm(n, generator=g)[:k]
                at = at.sort().values if (b + h) % 2 else at
                to = torch.randperm(K, generator=g)[:k] if holes else torch.arange(k)
                out[b, s, h, to] = at.to(torch.int32)
    return out


def padded(inp, pages, page):
    """The same lists with entries behind them that name nothing, so many that calls with more than 48 rows per
    list go through the stacked kernel."""
    B, sets, Hkv, K = pages.shape
    N, Hq, D = inp["q"].shape[1:]
    rows = N * Hq // Hkv
    most = 4000 * torch.cuda.get_device_properties(0).multi_processor_count
    long = -(-most // (B * Hkv * ((rows + 63) // 64) * page))
    out = torch.cat([pages, torch.full((B, sets, Hkv, max(0, long - K)), -1, dtype=torch.int32)], 3)
    assert sv.sv_sparse_attention_workspace_size(BF, B, N, Hq, Hkv, D, page, out.shape[3], 1) > 0
    return out


def stacks(inp, pages):
    return inp["q"].dtype == BF and pages.shape[1] == 1 and inp["q"].shape[1] * inp["q"].shape[2] // pages.shape[2] > 48


def call(inp, parent, pages, page, **kw):
    g = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
    cache = sv.KVCache(g["cache_k"], g["cache_v"], g["prefix_len"], g["block_table"], page)
    par = parent if not isinstance(parent[0], list) else torch.tensor(parent, dtype=torch.int32, device="cuda")
    return sv.sv_sparse_attention(g["q"], g["k_tree"], g["v_tree"], cache, par, g["q"].shape[-1] ** -0.5, pages.cuda(), **kw)


def check(inp, parent, pages, page, **kw):
    """The call, and where there are rows enough the same through the stacked kernel too."""
    outs = [call(inp, parent, p, page, **kw) for p in ([pages, padded(inp, pages, page)] if stacks(inp, pages) else [pages])]
    out = outs[0]
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0
    D = inp["q"].shape[-1]
    lens = inp["prefix_len"].tolist()

    def positions(b, n, h):
        return plain_pages.page_positions(pages[b, n if pages.shape[1] > 1 else 0, h].tolist(), page, lens[b])
    ref, spread = plain_pages.listed_attention(inp["q"], inp["k_tree"], inp["v_tree"], inp["cache_k"], inp["cache_v"],
                                               inp["prefix_len"], parent, D ** -0.5, positions, inp["block_table"], page)
    size = D ** -0.5 * inp["q"].float().norm(dim=-1).max().item() * max(
        inp["k_tree"].float().norm(dim=-1).max().item(), inp["cache_k"].float().norm(dim=-1).max().item())
    bound = plain_ops.attention_bound(ref, spread, inp["q"].dtype, D, size, pages.shape[3] * page + 64)
    for o in outs:
        err = (o.double().cpu() - ref).abs()
        worst = (err - bound).max().item()
        assert bool(torch.isfinite(o).all()) and worst <= 0, (worst, err.max().item())
    return out


LENS = [0, 1, 15, 16, 17, 40, 127, 128, 129, 200, 257, 300]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("per_node", [False, True])
@pytest.mark.parametrize("K", [1, 3, 9])
def test_lists_of_all_lengths(cuda_ok, dtype, paged, per_node, K):
    inp = wl.attention_inputs(len(LENS), 5, 8, 2, 64, LENS, dtype=dtype, paged=paged, seed=K)
    check(inp, wl.chain_parent(4), lists_of(LENS, 5 if per_node else 1, 2, K, 16, K), 16)


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (32, 4), (8, 1), (14, 2), (6, 2), (80, 2)])
@pytest.mark.parametrize("tree", list(TREES))
@pytest.mark.parametrize("paged", [True, False])
def test_trees_and_head_groups(cuda_ok, Hq, Hkv, tree, paged):
    """One to 2560 rows per list: the kernel of few rows, and the stacked one with one or two MMA tiles,
    several row tiles, and groups of heads that do not fill a tile."""
    par = TREES[tree]
    lens = [0, 40, 129, 290]
    inp = wl.attention_inputs(4, len(par), Hq, Hkv, 128, lens, dtype=BF, paged=paged, seed=3)
    check(inp, par, lists_of(lens, 1, Hkv, 12, 16, 4), 16)
    if len(par) in (5, 26) and Hq <= 32:
        check(inp, par, lists_of(lens, len(par), Hkv, 5, 16, 5), 16)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("paged", [True, False])
def test_page_sizes(cuda_ok, page, D, paged):
    lens = [5, 130, 257, 511, 600]
    for parent in (wl.chain_parent(4), wl.TREE_T26):
        inp = wl.attention_inputs(5, len(parent), 8, 2, D, lens, dtype=BF, paged=paged, block_size=page, seed=4)
        check(inp, parent, lists_of(lens, 1, 2, 7, page, page), page)
    inp = wl.attention_inputs(5, 3, 8, 2, D, lens, dtype=F32, paged=paged, block_size=page, seed=4)
    check(inp, wl.chain_parent(2), lists_of(lens, 3, 2, 4, page, page), page)


def test_all_pages_are_tree_attention(cuda_ok):
    """A list of every page gives the whole prefix; one longer than the pages, and the same list backwards."""
    lens = [700, 1003, 64, 333]
    for dtype, parent in ((BF, wl.chain_parent(4)), (BF, wl.TREE_T64), (F32, wl.TREE_EXAMPLE7)):
        inp = wl.attention_inputs(4, len(parent), 16, 4, 128, lens, dtype=dtype, paged=True, seed=6)
        pages = lists_of(lens, 1, 4, 70, 16, 1, holes=False)
        for p in (pages, pages.flip(3)):
            check(inp, parent, p.contiguous(), 16)


def test_a_page_listed_twice_counts_twice(cuda_ok):
    for N in (1, 26):
        parent = [-1] if N == 1 else wl.TREE_T26
        for dtype in (BF, F32):
            inp = wl.attention_inputs(2, N, 8, 2, 64, [100, 170], dtype=dtype, paged=True, seed=7)
            pages = torch.tensor([3, 1, 3, 0, 3, -1, 1], dtype=torch.int32).expand(2, 1, 2, 7).contiguous()
            check(inp, parent, pages, 16)


def test_entries_that_name_no_keys(cuda_ok):
    """Negative entries, pages behind the prefix and far past any table."""
    for N, dtype in ((1, BF), (26, BF), (3, F32)):
        parent = wl.TREE_T26 if N == 26 else wl.chain_parent(N - 1)
        inp = wl.attention_inputs(2, N, 8, 2, 128, [100, 96], dtype=dtype, paged=True, seed=8)
        pages = torch.tensor([7, 6, 2 ** 31 - 1, -2 ** 31, 2, -7, 100000], dtype=torch.int32).expand(2, 1, 2, 7).contiguous()
        check(inp, parent, pages, 16)
        none = torch.full((2, 1, 2, 3), -1, dtype=torch.int32)
        check(inp, parent, none, 16)


@pytest.mark.parametrize("paged", [True, False])
def test_long_lists_cut_over_many_ctas(cuda_ok, paged):
    inp = wl.attention_inputs(1, 26, 8, 1, 128, [9001], dtype=BF, paged=paged, seed=9)
    check(inp, wl.TREE_T26, lists_of([9001], 1, 1, 500, 16, 9, holes=False), 16)
    inp = wl.attention_inputs(4, 26, 16, 2, 64, [5003, 4801, 7, 4090], dtype=BF, paged=paged, seed=11)
    check(inp, wl.TREE_T26, lists_of([5003, 4801, 7, 4090], 1, 2, 300, 16, 12), 16)
    inp = wl.attention_inputs(2, 1, 8, 2, 128, [5000, 4100], dtype=BF, paged=paged, seed=10)
    check(inp, [-1], lists_of([5000, 4100], 1, 2, 256, 16, 10), 16)


def test_trees_of_each_sequence(cuda_ok):
    g = torch.Generator().manual_seed(6)
    parents = [[-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, 13)] for _ in range(4)]
    lens = [0, 64, 129, 300]
    for dtype, per_node in ((BF, False), (BF, True), (F32, True)):
        inp = wl.attention_inputs(4, 13, 8, 2, 128, lens, dtype=dtype, seed=7)
        check(inp, parents, lists_of(lens, 13 if per_node else 1, 2, 6, 16, 11), 16)


@pytest.mark.parametrize("N,stacked", [(2, False), (26, False), (26, True)])
def test_what_is_not_listed_may_hold_anything(cuda_ok, N, stacked):
    """NaN and infinity in unlisted pages and behind the prefix's end, and blocks that are no blocks."""
    parent = wl.TREE_T26 if N == 26 else wl.chain_parent(1)
    lens = [100, 250]
    inp = wl.attention_inputs(2, N, 8, 2, 128, lens, dtype=BF, paged=True, seed=12)
    pages = torch.full((2, 1, 2, 5), -1, dtype=torch.int32)
    pages[0, 0, :, :3] = torch.tensor([0, 6, 2], dtype=torch.int32)
    pages[1, 0, :, :4] = torch.tensor([15, 3, 8, 1], dtype=torch.int32)
    check(inp, parent, pages, 16)
    if stacked:
        pages = padded(inp, pages, 16)
    clean = call(inp, parent, pages, 16)
    for b, kept in ((0, [0, 2, 6]), (1, [1, 3, 8, 15])):
        for j in range(inp["block_table"].shape[1]):
            blk = int(inp["block_table"][b, j])
            if blk < 0:
                continue
            if j not in kept:
                inp["cache_k"][blk], inp["cache_v"][blk] = math.nan, math.inf
                inp["block_table"][b, j] = [-1, 10 ** 9][j % 2]
            elif (j + 1) * 16 > lens[b]:
                inp["cache_k"][blk, lens[b] % 16:], inp["cache_v"][blk, lens[b] % 16:] = math.inf, math.nan
    out = call(inp, parent, pages, 16)
    assert torch.equal(out, clean) and sv.sv_read_device_status() == 0


@pytest.mark.parametrize("N,dtype,stacked", [(2, BF, False), (26, BF, False), (26, BF, True), (2, F32, False)])
def test_bad_pages_are_left_out(cuda_ok, N, dtype, stacked):
    parent = wl.TREE_T26 if N == 26 else wl.chain_parent(1)
    inp = wl.attention_inputs(2, N, 8, 2, 128, [100, 250], dtype=dtype, paged=True, seed=13)
    pages = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32).expand(2, 1, 2, 5).contiguous()
    less = torch.tensor([0, -1, 2, -1, 4], dtype=torch.int32).expand(2, 1, 2, 5).contiguous()
    if stacked:
        pages, less = padded(inp, pages, 16), padded(inp, less, 16)
    want = call(inp, parent, less, 16)
    assert sv.sv_read_device_status() == 0
    inp["block_table"][:, 1], inp["block_table"][:, 3] = -1, inp["num_blocks"]
    got = call(inp, parent, pages, 16)
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
    assert torch.equal(got, want)


def test_prefix_outside_the_cache_is_clamped(cuda_ok):
    for N, stacked in ((1, False), (26, False), (26, True)):
        parent = wl.TREE_T26 if N == 26 else [-1]
        inp = wl.attention_inputs(2, N, 8, 2, 64, [96, 96], dtype=BF, paged=True, extra=0, seed=14)
        pages = torch.arange(6, dtype=torch.int32).expand(2, 1, 2, 6).contiguous()
        if stacked:
            pages = padded(inp, pages, 16)
        want = call(inp, parent, pages, 16)
        inp["prefix_len"][0] = 10 ** 6
        got = call(inp, parent, pages, 16)
        assert torch.equal(got, want) and sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
        inp["prefix_len"][0] = -4
        call(inp, parent, pages, 16)
        assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
