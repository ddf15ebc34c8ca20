"""Calls of so many units that each is a warp's: listed pages and own keys behind shared ones, with the masks,
lengths and bad entries of the few-unit tests."""
import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv
import test_gpu_shared_attention as shared
import test_gpu_sparse_attention as sparse
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def batch(units_each):
    """Sequences enough for four units per SM."""
    return -(-4 * torch.cuda.get_device_properties(0).multi_processor_count // units_each)


@pytest.mark.parametrize("N,Hq,Hkv,D,per_node", [(1, 8, 8, 64, False), (1, 64, 8, 128, False), (5, 32, 8, 128, True), (5, 32, 8, 128, False),
                                                 (7, 28, 4, 64, False), (64, 16, 8, 128, False), (13, 16, 2, 64, True)])
@pytest.mark.parametrize("paged", [True, False])
def test_listed_units(cuda_ok, N, Hq, Hkv, D, per_node, paged):
    B = batch(Hkv * (N if per_node else 1))
    lens = [(0, 1, 15, 16, 17, 40, 129, 200)[i % 8] for i in range(B)]
    par = wl.TREE_T64 if N == 64 else wl.chain_parent(N - 1)
    inp = wl.attention_inputs(B, N, Hq, Hkv, D, lens, dtype=BF, paged=paged, seed=N)
    pages = sparse.lists_of(lens, N if per_node else 1, Hkv, 4, 16, N)
    pages[0, 0, 0] = torch.tensor([2 ** 31 - 1, -2 ** 31, 7, -1], dtype=torch.int32)
    sparse.check(inp, par, pages, 16)


def test_listed_units_with_bad_pages_and_prefixes(cuda_ok):
    B = batch(8)
    inp = wl.attention_inputs(B, 2, 16, 8, 128, [100] * B, dtype=BF, paged=True, seed=1)
    pages = torch.tensor([0, 1, 2, 3, 6], dtype=torch.int32).expand(B, 1, 8, 5).contiguous()
    less = torch.tensor([0, -1, 2, -1, 6], dtype=torch.int32).expand(B, 1, 8, 5).contiguous()
    want = sparse.call(inp, [-1, 0], less, 16)
    assert sv.sv_read_device_status() == 0
    inp["block_table"][:, 1], inp["block_table"][:, 3] = -1, inp["num_blocks"]
    got = sparse.call(inp, [-1, 0], pages, 16)
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK and torch.equal(got, want)
    inp["prefix_len"][3] = -7
    got = sparse.call(inp, [-1, 0], less, 16)
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
    assert torch.equal(got[:3], want[:3]) and torch.equal(got[4:], want[4:])


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 8, 8, 64), (1, 64, 8, 128), (5, 32, 8, 128), (7, 28, 4, 64), (26, 8, 8, 128)])
@pytest.mark.parametrize("page", [0, 16, 48])
def test_joined_units(cuda_ok, N, Hq, Hkv, D, page):
    B = batch(Hkv)
    sizes = [B // 3, 1, B - B // 3 - 1]
    own = [(0, 1, 2, 15, 16, 17, 40)[i % 7] for i in range(B)]
    par = wl.TREE_T26 if N == 26 else wl.chain_parent(N - 1)
    shared.check(shared.shared_inputs(sizes, [130, 0, 177], own, N, Hq, Hkv, D, page=page, seed=N), par, page)


def test_joined_units_of_bad_groups(cuda_ok):
    B = batch(8)
    inp = shared.shared_inputs([B // 2, B - B // 2], [64, 40], [3] * B, 2, 16, 8, 64, seed=5)
    for starts, status in (([0, B, 3], sv.SV_DEV_BAD_GROUP), ([0, 1, 1], 0)):
        inp["group_start"] = torch.tensor(starts, dtype=torch.int32)
        shared.check(inp, [-1, 0], status=status)


def test_trees_of_each_sequence(cuda_ok):
    B = batch(8)
    g = torch.Generator().manual_seed(6)
    parents = [[-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, 6)] for _ in range(B)]
    shared.check(shared.shared_inputs([B], [33], [i % 20 for i in range(B)], 6, 16, 8, 64, seed=7), parents)
    lens = [i % 70 for i in range(B)]
    inp = wl.attention_inputs(B, 6, 16, 8, 64, lens, dtype=BF, seed=7)
    sparse.check(inp, parents, sparse.lists_of(lens, 1, 8, 3, 16, 11), 16)


@pytest.mark.parametrize("N,Hq,Hkv,D,per_node", [(64, 4, 4, 64, True), (26, 8, 8, 128, True), (5, 16, 4, 64, True), (5, 32, 4, 128, True),
                                                 (1, 8, 8, 128, False), (33, 3, 3, 64, False)])
@pytest.mark.parametrize("paged", [True, False])
def test_listed_units_of_float32(cuda_ok, N, Hq, Hkv, D, per_node, paged):
    """CTAs of two warps, of which several share an SM, each with one to eight rows."""
    B = batch(2 * Hkv * (N if per_node else 1)) if N > 1 else batch(Hkv)
    lens = [(0, 1, 15, 16, 17, 40, 29, 33)[i % 8] for i in range(B)]
    par = wl.TREE_T64 if N == 64 else wl.TREE_T26 if N == 26 else wl.chain_parent(N - 1)
    inp = wl.attention_inputs(B, N, Hq, Hkv, D, lens, dtype=torch.float32, paged=paged, seed=N)
    sparse.check(inp, par, sparse.lists_of(lens, N if per_node else 1, Hkv, 2, 16, N), 16)
