"""The stacked attention kernel where a tile of 128 rows is not full: what its other rows hold (other sequences' queries, or
what an earlier call left in shared memory) changes nothing, not the rounding either."""
import math

import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv
import test_gpu_shared_attention as shared
import test_gpu_sparse_attention as sparse
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


class Calls:
    """Both attentions over one cache, as their stacked forms take it."""

    def __init__(self, N, G, Hkv, D, page, seed=1):
        B = 3
        self.parent = wl.TREE_T64[:N] if N > 1 else [-1]
        inp = shared.shared_inputs([B], [600], [300, 0, 77], N, G * Hkv, Hkv, D, page=page, seed=seed)
        pages = sparse.padded(inp, sparse.lists_of(inp["prefix_len"].tolist(), 1, Hkv, 40, page or 16, seed), page or 16)
        inp = shared.roomy(inp, page)
        self.g = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
        # (scores that move the running maximum by more than the kernel lets it lag behind, now and then)
        self.g["cache_k"] *= 1 + 3 * torch.rand(self.g["cache_k"].shape[:2], generator=torch.Generator().manual_seed(seed)).to(BF).cuda()[..., None, None]
        g = self.g
        self.cache = sv.KVCache(g["cache_k"], g["cache_v"], g["prefix_len"], g["block_table"], page or 16)
        self.pages = pages.cuda()

    def sparse(self, q):
        g = self.g
        return sv.sv_sparse_attention(q, g["k_tree"], g["v_tree"], self.cache, self.parent, 0.1, self.pages)

    def shared(self, q):
        g = self.g
        return sv.sv_shared_attention(q, g["k_tree"], g["v_tree"], self.cache, self.parent, 0.1, g["group_start"], g["shared_len"])


SHAPES = [(64, 3, 2, 64, 16), (64, 5, 3, 64, 256), (26, 12, 2, 128, 16), (13, 40, 2, 128, 64), (5, 100, 2, 128, 16), (33, 7, 4, 128, 0),
          (64, 12, 1, 64, 0)]


@pytest.mark.parametrize("N,G,Hkv,D,page", SHAPES)
def test_what_earlier_calls_left_behind(cuda_ok, N, G, Hkv, D, page):
    c = Calls(N, G, Hkv, D, page)
    q = c.g["q"]
    for call in (c.sparse, c.shared):
        first = call(q)
        for k, other in enumerate((q * 16, torch.full_like(q, math.nan), -q * 5, q.flip(0) * 30, torch.zeros_like(q))):
            for way in (c.sparse, c.shared) if k % 2 else (c.shared, c.sparse):
                way(other)
            assert torch.equal(call(q), first), k
    assert bool(first.isfinite().all()) and sv.sv_read_device_status() == 0


@pytest.mark.parametrize("N,G,Hkv,D,page", SHAPES + [(64, 4, 2, 128, 16), (17, 4, 2, 64, 16)])
def test_the_next_sequences_queries(cuda_ok, N, G, Hkv, D, page):
    """A list is one sequence's: the rows behind its last one are the next sequence's, or none."""
    c = Calls(N, G, Hkv, D, page, seed=2)
    q = c.g["q"]
    first = c.sparse(q)
    for b in range(3):
        for factor in (30.0, math.nan):
            other = torch.cat([q[i:i + 1] * (1.0 if i == b else factor) for i in range(3)])
            assert torch.equal(c.sparse(other)[b], first[b]), (b, factor)
    assert sv.sv_read_device_status() == 0
