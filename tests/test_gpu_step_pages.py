"""Verify steps whose attention works on shared prefixes once, or on selected pages: the step's calls together,
step after step, against the definitions of each."""
import pytest
import torch

import plain_pages
import speculative_decoding_verify_sv_gb300 as sv
import test_gpu_shared_attention as shared
import test_gpu_sparse_attention as sparse
from speculative_decoding_verify_sv_gb300 import workloads as wl
from speculative_decoding_verify_sv_gb300.step import SparsePages, VerifyStep

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
V = 512


def step_inputs(B, N, Hq, Hkv, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(B, N, h, D, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
    logits = torch.randn(B, N, V, generator=g)
    tokens = torch.randint(0, V, (B, N), generator=g).to(torch.int32)
    for b in range(B):  # some drafts are what the target wants
        for n in range(1, N):
            if (b + n + seed) % 3:
                logits[b, n - 1, tokens[b, n]] = 20.0
    return q, k, v, logits.to(dtype), tokens


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("per_node,parent,Hq,Hkv", [(False, wl.chain_parent(4), 8, 2), (True, wl.chain_parent(4), 8, 2),
                                                    (False, wl.TREE_T26, 16, 4), (True, [-1], 4, 4)])
def test_sparse_steps(cuda_ok, dtype, paged, per_node, parent, Hq, Hkv):
    """Bounds, scores, selection, attention, acceptance with the commit, and the bounds again."""
    lens, N, D = [0, 30, 100, 257, 330], len(parent), 64
    inp = wl.attention_inputs(5, N, Hq, Hkv, D, lens, dtype=dtype, paged=paged, extra=N * 3, seed=2)
    cache = sv.KVCache(inp["cache_k"].cuda(), inp["cache_v"].cuda(), inp["prefix_len"].cuda(),
                       inp["block_table"].cuda() if paged else None, 16)
    table = inp["block_table"] if paged else None
    step = VerifyStep(parent, 5, Hq, Hkv, D, V, cache, dtype=dtype, mode=sv.GREEDY, sparse=SparsePages(6, 1, 2, per_node))
    step.reset_bounds()
    for rnd in range(4):
        before = cache.prefix_len.cpu()
        q, k, v, logits, tokens = step_inputs(5, N, Hq, Hkv, D, dtype, rnd)
        bounds = step.bounds.cpu()
        want = plain_pages.page_bounds(bounds, cache.k.cpu(), before, None, table, 16)
        assert torch.equal(bounds, want)  # (those of the cache's pages are up to date)
        n0 = sv.sv_kernel_launches()
        out, outs = step.run(q.cuda(), k.cuda(), v.cuda(), logits.cuda(), None, tokens.cuda())
        assert sv.sv_kernel_launches() - n0 == step.kernel_launches()
        torch.cuda.synchronize()
        assert sv.sv_read_device_status() == 0
        assert torch.equal(cache.prefix_len.cpu(), before + outs["num_accepted"].cpu() + 1)
        pages = plain_pages.select_pages(step.scores.cpu(), before, 16, 6, 1, 2)
        assert torch.equal(step.pages.cpu(), pages)
        now = {"q": q, "k_tree": k, "v_tree": v, "cache_k": cache.k.cpu(), "cache_v": cache.v.cpu(), "prefix_len": before,
               "block_table": table}
        assert torch.equal(sparse.check(now, parent, pages, 16), out)
    assert int((cache.prefix_len.cpu() - inp["prefix_len"]).max()) >= 4


@pytest.mark.parametrize("dtype,room", [(BF, False), (BF, True), (F32, False)])
@pytest.mark.parametrize("parent", [wl.chain_parent(4), wl.TREE_T26])
def test_shared_steps(cuda_ok, dtype, room, parent):
    """Two groups behind prompts of their own, step after step."""
    N, Hq, Hkv, D = len(parent), 8, 2, 64
    inp = shared.shared_inputs([3, 2], [130, 64], [0, 9, 33, 70, 1], N, Hq, Hkv, D, dtype=dtype, seed=10, extra=N * 3)
    if room:
        inp = shared.roomy(inp, 16)
    cache = sv.KVCache(inp["cache_k"].cuda(), inp["cache_v"].cuda(), inp["prefix_len"].cuda(), inp["block_table"].cuda(), 16)
    group = (inp["group_start"].cuda(), inp["shared_len"].cuda())
    step = VerifyStep(parent, 5, Hq, Hkv, D, V, cache, dtype=dtype, mode=sv.GREEDY, shared=group)
    for rnd in range(3):
        before = cache.prefix_len.cpu()
        q, k, v, logits, tokens = step_inputs(5, N, Hq, Hkv, D, dtype, rnd)
        n0 = sv.sv_kernel_launches()
        out, outs = step.run(q.cuda(), k.cuda(), v.cuda(), logits.cuda(), None, tokens.cuda())
        assert sv.sv_kernel_launches() - n0 == step.kernel_launches()
        torch.cuda.synchronize()
        assert sv.sv_read_device_status() == 0
        assert torch.equal(cache.prefix_len.cpu(), before + outs["num_accepted"].cpu() + 1)
        now = {"q": q, "k_tree": k, "v_tree": v, "cache_k": cache.k.cpu(), "cache_v": cache.v.cpu(), "prefix_len": before,
               "block_table": inp["block_table"], "group_start": inp["group_start"], "shared_len": inp["shared_len"]}
        shared.check(now, parent)
        assert torch.equal(shared.call(now, parent), out)


@pytest.mark.parametrize("kind", ["shared", "stacked", "sparse"])
def test_captured_steps_follow_the_lengths(cuda_ok, kind):
    """A step captured once and replayed: prefix lengths, bounds and pages move on by themselves."""
    parent, Hq, Hkv, D = wl.chain_parent(4), 8, 2, 64
    N = len(parent)

    def make():
        inp = shared.shared_inputs([3, 2], [130, 64], [0, 9, 33, 70, 1], N, Hq, Hkv, D, seed=10, extra=N * 4)
        if kind == "stacked":
            inp = shared.roomy(inp, 16)
        cache = sv.KVCache(inp["cache_k"].cuda(), inp["cache_v"].cuda(), inp["prefix_len"].cuda(), inp["block_table"].cuda(), 16)
        kw = dict(shared=(inp["group_start"].cuda(), inp["shared_len"].cuda())) if kind != "sparse" else dict(sparse=SparsePages(5))
        step = VerifyStep(parent, 5, Hq, Hkv, D, V, cache, mode=sv.GREEDY, **kw)
        if kind == "sparse":
            step.reset_bounds()
        return step, cache

    eager, cache = make()
    replayed, other = make()
    ins = [t.cuda() for t in step_inputs(5, N, Hq, Hkv, D, BF, 0)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        saved = [t.clone() for t in (other.k, other.v, other.prefix_len)]
        replayed.run(ins[0], ins[1], ins[2], ins[3], None, ins[4], stream=stream)  # (not captured: the kernels load)
        stream.synchronize()
        for t, s in zip((other.k, other.v, other.prefix_len), saved):
            t.copy_(s)
        if kind == "sparse":
            replayed.reset_bounds(stream)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            replayed.run(ins[0], ins[1], ins[2], ins[3], None, ins[4])
    for rnd in range(3):
        for to, t in zip(ins, step_inputs(5, N, Hq, Hkv, D, BF, rnd)):
            to.copy_(t)
        graph.replay()
        out, outs = eager.run(ins[0], ins[1], ins[2], ins[3], None, ins[4])
        torch.cuda.synchronize()
        assert torch.equal(replayed.out, out) and torch.equal(other.prefix_len, cache.prefix_len)
        assert torch.equal(other.k, cache.k) and torch.equal(replayed.outs["tokens"], outs["tokens"])
    assert sv.sv_read_device_status() == 0


def test_one_kind_of_attention_at_a_time(cuda_ok):
    cache = sv.KVCache(*(torch.zeros(2, 64, 2, 64, dtype=BF, device="cuda") for _ in "kv"),
                       torch.zeros(2, dtype=torch.int32, device="cuda"))
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    for kw in (dict(window=16, sparse=SparsePages(2)), dict(shared=(one, one), sparse=SparsePages(2)), dict(window=16, shared=(one, one))):
        with pytest.raises(ValueError):
            VerifyStep([-1], 2, 4, 2, 64, V, cache, **kw)
