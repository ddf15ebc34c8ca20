"""The bounds that a verify step over selected pages keeps: there before the first selection, whether or not they were
asked for, and renewed for one sequence of the batch alone."""
import pytest
import torch

import plain_pages
import speculative_decoding_verify_sv_gb300 as sv
import test_gpu_sparse_attention as sparse
import test_gpu_step_pages as steps
from speculative_decoding_verify_sv_gb300 import workloads as wl
from speculative_decoding_verify_sv_gb300.step import SparsePages, VerifyStep

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
B, Hq, Hkv, D, PARENT = 5, 8, 2, 64, wl.chain_parent(4)
N = len(PARENT)


def make(dtype, paged, seed=2, lens=(0, 30, 100, 257, 330)):
    inp = wl.attention_inputs(B, N, Hq, Hkv, D, list(lens), dtype=dtype, paged=paged, extra=N * 4, seed=seed)
    cache = sv.KVCache(inp["cache_k"].cuda(), inp["cache_v"].cuda(), inp["prefix_len"].cuda(),
                       inp["block_table"].cuda() if paged else None, 16)
    step = VerifyStep(PARENT, B, Hq, Hkv, D, steps.V, cache, dtype=dtype, mode=sv.GREEDY, sparse=SparsePages(4, 1, 1))
    return inp, cache, step


def run_and_check(step, cache, table, dtype, seed):
    """A step against the definitions of its parts, from the cache as it is."""
    before = cache.prefix_len.cpu()
    q, k, v, logits, tokens = steps.step_inputs(B, N, Hq, Hkv, D, dtype, seed)
    kc, vc = cache.k.cpu(), cache.v.cpu()
    out, _ = step.run(q.cuda(), k.cuda(), v.cuda(), logits.cuda(), None, tokens.cuda())
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0
    rows = torch.zeros_like(step.bounds.cpu())
    bounds = plain_pages.page_bounds(rows, kc, before, None, table, 16)
    ref, size = plain_pages.page_scores(q, bounds, before, 16, table)
    # (sums of 2 D products in fp32, each rounded to half a step of 2^-23 and less)
    err = (step.scores.double().cpu() - ref).abs().nan_to_num()
    assert bool((err <= (2 * D + 2) * 2.0 ** -23 * size).all())
    pages = plain_pages.select_pages(step.scores.cpu(), before, 16, 4, 1, 1)
    assert torch.equal(step.pages.cpu(), pages)
    now = {"q": q, "k_tree": k, "v_tree": v, "cache_k": kc, "cache_v": vc, "prefix_len": before, "block_table": table}
    assert torch.equal(sparse.check(now, PARENT, pages, 16), out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("paged", [True, False])
def test_prompts_in_the_cache_are_looked_at_without_being_asked_for(cuda_ok, dtype, paged):
    inp, cache, step = make(dtype, paged)
    for seed in range(3):
        run_and_check(step, cache, inp["block_table"] if paged else None, dtype, seed)
    assert int((cache.prefix_len.cpu() - inp["prefix_len"]).max()) >= 3


@pytest.mark.parametrize("paged", [True, False])
def test_a_commit_before_the_first_attention(cuda_ok, paged):
    """Pages with bounds beside pages that have none yet."""
    inp, cache, step = make(BF, paged)
    q, k, v, logits, tokens = (t.cuda() for t in steps.step_inputs(B, N, Hq, Hkv, D, BF, 7))
    step.accept_commit(logits, None, tokens, k, v)
    run_and_check(step, cache, inp["block_table"] if paged else None, BF, 8)


@pytest.mark.parametrize("paged", [True, False])
def test_one_sequence_is_replaced(cuda_ok, paged):
    """A batch's slot gets another request: its bounds alone are made again."""
    inp, cache, step = make(BF, paged)
    table = inp["block_table"] if paged else None
    for seed in range(2):
        run_and_check(step, cache, table, BF, seed)
    # slot 3: another prompt of 300 positions in its old place
    other, _, _ = make(BF, paged, seed=9)
    for to, new in ((cache.k, other["cache_k"]), (cache.v, other["cache_v"])):
        if paged:
            mine = table[3][table[3] >= 0].long()
            to[mine.cuda()] = new[other["block_table"][3][other["block_table"][3] >= 0].long()[:mine.numel()]].cuda()
        else:
            to[3] = new[3].cuda()
    cache.prefix_len[3] = 240
    start = cache.prefix_len.clone()
    start[3] = 0
    kept = step.bounds.clone()
    n0 = sv.sv_kernel_launches()
    step.reset_bounds(start=start)
    torch.cuda.synchronize()
    assert sv.sv_kernel_launches() == n0 + 1
    changed = (step.bounds != kept).flatten(1).any(1) if paged else (step.bounds != kept).flatten(2).any(2)
    if paged:
        assert set(changed.nonzero().flatten().tolist()) == set(table[3][:15].tolist())
    else:
        assert set(changed.nonzero()[:, 0].tolist()) == {3}
    for seed in range(2, 4):
        run_and_check(step, cache, table, BF, seed)


def test_a_captured_first_step(cuda_ok):
    """The bounds are made in the capture then, and again at each replay."""
    inp, cache, step = make(BF, True)
    inp2, cache2, eager = make(BF, True)
    ins = [t.cuda() for t in steps.step_inputs(B, N, Hq, Hkv, D, BF, 0)]
    eager.attention(*ins[:3])  # (not captured: the kernels load)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.attention(*ins[:3])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, eager.out) and torch.equal(step.pages, eager.pages)
    cache.k.copy_(cache.k.flip(0))
    cache2.k.copy_(cache.k)
    eager.reset_bounds()
    eager.attention(*ins[:3])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, eager.out) and torch.equal(step.pages, eager.pages)
    assert sv.sv_read_device_status() == 0


@pytest.mark.parametrize("asked", [False, True])
def test_a_capture_makes_no_bounds_yet(cuda_ok, asked):
    """A call behind the capture of the first step, before any replay."""
    inp, cache, step = make(BF, True)
    inp2, cache2, eager = make(BF, True)
    ins = [t.cuda() for t in steps.step_inputs(B, N, Hq, Hkv, D, BF, 0)]
    eager.attention(*ins[:3])
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        if asked:
            step.reset_bounds(stream)
        step.attention(*ins[:3])
    step.attention(*ins[:3], stream=stream.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(step.out, eager.out) and torch.equal(step.pages, eager.pages)
    step.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, eager.out) and sv.sv_read_device_status() == 0


def test_steps_that_keep_no_bounds_have_none_to_make(cuda_ok):
    _, cache, _ = make(BF, True)
    step = VerifyStep(PARENT, B, Hq, Hkv, D, steps.V, cache, mode=sv.GREEDY)
    with pytest.raises(ValueError):
        step.reset_bounds()
