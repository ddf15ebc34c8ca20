"""The operators around the KV cache as a server uses them, with the framework's acceptance and
commit: block tables and slots for the prompts, their K/V normalised, rotated and written into
the pages, then rounds of tree rows, windowed attention, acceptance and commit, page by page."""
import numpy as np
import pytest
import torch

import plain_ops
import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl
from speculative_decoding_verify_sv_gb300.step import VerifyStep

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
B, Hq, Hkv, D, V, BS, W, S = 4, 8, 2, 64, 512, 16, 37, 3
PARENT = wl.TREE_EXAMPLE7
N, WIDTH = len(PARENT), (Hq + 2 * Hkv) * D


def _gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("graph", [False, True])
def test_prompts_then_rounds(cuda_ok, graph):
    prompt = torch.tensor([70, 1, 16, 33], dtype=torch.int32)
    columns, blocks = 12, 80
    order = torch.randperm(blocks, generator=_gen(1)).to(torch.int32)
    qw, kw = 1 + 0.2 * torch.randn(D, generator=_gen(2)), 1 + 0.2 * torch.randn(D, generator=_gen(3))
    inv = torch.tensor([10000.0 ** (-2 * i / D) for i in range(D // 2)], dtype=torch.float64)
    table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
    free = order.cuda()
    cache = sv.KVCache(torch.zeros(blocks, BS, Hkv, D, dtype=BF, device="cuda"),
                       torch.zeros(blocks, BS, Hkv, D, dtype=BF, device="cuda"),
                       torch.zeros(B, dtype=torch.int32, device="cuda"), table, BS)
    weights = (qw.cuda(), kw.cuda(), inv.cuda())

    # prompts: pages, slots, K and V into the pages (the slot map is longer than the prompts)
    r = sv.sv_block_tables(cache.prefix_len, prompt.cuda(), table, free, BS, blocks, 128)
    total = int(prompt.sum())
    qkv = torch.randn(128, WIDTH, generator=_gen(4)).to(BF)
    q, _, _ = sv.sv_qk_norm_rope(qkv.cuda(), Hq, Hkv, *weights, r["positions"], slots=r["slots"], k_out=cache.k, v_out=cache.v)
    cache.prefix_len.copy_(prompt)
    head = r["free_head"]

    # the same by hand, in dense rows: hist[b] = [(k, v)] as the kernels rounded them
    positions = np.concatenate([np.arange(int(n)) for n in prompt])
    (rq, rk, rv), (sq, skk) = plain_ops.qk_norm_rope(qkv[:total], Hq, Hkv, qw, kw, inv, torch.tensor(positions), 1e-6, False)
    rows = r["slots"][:total].long().cpu()
    assert (r["slots"][total:] == -1).all() and len(set(rows.tolist())) == total
    pk, pv = cache.k.cpu().view(-1, Hkv, D)[rows], cache.v.cpu().view(-1, Hkv, D)[rows]
    assert ((q[:total].double().cpu() - rq).abs() <= plain_ops.rope_bound(rq, sq, BF, D)).all()
    assert ((pk.double() - rk).abs() <= plain_ops.rope_bound(rk, skk, BF, D)).all()
    assert torch.equal(pv.double(), rv)
    untouched = torch.ones(blocks * BS, dtype=torch.bool)
    untouched[rows] = False
    assert (cache.k.cpu().view(-1, Hkv, D)[untouched] == 0).all()
    hist, at = [], 0
    for n in prompt.tolist():
        hist.append([pk[at:at + n], pv[at:at + n]])
        at += n

    step = VerifyStep(PARENT, B, Hq, Hkv, D, V, cache, mode=sv.GREEDY, window=W, sinks=S)
    new = torch.full((B,), max(wl.depths(PARENT)) + 1, dtype=torch.int32, device="cuda")  # the longest path
    inputs = dict(qkv=torch.zeros(B, N, WIDTH, dtype=BF, device="cuda"), logits=torch.zeros(B, N, V, dtype=BF, device="cuda"),
                  tokens=torch.zeros(B, N, dtype=torch.int32, device="cuda"))
    rope_outs = sv.sv_tree_qk_norm_rope(inputs["qkv"], Hq, Hkv, *weights, cache.prefix_len, PARENT)
    maps = {k: torch.empty_like(v) for k, v in sv.sv_block_tables(cache.prefix_len, new, table.clone(), free, BS, blocks, 64,
                                                                free_head=head).items()}
    start = head.clone()

    def one_round():
        sv.sv_block_tables(cache.prefix_len, new, table, free, BS, blocks, 64, free_head=start, outs=maps)
        qt, kt, vt = sv.sv_tree_qk_norm_rope(inputs["qkv"], Hq, Hkv, *weights, cache.prefix_len, PARENT, outs=rope_outs)
        step.attention(qt, kt, vt)
        step.accept_commit(inputs["logits"], None, inputs["tokens"], kt, vt)
        start.copy_(maps["free_head"])

    captured = None
    saved = (cache.prefix_len.clone(), start.clone())
    if graph:
        one_round()  # a trial of the round's calls, undone below
        cache.prefix_len.copy_(saved[0])
        start.copy_(saved[1])
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            one_round()
    given = int(saved[1])
    for rnd in range(6):
        g = _gen(100 + rnd)
        qkv = torch.randn(B, N, WIDTH, generator=g).to(BF)
        logits = torch.randn(B, N, V, generator=g).to(BF)
        tokens = torch.randint(0, V, (B, N), generator=g).to(torch.int32)
        for b in range(B):  # some drafts are what the target says
            for n in range(1, N):
                if (b + n + rnd) % 2:
                    tokens[b, n] = int(logits[b, PARENT[n]].float().argmax())
        for k, x in (("qkv", qkv), ("logits", logits), ("tokens", tokens)):
            inputs[k].copy_(x)
        L = cache.prefix_len.cpu()
        if captured is not None:
            captured.replay()
        else:
            one_round()
        torch.cuda.synchronize()
        assert sv.sv_read_device_status() == 0
        # pages: only what the longest path may need, none given out twice
        held = -(-L // BS)
        given += int((-(-(L + new.cpu()) // BS) - held).sum())
        assert int(start) == given
        # rotation at prefix + depth
        pos = torch.tensor([[int(n) + d for d in wl.depths(PARENT)] for n in L])
        (rq, rk, _), (sq, skk) = plain_ops.qk_norm_rope(qkv.view(B * N, -1), Hq, Hkv, qw, kw, inv, pos, 1e-6, False)
        qt, kt, vt = (x.cpu() for x in rope_outs)
        assert ((qt.double().view(rq.shape) - rq).abs() <= plain_ops.rope_bound(rq, sq, BF, D)).all()
        assert ((kt.double().view(rk.shape) - rk).abs() <= plain_ops.rope_bound(rk, skk, BF, D)).all()
        # attention over the history kept by hand
        longest = int(L.max())
        ck, cv = torch.zeros(B, longest, Hkv, D, dtype=BF), torch.zeros(B, longest, Hkv, D, dtype=BF)
        for b in range(B):
            ck[b, :int(L[b])], cv[b, :int(L[b])] = hist[b]
        ref, spread = plain_ops.window_attention(qt, kt, vt, ck, cv, L, PARENT, D ** -0.5, W, S)
        size = D ** -0.5 * qt.float().norm(dim=-1).max().item() * max(kt.float().norm(dim=-1).max().item(),
                                                                      ck.float().norm(dim=-1).max().item())
        bound = plain_ops.attention_bound(ref, spread, BF, D, size, W + S + N)
        assert ((step.out.double().cpu() - ref).abs() <= bound).all()
        # the accepted path joins the history
        path, acc = step.outs["path_nodes"].cpu(), step.outs["num_accepted"].cpu()
        for b in range(B):
            nodes = path[b, :int(acc[b]) + 1].long()
            hist[b] = [torch.cat([hist[b][0], kt[b, nodes]]), torch.cat([hist[b][1], vt[b, nodes]])]
        assert torch.equal(cache.prefix_len.cpu(), L + acc + 1)
        # pages left over from a shorter path are held by the table already: the next round counts
        # them by the length, so the head goes back to the first page nobody's length reaches
        reach = -(-(L + acc + 1) // BS)
        over = (-(-(L + new.cpu()) // BS)) - torch.maximum(reach, held)
        if int(over.sum()):
            _give_back(table, free, start, held, reach, L + new.cpu())
            given = int(start)


def _give_back(table, free, start, held, reach, asked):
    """Pages that a round took and its accepted paths did not reach go back to the free list, in
    the list's order (host bookkeeping of a server)."""
    t, f, head = table.cpu(), free.cpu(), int(start)
    back = []
    for b in range(B):
        for j in range(max(int(held[b]), int(reach[b])), -(-int(asked[b]) // BS)):
            back.append(int(t[b, j]))
            t[b, j] = -1
    f[head - len(back):head] = torch.tensor(back, dtype=torch.int32)
    table.copy_(t)
    free.copy_(f)
    start.sub_(len(back))


def test_window_of_the_step_is_the_operator(cuda_ok):
    """VerifyStep(window=...) runs sv_window_attention, and refuses sinks without a window."""
    inp = wl.attention_inputs(2, 5, 8, 2, 64, [90, 40], dtype=BF, seed=5)
    g = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
    cache = sv.KVCache(g["cache_k"], g["cache_v"], g["prefix_len"])
    step = VerifyStep(wl.chain_parent(4), 2, 8, 2, 64, 512, cache, window=20, sinks=2)
    got = step.attention(g["q"], g["k_tree"], g["v_tree"])
    want = sv.sv_window_attention(g["q"], g["k_tree"], g["v_tree"], cache, wl.chain_parent(4), 64 ** -0.5, 20, sinks=2)
    assert torch.equal(got, want)
    with pytest.raises(ValueError):
        VerifyStep(wl.chain_parent(4), 2, 8, 2, 64, 512, cache, sinks=2)


@pytest.mark.parametrize("handle", [False, True])
def test_calls_on_another_stream_keep_their_memory_apart(cuda_ok, handle):
    """What a call on a given stream makes is not memory that the current stream still writes."""
    side = torch.cuda.Stream()
    given = side.cuda_stream if handle else side
    b, n, hq, hkv, d = 16, 26, 64, 8, 128
    inp = wl.attention_inputs(b, n, hq, hkv, d, [2100] * b, dtype=BF, seed=3)
    g = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
    cache = sv.KVCache(g["cache_k"], g["cache_v"], g["prefix_len"])
    assert sv.sv_window_attention_workspace_size(BF, b, n, hq, hkv, d, cache.max_prefix, 2048) > 0
    qkv = torch.randn(b, n, (hq + 2 * hkv) * d, generator=_gen(6)).to(BF).cuda()
    w = torch.ones(d, device="cuda")
    freq = torch.tensor([10000.0 ** (-i / 64) for i in range(64)], dtype=torch.float64, device="cuda")
    pos = torch.arange(b * n, dtype=torch.int32, device="cuda")
    new = torch.arange(300, dtype=torch.int32, device="cuda")
    length, table = torch.zeros_like(new), torch.full((300, 40), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(9000, dtype=torch.int32, device="cuda")

    def table_call(**kw):
        r = sv.sv_block_tables(length, new, table, free, 16, 9000, 50000, **kw)
        return r["slots"], r["positions"], r["token_start"], r["free_head"]
    par = wl.chain_parent(n - 1)
    calls = (lambda **kw: (sv.sv_window_attention(g["q"], g["k_tree"], g["v_tree"], cache, par, d ** -0.5, 2048, **kw),),
             lambda **kw: (sv.sv_window_attention(g["q"], g["k_tree"], g["v_tree"], cache, par, d ** -0.5, 17, **kw),),
             lambda **kw: sv.sv_qk_norm_rope(qkv.view(b * n, -1), hq, hkv, w, w, freq, pos, **kw),
             lambda **kw: sv.sv_tree_qk_norm_rope(qkv, hq, hkv, w, w, freq, g["prefix_len"], par, **kw), table_call)
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        sizes = [x.untyped_storage().nbytes() for x in want]
        for size in sizes:
            old = torch.empty(size, dtype=torch.uint8, device="cuda")
            torch.cuda._sleep(20_000_000)
            old.fill_(255)
            del old  # free for the current stream, which has yet to write it
        got = call(stream=given)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert sv.sv_read_device_status() == 0
