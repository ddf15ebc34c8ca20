"""How the operators for shared prefixes and selected pages are called: streams, captured graphs, workspaces, empty
batches, launches that fail, waits that run out, caches of more than 2^31 elements."""
import time

import pytest
import torch

import plain_pages
import speculative_decoding_verify_sv_gb300 as sv
import test_gpu_shared_attention as shared
import test_gpu_sparse_attention as sparse
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


class Chain:
    """Bounds, scores, selection and both attentions over one cache; `stacked`: rows and lists for the stacked kernel."""

    def __init__(self, seed, stacked=True, dtype=BF, lens=(190, 260, 201, 177)):
        self.parent = wl.TREE_T26 if stacked else wl.chain_parent(2)
        N = len(self.parent)
        sizes, own = [2, 2], [lens[0] - 160, lens[1] - 160, lens[2] - 96, lens[3] - 96]
        self.inp = inp = shared.shared_inputs(sizes, [160, 96], own, N, 16, 4, 128, dtype=dtype, seed=seed)
        if stacked and dtype == BF:
            inp = self.inp = shared.roomy(inp, 16)
        self.g = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
        g = self.g
        self.cache = sv.KVCache(g["cache_k"], g["cache_v"], g["prefix_len"], g["block_table"], 16)
        self.long = 2000 * torch.cuda.get_device_properties(0).multi_processor_count // 64 if stacked else 6
        self.bounds = torch.zeros(inp["num_blocks"], 4, 2, 128, dtype=dtype, device="cuda")
        self.scores = torch.zeros(4, 1, 4, inp["block_table"].shape[1], device="cuda")
        self.pages = torch.full((4, 1, 4, self.long), -1, dtype=torch.int32, device="cuda")
        self.outs = [torch.zeros_like(g["q"]) for _ in range(2)]
        need = (sv.sv_sparse_attention_workspace_size(dtype, 4, N, 16, 4, 128, 16, self.long),
                sv.sv_shared_attention_workspace_size(dtype, 4, N, 16, 4, 128, self.cache.max_prefix, 2))
        assert dtype == F32 or (need[0] > 0) == (need[1] > 0) == stacked
        self.work = [torch.full((max(16, n),), 255, dtype=torch.uint8, device="cuda") for n in need]  # (of NaNs)

    def calls(self, stream=None):
        g, c = self.g, self.cache
        sv.sv_page_bounds(c, self.bounds, stream=stream)
        sv.sv_page_scores(g["q"], self.bounds, c.prefix_len, 16, block_table=c.block_table, out=self.scores, stream=stream)
        # (for the stacked kernel lists are long: every page, then entries that are none)
        sv.sv_select_pages(self.scores, c.prefix_len, 16, self.long, out=self.pages, stream=stream)
        sv.sv_sparse_attention(g["q"], g["k_tree"], g["v_tree"], c, self.parent, 0.09, self.pages, out=self.outs[0],
                               workspace=self.work[0], stream=stream)
        sv.sv_shared_attention(g["q"], g["k_tree"], g["v_tree"], c, self.parent, 0.09, g["group_start"], g["shared_len"],
                               out=self.outs[1], workspace=self.work[1], stream=stream)

    def results(self):
        return [t.clone() for t in (self.bounds, self.scores, self.pages, *self.outs)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("stacked", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_repeated_calls_give_the_same(cuda_ok, stacked, dtype):
    """Nothing that a call leaves in a workspace, and no order of CTAs, changes the next one."""
    c = Chain(1, stacked, dtype)
    c.calls()
    first = c.results()
    for _ in range(10):
        c.work[0].random_(0, 256)
        c.work[1].random_(0, 256)
        c.calls()
        assert same(c.results(), first)
    assert sv.sv_read_device_status() == 0


@pytest.mark.parametrize("stacked", [True, False])
def test_two_streams_with_workspaces_of_their_own(cuda_ok, stacked):
    a, b = Chain(2, stacked), Chain(3, stacked)
    a.calls(), b.calls()
    torch.cuda.synchronize()
    want = [a.results(), b.results()]
    for t in (*a.outs, *b.outs):
        t.zero_()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        for c, s in zip((a, b), streams):
            c.calls(s)
    torch.cuda.synchronize()
    assert same(a.results(), want[0]) and same(b.results(), want[1])
    a.calls(streams[0].cuda_stream)  # a handle
    torch.cuda.synchronize()
    assert same(a.results(), want[0]) and sv.sv_read_device_status() == 0


@pytest.mark.parametrize("stacked", [True, False])
def test_captured_calls_follow_what_is_on_the_device(cuda_ok, stacked):
    """Lengths, groups, tables and queries change between replays; two graphs share the workspaces."""
    c = Chain(4, stacked)
    c.calls()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.calls()
    for k, lens in enumerate(((190, 260, 201, 177), (160, 161, 96, 190), (208, 200, 112, 96))):
        c.g["q"].copy_(torch.randn(c.g["q"].shape, generator=torch.Generator().manual_seed(k)))
        c.cache.prefix_len.copy_(torch.tensor(lens, dtype=torch.int32))
        c.g["shared_len"].copy_(torch.tensor((160, 96) if k < 2 else (128, 0), dtype=torch.int32))
        c.g["group_start"].copy_(torch.tensor((0, 2, 4) if k != 1 else (0, 2, 2), dtype=torch.int32))
        graphs[k % 2].replay()
        graphs[(k + 1) % 2].replay()
        torch.cuda.synchronize()
        got = c.results()
        for t in c.outs:
            t.zero_()
        c.calls()
        torch.cuda.synchronize()
        assert same(got, c.results())
    assert sv.sv_read_device_status() == 0


def test_small_and_unaligned_workspaces_are_refused(cuda_ok):
    c = Chain(5)
    for i in range(2):
        assert c.work[i].numel() > 1000
        work = list(c.work)
        for bad in (c.work[i][:-256], c.work[i][4:]):
            c.work[i] = bad
            with pytest.raises(sv.SVError) as err:
                c.calls()
            assert err.value.code in (sv.SV_ERR_WORKSPACE, sv.SV_ERR_INVALID_ARG)
        c.work = work


def test_arguments_that_are_refused(cuda_ok):
    c = Chain(6, False)
    g, cache = c.g, c.cache

    def sparse_call(pages=c.pages, cache=cache, **kw):
        return sv.sv_sparse_attention(g["q"], g["k_tree"], g["v_tree"], cache, c.parent, 0.09, pages, **kw)

    def shared_call(start=g["group_start"], length=g["shared_len"], **kw):
        return sv.sv_shared_attention(g["q"], g["k_tree"], g["v_tree"], cache, c.parent, 0.09, start, length, **kw)

    wide = torch.zeros(4, 1, 4, 12, dtype=torch.int32, device="cuda")
    for call in (lambda: sparse_call(c.pages.long()), lambda: sparse_call(wide[..., ::2]), lambda: sparse_call(c.pages[:, :, :2].contiguous()),
                 lambda: sparse_call(c.pages.expand(4, 2, 4, 6).contiguous()), lambda: sparse_call(c.pages.cpu()),
                 lambda: sparse_call(c.pages[0]), lambda: sparse_call(out=g["q"].float()), lambda: sparse_call(out=g["q"][:, :1]),
                 lambda: shared_call(g["group_start"][:2]), lambda: shared_call(length=g["shared_len"].long()),
                 lambda: shared_call(g["group_start"].cpu()), lambda: shared_call(length=g["shared_len"].view(2, 1)),
                 lambda: sv.sv_page_bounds(cache, c.bounds.float()), lambda: sv.sv_page_bounds(cache, c.bounds[:-1]),
                 lambda: sv.sv_page_bounds(cache, c.bounds, start=g["prefix_len"][:2]),
                 lambda: sv.sv_page_scores(g["q"].float(), c.bounds, cache.prefix_len, 16, block_table=cache.block_table),
                 lambda: sv.sv_page_scores(g["q"], c.bounds, cache.prefix_len, 16),
                 lambda: sv.sv_page_scores(g["q"], c.bounds, cache.prefix_len[:3], 16, block_table=cache.block_table),
                 lambda: sv.sv_select_pages(c.scores.to(BF), cache.prefix_len, 16, 4),
                 lambda: sv.sv_select_pages(c.scores, cache.prefix_len.long(), 16, 4),
                 lambda: sv.sv_select_pages(c.scores, cache.prefix_len, 16, 4, out=c.pages)):
        with pytest.raises((TypeError, ValueError)):
            call()
    for call in (lambda: sparse_call(out=g["q"]), lambda: shared_call(out=g["q"]), lambda: sv.sv_select_pages(c.scores, cache.prefix_len, 16, 2, 2, 1),
                 lambda: sv.sv_select_pages(c.scores, cache.prefix_len, 16, 0), lambda: sv.sv_select_pages(c.scores, cache.prefix_len, 0, 4)):
        with pytest.raises(sv.SVError):
            call()
    # (a slice that is whole rows is as good as any tensor)
    c.calls()
    want = c.outs[0].clone()
    assert torch.equal(sparse_call(torch.cat([c.pages, c.pages])[4:]), want)


def test_empty_batches(cuda_ok):
    n0 = sv.sv_kernel_launches()
    i32 = dict(dtype=torch.int32, device="cuda")
    q, kt = torch.empty(0, 5, 8, 64, dtype=BF, device="cuda"), torch.empty(0, 5, 2, 64, dtype=BF, device="cuda")
    cache = sv.KVCache(torch.empty(0, 64, 2, 64, dtype=BF, device="cuda"), torch.empty(0, 64, 2, 64, dtype=BF, device="cuda"),
                       torch.empty(0, **i32))
    par = wl.chain_parent(4)
    assert sv.sv_shared_attention(q, kt, kt, cache, par, 0.1, torch.zeros(2, **i32), torch.zeros(1, **i32)).shape == q.shape
    assert sv.sv_sparse_attention(q, kt, kt, cache, par, 0.1, torch.empty(0, 1, 2, 4, **i32)).shape == q.shape
    bounds = sv.sv_page_bounds(cache)
    assert bounds.shape == (0, 4, 2, 2, 64)
    scores = sv.sv_page_scores(q, bounds, cache.prefix_len, 16)
    assert scores.shape == (0, 1, 2, 4) and sv.sv_select_pages(scores, cache.prefix_len, 16, 3).shape == (0, 1, 2, 3)
    torch.cuda.synchronize()
    assert sv.sv_kernel_launches() == n0 and sv.sv_read_device_status() == 0


@pytest.mark.parametrize("stacked", [True, False])
def test_failed_launches_are_reported_and_harmless(cuda_ok, stacked):
    """Each launch of each operator in turn (no fault: the host reports the failure in the launch's place)."""
    c = Chain(7, stacked)
    c.calls()
    torch.cuda.synchronize()
    want, n0 = c.results(), sv.sv_kernel_launches()
    c.calls()
    launches = sv.sv_kernel_launches() - n0
    assert launches == (7 if stacked else 5)
    g, cache = c.g, c.cache
    for call in (lambda: sv.sv_page_bounds(cache, c.bounds), lambda: sv.sv_select_pages(c.scores, cache.prefix_len, 16, c.long, out=c.pages),
                 lambda: sv.sv_page_scores(g["q"], c.bounds, cache.prefix_len, 16, block_table=cache.block_table, out=c.scores),
                 lambda: sv.sv_sparse_attention(g["q"], g["k_tree"], g["v_tree"], cache, c.parent, 0.09, c.pages, out=c.outs[0], workspace=c.work[0]),
                 lambda: sv.sv_shared_attention(g["q"], g["k_tree"], g["v_tree"], cache, c.parent, 0.09, g["group_start"], g["shared_len"],
                                                out=c.outs[1], workspace=c.work[1])):
        n0 = sv.sv_kernel_launches()
        sv.sv_inject_launch_failures(1)
        with pytest.raises(sv.SVError) as err:
            call()
        assert err.value.code == sv.SV_ERR_CUDA and "launch" in str(err.value) and sv.sv_kernel_launches() == n0
        torch.cuda.synchronize()
        assert same(c.results(), want)
    c.calls()
    torch.cuda.synchronize()
    assert same(c.results(), want) and sv.sv_read_device_status() == 0


@pytest.mark.parametrize("kind", ["stacked", "warps", "units", "clusters", "far clusters"])
def test_a_wait_that_runs_out_is_reported(cuda_ok, kind):
    """With a limit far below a copy's time calls end soon and say so, and the next one is right.  (Nothing
    hangs: the waits are bounded, the test shortens their bound.)"""
    B, N, K = {"stacked": (16, 26, 256), "warps": (100, 1, 128), "units": (30, 5, 128), "clusters": (2, 1, 600),
               "far clusters": (8, 1, 1200)}[kind]
    Hq, Hkv, D = 32, 8, 128
    par = wl.TREE_T26 if N == 26 else wl.chain_parent(N - 1)
    g = torch.Generator(device="cuda").manual_seed(B)
    q, kt, vt = (torch.randn(B, N, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    P = K + 8
    k, v = (torch.empty(B * P, 16, Hkv, D, dtype=BF, device="cuda").normal_(generator=g) for _ in "kv")
    table = torch.randperm(B * P, generator=g, device="cuda").to(torch.int32).view(B, P)
    cache = sv.KVCache(k, v, torch.full((B,), P * 16 - 70, dtype=torch.int32, device="cuda"), table, 16)
    pages = torch.arange(K, dtype=torch.int32, device="cuda").expand(B, 1, Hkv, K).contiguous()
    start, length = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, B], [K * 8]))
    outs = [torch.empty_like(q) for _ in range(2)]

    def call():
        sv.sv_sparse_attention(q, kt, vt, cache, par, D ** -0.5, pages, out=outs[0])
        sv.sv_shared_attention(q, kt, vt, cache, par, D ** -0.5, start, length, out=outs[1])
        torch.cuda.synchronize()
        return sv.sv_read_device_status()

    assert call() == 0
    want, found = [o.clone() for o in outs], []
    for _ in range(12):
        try:
            sv.sv_set_wait_limit_ns(1)
            begin = time.perf_counter()
            found.append(call())
            took = time.perf_counter() - begin
        finally:
            sv.sv_set_wait_limit_ns(0)
        assert took < 1.0
        assert call() == 0 and all(torch.equal(o, w) for o, w in zip(outs, want))
    assert set(found) <= {0, sv.SV_DEV_TIMEOUT}
    # (a cache of 39 MB stays in the L2, from where every copy lands within the first try to wait for it)
    assert sv.SV_DEV_TIMEOUT in found or kind == "clusters"


def test_caches_past_two_to_the_31_elements(cuda_ok):
    """Pools of more than 2^31 elements (and 2^32 bytes), whose last blocks are the ones in use."""
    Hkv, D, page, N = 8, 128, 16, 26
    blocks = 2 ** 31 // (page * Hkv * D) + 600
    free = torch.cuda.mem_get_info()[0]
    if free < 3 * blocks * page * Hkv * D * 2:
        pytest.skip("not enough memory")
    k = torch.zeros(blocks, page, Hkv, D, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    lens = [3000, 2900]
    P = 188
    table = (blocks - 1 - torch.arange(2 * P)).view(2, P).to(torch.int32)
    g = torch.Generator().manual_seed(3)
    for t in (k, v):
        t[blocks - 2 * P:] = torch.randn(2 * P, page, Hkv, D, generator=g).to(BF).cuda()
    q, kt, vt = (torch.randn(2, N, h, D, generator=g).to(BF) for h in (16, Hkv, Hkv))
    cache = sv.KVCache(k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda(), page)
    bounds = sv.sv_page_bounds(cache)
    scores = sv.sv_page_scores(q.cuda(), bounds, cache.prefix_len, page, block_table=cache.block_table)
    pages = sv.sv_select_pages(scores, cache.prefix_len, page, 100)
    # the same in a small pool
    small = table - (blocks - 2 * P)
    part = {"q": q, "k_tree": kt, "v_tree": vt, "cache_k": k[blocks - 2 * P:].cpu(), "cache_v": v[blocks - 2 * P:].cpu(),
            "prefix_len": torch.tensor(lens, dtype=torch.int32), "block_table": small, "num_blocks": 2 * P}
    want = plain_pages.page_bounds(torch.zeros(2 * P, Hkv, 2, D, dtype=BF), part["cache_k"], part["prefix_len"], None, small, page)
    kept = sorted(int(small[b, j]) for b in range(2) for j in range(-(-lens[b] // page)))
    assert torch.equal(bounds[blocks - 2 * P:].cpu()[kept], want[kept])
    ref, size = plain_pages.page_scores(q, want, part["prefix_len"], page, small)
    err = (scores.double().cpu() - ref).abs().nan_to_num()
    assert bool((err <= (2 * D + 2) * 2.0 ** -23 * size).all())
    for kind in (pages, sparse.padded(part, pages.cpu(), page).cuda()):
        out = sv.sv_sparse_attention(q.cuda(), kt.cuda(), vt.cuda(), cache, wl.TREE_T26, D ** -0.5, kind)
        assert torch.equal(out, sparse.call(part, wl.TREE_T26, kind.cpu(), page))
    groups = torch.tensor([0, 1, 2], dtype=torch.int32), torch.tensor([2900, 1600], dtype=torch.int32)
    out = sv.sv_shared_attention(q.cuda(), kt.cuda(), vt.cuda(), cache, wl.TREE_T26, D ** -0.5, groups[0].cuda(), groups[1].cuda())
    part.update(group_start=groups[0], shared_len=groups[1])
    assert torch.equal(out, shared.call(part, wl.TREE_T26, page)) and sv.sv_read_device_status() == 0
    few = sv.sv_sparse_attention(q[:, :1].cuda(), kt[:, :1].cuda(), vt[:, :1].cuda(), cache, [-1], D ** -0.5, pages)
    one = {**part, "q": q[:, :1].contiguous(), "k_tree": kt[:, :1].contiguous(), "v_tree": vt[:, :1].contiguous()}
    assert torch.equal(few, sparse.call(one, [-1], pages.cpu(), page))
