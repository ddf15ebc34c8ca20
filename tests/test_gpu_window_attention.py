"""Windowed tree attention with sinks against its definition in 64 bits."""
import math

import pytest
import torch

import plain_ops
import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _cuda(inp):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}


def _call(g, parent, window, sinks, block_size=16, **kw):
    cache = sv.KVCache(g["cache_k"], g["cache_v"], g["prefix_len"], g["block_table"], block_size)
    return sv.sv_window_attention(g["q"], g["k_tree"], g["v_tree"], cache, parent,
                                  g["q"].shape[-1] ** -0.5, window, sinks=sinks, **kw)


def _bound(inp, ref, spread, window, sinks):
    D = inp["q"].shape[-1]
    # scale * sum |q_i k_i| <= scale * |q| |k|
    size = D ** -0.5 * inp["q"].float().norm(dim=-1).max().item() * max(
        inp["k_tree"].float().norm(dim=-1).max().item(), inp["cache_k"].float().norm(dim=-1).nan_to_num().max().item())
    keys = min(window, int(inp["prefix_len"].max())) + sinks + 64
    return plain_ops.attention_bound(ref, spread, inp["q"].dtype, D, size, keys)


def _check(inp, parent, window, sinks, block_size=16):
    out = _call(_cuda(inp), parent if not isinstance(parent[0], list) else
                torch.tensor(parent, dtype=torch.int32, device="cuda"), window, sinks, block_size)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0
    ref, spread = plain_ops.window_attention(inp["q"], inp["k_tree"], inp["v_tree"], inp["cache_k"], inp["cache_v"],
                                             inp["prefix_len"], parent, inp["q"].shape[-1] ** -0.5, window, sinks,
                                             inp["block_table"], block_size)
    err = (out.double().cpu() - ref).abs()
    bound = _bound(inp, ref, spread, window, sinks)
    assert torch.isfinite(out).all() and (err <= bound).all(), ((err - bound).max().item(), err.max().item())
    return out


LENS = [0, 1, 2, 3, 15, 16, 17, 63, 127, 128, 129, 130, 143, 255, 256, 257, 300, 401]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (3, 0), (16, 4), (17, 64), (64, 5), (127, 1),
                                          (128, 16), (129, 17), (130, 33), (256, 48), (1000, 4), (2 ** 31 - 1, 64)])
def test_windows_and_sinks(cuda_ok, dtype, paged, window, sinks):
    inp = wl.attention_inputs(len(LENS), 5, 8, 2, 64, LENS, dtype=dtype, paged=paged, seed=1 + window % 97)
    _check(inp, wl.chain_parent(4), window, sinks)


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (32, 4), (8, 1), (14, 2), (6, 2)])
@pytest.mark.parametrize("tree", ["root", "t26", "t64", "example7"])
def test_trees_and_head_groups(cuda_ok, Hq, Hkv, tree):
    """Grouped heads that divide a 128-row tile and that do not, one to four row tiles."""
    par = {"root": [-1], "t26": wl.TREE_T26, "t64": wl.TREE_T64, "example7": wl.TREE_EXAMPLE7}[tree]
    lens = [0, 40, 129, 290]
    inp = wl.attention_inputs(4, len(par), Hq, Hkv, 128, lens, dtype=BF, seed=3)
    _check(inp, par, 33, 4)
    _check(inp, par, 2, 1)


@pytest.mark.parametrize("block_size", [16, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(cuda_ok, block_size, D):
    lens = [5, 130, 257, 511, 600]
    inp = wl.attention_inputs(5, 5, 8, 2, D, lens, dtype=BF, paged=True, block_size=block_size, seed=4)
    for window, sinks in ((40, 4), (140, 64), (300, 0)):
        _check(inp, wl.chain_parent(4), window, sinks, block_size)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_deep_chain_beyond_its_window(cuda_ok, dtype):
    """A 64-node chain with windows shorter than itself: nodes lose their own root path's start,
    except the part that stands among the sinks."""
    inp = wl.attention_inputs(4, 64, 4, 2, 64, [0, 3, 20, 70], dtype=dtype, seed=5)
    for window, sinks in ((1, 0), (5, 0), (5, 10), (33, 64), (63, 1), (64, 0), (65, 0)):
        _check(inp, wl.chain_parent(63), window, sinks)


def test_trees_of_each_sequence(cuda_ok):
    g = torch.Generator().manual_seed(6)
    parents = [[-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, 13)] for _ in range(6)]
    for dtype in (BF, F32):
        inp = wl.attention_inputs(6, 13, 8, 2, 128, [0, 7, 64, 100, 129, 300], dtype=dtype, seed=7)
        _check(inp, parents, 6, 2)
        _check(inp, parents, 3, 40)


@pytest.mark.parametrize("paged", [False, True])
def test_long_unit_cut_over_many_ctas(cuda_ok, paged):
    """One sequence and KV head with a long window: its tiles are split and joined again."""
    inp = wl.attention_inputs(1, 5, 8, 1, 128, [9001], dtype=BF, paged=paged, seed=8)
    _check(inp, wl.chain_parent(4), 8500, 64)
    inp = wl.attention_inputs(2, 26, 16, 2, 128, [5000, 4100], dtype=BF, paged=paged, seed=9)
    _check(inp, wl.TREE_T26, 4096, 4)


# (nodes, group heads) -> units with 64, 104, 208 and 512 query rows, where many units with long
# enough windows go to the 128-row tensor-core kernel: two row copies, one tile, two tiles, two
# groups of two tiles
@pytest.mark.parametrize("N,G,B,window", [(16, 4, 40, 3500), (26, 4, 64, 260), (26, 8, 48, 40), (26, 8, 48, 300),
                                          (64, 8, 24, 17), (64, 8, 24, 200)])
@pytest.mark.parametrize("D,block_size", [(128, 0), (128, 16), (64, 32), (128, 128), (64, 0)])
def test_many_units_of_many_rows(cuda_ok, N, G, B, window, D, block_size):
    Hkv = 8 if B > 24 else 4
    par = wl.TREE_T26 if N == 26 else (wl.TREE_T64 if N == 64 else wl.chain_parent(N - 1))
    g = torch.Generator().manual_seed(N + B)
    lens = torch.randint(0, window + 150, (B,), generator=g).tolist()
    lens[:4] = [0, 1, window, window + 17]
    inp = wl.attention_inputs(B, N, G * Hkv, Hkv, D, lens, dtype=BF, paged=block_size > 0,
                              block_size=block_size or 16, seed=16)
    limit = inp["cache_k"].shape[1] if not block_size else inp["block_table"].shape[1] * block_size
    assert sv.sv_window_attention_workspace_size(BF, B, N, G * Hkv, Hkv, D, limit, window) > 0
    for sinks in (4, 0, 49):
        _check(inp, par, window, sinks, block_size or 16)


def test_whole_prefix_is_tree_attention(cuda_ok):
    """A window beyond every position sees what sv_tree_attention sees."""
    par = wl.TREE_T26
    inp = _cuda(wl.attention_inputs(3, 26, 16, 4, 128, [900, 0, 300], dtype=BF, seed=10))
    cache = sv.KVCache(inp["cache_k"], inp["cache_v"], inp["prefix_len"])
    full = sv.sv_tree_attention(inp["q"], inp["k_tree"], inp["v_tree"], cache, par, 0.1).double()
    win = sv.sv_window_attention(inp["q"], inp["k_tree"], inp["v_tree"], cache, par, 0.1, 5000, sinks=7).double()
    assert (full - win).abs().max().item() <= 2.0 ** -7 * full.abs().max().item()


@pytest.mark.parametrize("dtype,B,N,Hq,Hkv,D", [(BF, 5, 7, 8, 2, 128), (F32, 5, 7, 8, 2, 128), (BF, 5, 26, 8, 4, 64),
                                                (BF, 64, 26, 64, 8, 128), (BF, 64, 26, 64, 8, 64)])
@pytest.mark.parametrize("paged", [False, True])
def test_nothing_leaks_from_what_no_row_sees(cuda_ok, dtype, B, N, Hq, Hkv, D, paged):
    """NaN and infinity in every cache position outside the window and the sinks, in the room
    behind the prefixes and in the neighbours' rows change no bit; freed pages may hold any id.
    (The last two shapes go to the 128-row kernel.)"""
    par = wl.TREE_EXAMPLE7 if N == 7 else wl.TREE_T26
    window, sinks = (37, 5) if B == 5 else (150, 21)
    lens = ([300, 40, 129, 33, 0] * 15)[:B]
    inp = wl.attention_inputs(B, N, Hq, Hkv, D, lens, dtype=dtype, paged=paged, seed=11)
    if B > 5:
        assert sv.sv_window_attention_workspace_size(dtype, B, N, Hq, Hkv, D, 300, window) > 0
    clean = _check(inp, par, window, sinks)
    seen = torch.zeros(inp["cache_k"].shape[:2], dtype=torch.bool)
    table = inp["block_table"]
    for b, L in enumerate(lens):
        for p in list(range(max(0, L - window + 1), L)) + list(range(min(sinks, L))):
            if paged:
                seen[table[b, p // 16], p % 16] = True
            else:
                seen[b, p] = True
    for bad in (float("nan"), float("inf"), -float("inf")):
        g = _cuda(inp)
        g["cache_k"] = inp["cache_k"].masked_fill(~seen[..., None, None], bad).cuda()
        g["cache_v"] = inp["cache_v"].masked_fill(~seen[..., None, None], bad).cuda()
        assert torch.equal(_call(g, par, window, sinks), clean)
    if paged:
        g = _cuda(inp)
        for b, L in enumerate(lens):
            for j in range(table.shape[1]):
                if not any(j == p // 16 for p in list(range(max(0, L - window + 1), L)) + list(range(min(sinks, L)))):
                    g["block_table"][b, j] = (-1, 10 ** 9)[j % 2]
        assert torch.equal(_call(g, par, window, sinks), clean)
    # one sequence's tree rows hold NaN: the others' results keep their bits
    g = _cuda(inp)
    for k in ("k_tree", "v_tree"):
        g[k][1] = float("nan")
    out = _call(g, par, window, sinks)
    keep = [0] + list(range(2, B))
    assert torch.equal(out[keep], clean[keep])
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0


def test_bad_blocks_and_prefixes_are_reported(cuda_ok):
    inp = wl.attention_inputs(3, 5, 8, 2, 128, [300, 200, 100], dtype=BF, paged=True, seed=12)
    good = _call(_cuda(inp), wl.chain_parent(4), 50, 4)
    g = _cuda(inp)
    g["block_table"][1, 199 // 16] = 10 ** 6
    out = _call(g, wl.chain_parent(4), 50, 4)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
    assert torch.equal(out[[0, 2]], good[[0, 2]])
    g = _cuda(inp)
    g["block_table"][2, 0] = -1  # a page of the sinks
    out = _call(g, wl.chain_parent(4), 50, 4)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
    assert torch.equal(out[:2], good[:2])
    g = _cuda(inp)
    g["prefix_len"][0] = 10 ** 6
    _call(g, wl.chain_parent(4), 50, 4)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() & sv.SV_DEV_BAD_PREFIX


def test_streams_graphs_and_a_shared_workspace(cuda_ok):
    """The same bits from another stream, from a replayed graph with new contents, and from
    calls of several shapes and of sv_tree_attention that share one workspace in order."""
    par = wl.chain_parent(4)
    inp = wl.attention_inputs(4, 5, 32, 8, 128, [700, 90, 129, 2000], dtype=BF, seed=13)
    other = _cuda(wl.attention_inputs(1, 26, 32, 8, 128, [1500], dtype=BF, seed=14))
    g = _cuda(inp)
    cache = sv.KVCache(g["cache_k"], g["cache_v"], g["prefix_len"])
    first = _call(g, par, 256, 4)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(first)
    for _ in range(3):
        sv.sv_window_attention(g["q"], g["k_tree"], g["v_tree"], cache, par, 128 ** -0.5, 256, sinks=4, out=out,
                               workspace=ws, stream=s)
        with torch.cuda.stream(s):
            _call(other, wl.TREE_T26, 1000, 0, workspace=ws)
            sv.sv_tree_attention(g["q"], g["k_tree"], g["v_tree"], cache, par, 128 ** -0.5, workspace=ws)
    s.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sv_window_attention(g["q"], g["k_tree"], g["v_tree"], cache, par, 128 ** -0.5, 256, sinks=4, out=out,
                               workspace=ws)
    g["prefix_len"].copy_(torch.tensor([3, 400, 1999, 0], dtype=torch.int32))
    g["q"].mul_(-1)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, _call(g, par, 256, 4))
    assert sv.sv_read_device_status() == 0


def test_refusals_and_empty_batch(cuda_ok):
    inp = _cuda(wl.attention_inputs(2, 5, 8, 2, 128, [30, 20], dtype=BF, seed=15))
    par = wl.chain_parent(4)
    for window, sinks, code in ((0, 0, sv.SV_ERR_INVALID_ARG), (-3, 0, sv.SV_ERR_INVALID_ARG),
                                (4, -1, sv.SV_ERR_INVALID_ARG), (4, 65, sv.SV_ERR_UNSUPPORTED)):
        with pytest.raises(sv.SVError) as e:
            _call(inp, par, window, sinks)
        assert e.value.code == code
    for scale in (0.0, -0.1, float("nan"), float("inf")):
        with pytest.raises(sv.SVError) as e:
            sv.sv_window_attention(inp["q"], inp["k_tree"], inp["v_tree"],
                                   sv.KVCache(inp["cache_k"], inp["cache_v"], inp["prefix_len"]), par, scale, 4)
        assert e.value.code == sv.SV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        _call(inp, par, 2 ** 31, 0)
    with pytest.raises(ValueError):
        _call(dict(inp, cache_k=inp["cache_k"][:1], cache_v=inp["cache_v"][:1]), par, 4, 0)
    big = _cuda(wl.attention_inputs(64, 26, 32, 4, 64, [300] * 64, dtype=BF, seed=17))
    need = sv.sv_window_attention_workspace_size(BF, 64, 26, 32, 4, 64, big["cache_k"].shape[1], 300)
    with pytest.raises(sv.SVError) as e:
        _call(big, wl.TREE_T26, 300, 0, workspace=torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))
    assert need > 0 and e.value.code == sv.SV_ERR_WORKSPACE
    n0 = sv.sv_kernel_launches()
    empty = dict(inp, **{k: inp[k][:0] for k in ("q", "k_tree", "v_tree", "cache_k", "cache_v", "prefix_len")})
    assert _call(empty, par, 4, 0).shape == (0, 5, 8, 128)
    assert sv.sv_kernel_launches() == n0 and sv.sv_read_device_status() == 0


def test_injected_launch_failure_writes_nothing(cuda_ok):
    """Each kernel's call reports the failure, launches nothing and works at the next try."""
    for dtype, B, N, Hq, Hkv, D in ((BF, 3, 5, 8, 2, 128), (F32, 3, 5, 8, 2, 64), (BF, 64, 26, 32, 4, 64)):
        par = wl.TREE_T26 if N == 26 else wl.chain_parent(4)
        inp = _cuda(wl.attention_inputs(B, N, Hq, Hkv, D, [300] * B, dtype=dtype, seed=18))
        want = _call(inp, par, 300, 4)
        out = torch.full_like(want, 7.0)
        n0 = sv.sv_kernel_launches()
        sv.sv_inject_launch_failures(1)
        try:
            with pytest.raises(sv.SVError) as e:
                _call(inp, par, 300, 4, out=out)
        finally:
            sv.sv_inject_launch_failures(0)
        assert e.value.code == sv.SV_ERR_CUDA and sv.sv_kernel_launches() == n0
        torch.cuda.synchronize()
        assert (out == 7.0).all()
        assert torch.equal(_call(inp, par, 300, 4, out=out), want)


def test_waits_that_run_out_return(cuda_ok):
    """With the wait limit far below a copy's time the call returns and reports it; the next one is
    right.  (Nothing hangs: the waits are bounded, the test shortens their bound.)"""
    for N, Hq in ((1, 8), (16, 64)):
        inp = wl.attention_inputs(2, N, Hq, 2, 128, [1500, 900], dtype=BF, seed=19)
        g, par = _cuda(inp), wl.chain_parent(N - 1)
        want = _call(g, par, 1024, 4)
        sv.sv_read_device_status()
        try:
            sv.sv_set_wait_limit_ns(100)
            _call(g, par, 1024, 4)
            torch.cuda.synchronize()
            st = sv.sv_read_device_status()
        finally:
            sv.sv_set_wait_limit_ns(0)
        assert st & ~sv.SV_DEV_TIMEOUT == 0
        assert torch.equal(_call(g, par, 1024, 4), want)
        assert sv.sv_read_device_status() == 0
