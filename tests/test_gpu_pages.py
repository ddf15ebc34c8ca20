"""Bounds, scores and selection of pages against their definitions."""
import math

import pytest
import torch

import plain_pages
import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LENS = [0, 1, 15, 16, 17, 100, 129, 333]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [1, 16, 32, 48, 80, 256])
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (2, 128), (8, 128)])
def test_bounds(cuda_ok, dtype, page, paged, Hkv, D):
    inp = wl.attention_inputs(len(LENS), 1, Hkv, Hkv, D, LENS, dtype=dtype, paged=paged, block_size=page, seed=page)
    g = torch.Generator().manual_seed(1)
    start = torch.tensor([0, 5, 14, -3, 16, 50, 500, 320], dtype=torch.int32)
    rows = (inp["num_blocks"],) if paged else (len(LENS), -(-inp["cache_k"].shape[1] // page))
    before = torch.randn(*rows, Hkv, 2, D, generator=g).to(dtype)
    bt = inp["block_table"]
    cache = sv.KVCache(inp["cache_k"].cuda(), inp["cache_v"].cuda(), inp["prefix_len"].cuda(), bt.cuda() if paged else None, page)
    for s in (start, None):
        to = before.cuda()
        out = sv.sv_page_bounds(cache, to, start=s.cuda() if s is not None else None)
        assert out.data_ptr() == to.data_ptr() and sv.sv_read_device_status() == 0
        want = plain_pages.page_bounds(before, inp["cache_k"], inp["prefix_len"], s, bt, page)
        assert torch.equal(out.cpu(), want)
    new = sv.sv_page_bounds(cache)
    assert new.shape == before.shape
    if paged:  # (rows that hold keys are written)
        at = int(bt[-1, LENS[-1] // page - 1]) if LENS[-1] >= page else int(bt[-1, 0])
        assert torch.equal(new[at].cpu(), want[at])
    else:
        assert torch.equal(new[-1, 0].cpu(), want[-1, 0])


def test_pages_larger_than_the_cache(cuda_ok):
    """One page holds all of a sequence, up to the largest size that there is."""
    inp = wl.attention_inputs(3, 1, 2, 2, 64, [40, 0, 33], paged=False, extra=8, seed=5)
    cache = sv.KVCache(inp["cache_k"].cuda(), inp["cache_v"].cuda(), inp["prefix_len"].cuda(), None, 2 ** 31 - 1)
    bounds = sv.sv_page_bounds(cache, torch.zeros(3, 1, 2, 2, 64, dtype=BF, device="cuda"))
    want = plain_pages.page_bounds(torch.zeros(3, 1, 2, 2, 64, dtype=BF), inp["cache_k"], inp["prefix_len"], None, None, 2 ** 31 - 1)
    assert torch.equal(bounds.cpu(), want)
    _scores(inp["q"], want, inp["prefix_len"], 2 ** 31 - 1, None, False)
    out = sv.sv_select_pages(torch.zeros(3, 1, 2, 1, device="cuda"), cache.prefix_len, 2 ** 31 - 1, 2)
    assert out.cpu().tolist() == [[[[0, -1]] * 2], [[[-1, -1]] * 2], [[[0, -1]] * 2]]
    assert sv.sv_read_device_status() == 0


def test_bounds_keep_what_is_no_number(cuda_ok):
    for dtype in (BF, F32):
        k = torch.randn(1, 48, 2, 64).to(dtype)
        k[0, 3, 1, 5], k[0, 20, 0, 7], k[0, 33, 1, 9] = math.nan, math.inf, -math.inf
        k[0, 47] = math.nan  # (behind the prefix)
        cache = sv.KVCache(k.cuda(), k.cuda(), torch.tensor([47], dtype=torch.int32).cuda(), None, 16)
        out = sv.sv_page_bounds(cache).cpu()
        want = plain_pages.page_bounds(torch.zeros_like(out), k, torch.tensor([47]), None, None, 16)
        assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.nan_to_num(), want.nan_to_num())
        assert out[0, 0, 1, :, 5].isnan().all()


def test_bounds_of_bad_pages_and_prefixes(cuda_ok):
    inp = wl.attention_inputs(2, 1, 2, 2, 64, [40, 40], paged=True, extra=8, seed=3)
    bt = inp["block_table"].clone()
    bt[0, 1], bt[1, 0] = -1, inp["num_blocks"]
    cache = sv.KVCache(inp["cache_k"].cuda(), inp["cache_v"].cuda(), inp["prefix_len"].cuda(), bt.cuda(), 16)
    before = torch.full((inp["num_blocks"], 2, 2, 64), 7.0, dtype=BF)
    out = sv.sv_page_bounds(cache, before.cuda()).cpu()
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
    written = [int(bt[0, 0]), int(bt[0, 2]), int(bt[1, 1]), int(bt[1, 2])]
    for i in range(inp["num_blocks"]):
        assert bool((out[i] == 7).all()) == (i not in written)
    cache.block_table.copy_(inp["block_table"])
    cache.prefix_len[:] = torch.tensor([10 ** 6, -1], dtype=torch.int32)
    out = sv.sv_page_bounds(cache, before.cuda()).cpu()
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
    want = plain_pages.page_bounds(before, inp["cache_k"], torch.tensor([48, 0]), None, inp["block_table"], 16)
    assert torch.equal(out, want)


def _scores(q, bounds, lens, page, bt, per_node):
    out = sv.sv_page_scores(q.cuda(), bounds.cuda(), lens.cuda(), page, block_table=bt.cuda() if bt is not None else None, per_node=per_node)
    assert sv.sv_read_device_status() == 0
    want, size = plain_pages.page_scores(q, bounds, lens, page, bt, per_node)
    out = out.double().cpu()
    assert torch.equal(out.isinf(), want.isinf()) and bool((out[out.isinf()] < 0).all())
    # 2 D products, exact in bf16 and off by 2^-24 in fp32, and as many fp32 additions, which the tensor
    # cores may cut instead of rounding (2^-23 each)
    D = q.shape[-1]
    bound = (2 * D + 2) * 2.0 ** -23 * size
    err = (out - want).abs().nan_to_num()
    assert bool((err <= bound).all()), (err - bound).max()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("per_node", [False, True])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 8, 8, 64), (1, 8, 2, 128), (5, 4, 2, 64), (5, 6, 2, 128), (7, 14, 2, 64),
                                        (26, 16, 2, 128), (64, 12, 1, 64), (64, 20, 1, 128)])
def test_scores(cuda_ok, dtype, paged, per_node, N, Hq, Hkv, D):
    """Sets of 1 to 1280 rows: parts of a step of columns, several steps, several passes over the rows."""
    g = torch.Generator().manual_seed(N + Hq)
    lens = torch.tensor([0, 1, 100, 300, 257, 289], dtype=torch.int32)
    P, page = 19, 16
    q = torch.randn(6, N, Hq, D, generator=g).to(dtype)
    bt = torch.randperm(6 * P, generator=g).to(torch.int32).view(6, P) if paged else None
    x = torch.randn(*((6 * P,) if paged else (6, P)), Hkv, 2, D, generator=g).to(dtype)
    bounds = torch.stack([x.amin(-2), x.amax(-2)], -2).contiguous()
    _scores(q, bounds, lens, page, bt, per_node)


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("per_node", [False, True])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 8, 8, 64), (5, 6, 2, 128), (26, 16, 2, 128), (64, 12, 1, 64), (64, 20, 1, 128)])
def test_scores_of_many_pages(cuda_ok, paged, per_node, N, Hq, Hkv, D):
    """Tiles that are full, partly full and behind the prefix, where the tensor cores are worth it."""
    g = torch.Generator().manual_seed(N + Hq)
    lens = torch.tensor([0, 1, 100, 16 * 700, 16 * 128, 16 * 511 + 3], dtype=torch.int32)
    P, page = 700, 16
    q = torch.randn(6, N, Hq, D, generator=g).to(BF)
    bt = torch.randperm(6 * P, generator=g).to(torch.int32).view(6, P) if paged else None
    x = torch.randn(*((6 * P,) if paged else (6, P)), Hkv, 2, D, generator=g).to(BF)
    bounds = torch.stack([x.amin(-2), x.amax(-2)], -2).contiguous()
    _scores(q, bounds, lens, page, bt, per_node)


def test_scores_bound_every_key(cuda_ok):
    """The chain of operators: no key of a page has a larger product with any row than the page's score."""
    inp = wl.attention_inputs(3, 5, 8, 2, 128, [50, 161, 300], paged=True, seed=9)
    cache = sv.KVCache(inp["cache_k"].cuda(), inp["cache_v"].cuda(), inp["prefix_len"].cuda(), inp["block_table"].cuda(), 16)
    bounds = sv.sv_page_bounds(cache)
    s = sv.sv_page_scores(inp["q"].cuda(), bounds, cache.prefix_len, 16, block_table=cache.block_table, per_node=True).cpu()
    for b, L in enumerate([50, 161, 300]):
        for p in range(L):
            k = inp["cache_k"][int(inp["block_table"][b, p // 16]), p % 16].double()
            for h in range(2):
                y = (inp["q"][b, :, 4 * h:4 * h + 4].double() @ k[h]).amax(-1)
                assert bool((y <= s[b, :, h, p // 16].double() + 1e-3).all())


def test_scores_of_bad_pages_prefixes_and_numbers(cuda_ok):
    q = torch.randn(1, 2, 4, 64).to(BF).cuda()
    bounds = torch.randn(8, 2, 2, 64).to(BF)
    bounds[3, 1, 0, 5] = math.nan
    bt = torch.tensor([[0, 8, 3, -1, 2]], dtype=torch.int32).cuda()
    L = torch.tensor([80], dtype=torch.int32).cuda()
    for dtype in (BF, F32):
        s = sv.sv_page_scores(q.to(dtype), bounds.to(dtype).cuda(), L, 16, block_table=bt).cpu()
        assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
        assert bool(s[0, 0, :, [1, 3]].isneginf().all()) and bool(s[0, 0, :, [0, 4]].isfinite().all())
        assert bool(s[0, 0, 1, 2].isnan()) and bool(s[0, 0, 0, 2].isfinite())
        for n in (10 ** 6, -1):
            s = sv.sv_page_scores(q.to(dtype), bounds.to(dtype).cuda(), torch.full_like(L, n), 16, block_table=bt.clamp(0, 7)).cpu()
            assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
            assert bool(s.isneginf().all()) == (n < 0) and (n < 0 or not bool(s.isneginf().any()))
    # the same entries in a long table, for the tensor cores
    wide = torch.cat([bt] + [bt.clamp(0, 7)] * 399, 1)
    s = sv.sv_page_scores(q, bounds.cuda(), torch.full_like(L, 32000), 16, block_table=wide).cpu()
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
    assert bool(s[0, 0, :, [1, 3]].isneginf().all()) and bool(s[0, 0, 0, 4:].isfinite().all())
    assert bool(s[0, 0, 1, 2].isnan()) and bool(s[0, 0, 0, 2].isfinite()) and bool(s[0, 0, 1, 7::5].isnan().all())
    for n in (10 ** 6, -1):
        s = sv.sv_page_scores(q, bounds.cuda(), torch.full_like(L, n), 16, block_table=wide.clamp(0, 7)).cpu()
        assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
        assert bool(s.isneginf().all()) == (n < 0) and (n < 0 or not bool(s.isneginf().any()))


@pytest.mark.parametrize("P,count,first,last", [(1, 1, 0, 0), (5, 3, 1, 1), (40, 1, 0, 0), (40, 1, 1, 0), (40, 2, 1, 1), (300, 64, 4, 2),
                                                (300, 300, 0, 0), (300, 299, 0, 0), (2048, 256, 1, 4), (2500, 17, 0, 3),
                                                (12000, 512, 1, 1)])
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "wide", "odd"])
def test_select(cuda_ok, P, count, first, last, kind):
    g = torch.Generator().manual_seed(P + count)
    page = 16
    lens = torch.tensor([P * page, max(0, P * page - 15), (P * page) // 2, 0, 1, min(P, count + 1) * page], dtype=torch.int32)
    B, S, H = 6, 3, 2
    x = torch.randn(B, S, H, P, generator=g)
    if kind == "ties":
        x = (x * 2).round()
    elif kind == "equal":
        x = torch.full_like(x, -2.5)
    elif kind == "wide":
        x = x * torch.exp(40 * torch.randn(B, S, H, P, generator=g))
    elif kind == "odd":  # zeros of both signs, infinities, NaN
        x = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, 1e-42, -1e-42, 3.0])[torch.randint(0, 8, x.shape, generator=g)]
    out = sv.sv_select_pages(x.cuda(), lens.cuda(), page, count, first=first, last=last)
    assert sv.sv_read_device_status() == 0
    assert torch.equal(out.cpu(), plain_pages.select_pages(x, lens, page, count, first, last))


def test_select_at_the_largest_size(cuda_ok):
    x = torch.randn(1, 1, 2, 32768, generator=torch.Generator().manual_seed(2))
    lens = torch.tensor([32768 * 16], dtype=torch.int32)
    out = sv.sv_select_pages(x.cuda(), lens.cuda(), 16, 2000, first=1, last=1)
    assert torch.equal(out.cpu(), plain_pages.select_pages(x, lens, 16, 2000, 1, 1))


def test_select_clamps_prefixes(cuda_ok):
    x = torch.randn(2, 1, 1, 10).cuda()
    out = sv.sv_select_pages(x, torch.tensor([1000, -5], dtype=torch.int32).cuda(), 16, 4).cpu()
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
    assert bool((out[1] == -1).all())
    assert torch.equal(out[:1], plain_pages.select_pages(x[:1].cpu(), torch.tensor([160]), 16, 4, 1, 1))
