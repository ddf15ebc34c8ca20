"""Selection of pages in the shapes that many lists go to (a warp per list, more scores per thread): ties, equal
scores, infinities and NaN, more candidates than fit, short and empty prefixes."""
import math

import pytest
import torch

import plain_pages
import speculative_decoding_verify_sv_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,count,first,last", [(1, 1, 0, 1), (33, 5, 1, 1), (500, 64, 4, 2), (512, 511, 0, 0), (513, 8, 0, 0), (1000, 200, 1, 4),
                                                (1024, 1, 0, 0), (1025, 1, 1, 0), (2048, 100, 1, 1), (8192, 64, 1, 1), (8200, 64, 1, 1)])
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "outlier", "odd"])
def test_select_of_many_lists(cuda_ok, P, count, first, last, kind):
    lists = -(-4 * torch.cuda.get_device_properties(0).multi_processor_count // 8)
    B, page = lists, 16
    g = torch.Generator().manual_seed(P + count)
    lens = torch.tensor([(P * page, max(0, P * page - 15), (P * page) // 2, 0, 1, min(P, count + 1) * page)[i % 6] for i in range(B)],
                        dtype=torch.int32)
    x = torch.randn(B, 4, 2, P, generator=g)
    if kind == "ties":
        x = (x * 2).round()
    elif kind == "equal":
        x[:] = -2.5
    elif kind == "outlier":  # nearly all of the scores in one part of their range
        x[..., P // 2] = 1e30
    elif kind == "odd":
        x[..., ::5], x[..., 1::7], x[..., 2::11] = math.inf, -math.inf, math.nan
        x[1] = -math.inf
        x[2] = math.nan
    out = sv.sv_select_pages(x.cuda(), lens.cuda(), page, count, first, last)
    assert sv.sv_read_device_status() == 0
    some = [0, 1, 2, 3, 4, 5, B - 1]  # (the oracle is slow: sequences of each length, and the last)
    want = plain_pages.select_pages(x[some], lens[some], page, count, first, last)
    assert torch.equal(out.cpu()[some], want)
    assert bool((out.cpu()[lens == 0] == -1).all())
    for b in range(6, B - 1, 29):
        n = -(-int(lens[b]) // page)
        if n > count:
            assert torch.equal(out[b].cpu(), plain_pages.select_pages(x[b:b + 1], lens[b:b + 1], page, count, first, last)[0])


def test_lists_with_bad_prefixes(cuda_ok):
    B = -(-4 * torch.cuda.get_device_properties(0).multi_processor_count // 8)
    x = torch.randn(B, 4, 2, 100, device="cuda")
    lens = torch.full((B,), 1600, dtype=torch.int32, device="cuda")
    want = sv.sv_select_pages(x, lens, 16, 7)
    assert sv.sv_read_device_status() == 0
    lens[5], lens[9] = 10 ** 6, -3
    got = sv.sv_select_pages(x, lens, 16, 7)
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
    want[9] = -1
    assert torch.equal(got, want)
