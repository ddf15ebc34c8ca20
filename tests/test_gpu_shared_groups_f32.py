"""What sv_shared_attention says of groups that are none, in float32, where every sequence's own rows are read: the
status that the header names, and the same outputs as without groups."""
import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv
import test_gpu_shared_attention as shared
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

F32 = torch.float32
# sequences with one CTA per unit, and with a cluster of them
SIZES = [([3, 2], [200, 100], [0, 5, 33, 8, 9], 5, 8, 2, 128), ([1, 1], [900, 700], [3, 40], 1, 4, 2, 64),
         ([40, 30], [64, 16], [3] * 70, 26, 16, 8, 64)]


def tree(N):
    return wl.TREE_T26 if N == 26 else wl.chain_parent(N - 1)


@pytest.mark.parametrize("sizes,lens,own,N,Hq,Hkv,D", SIZES)
@pytest.mark.parametrize("page", [0, 16])
def test_bad_groups_are_reported(cuda_ok, sizes, lens, own, N, Hq, Hkv, D, page):
    inp = shared.shared_inputs(sizes, lens, own, N, Hq, Hkv, D, dtype=F32, page=page, seed=1)
    want = shared.call(inp, tree(N), page)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0
    B = sum(sizes)
    for starts in ([0, B, B - 1], [-1, 1, B], [0, 1, B + 1], [2, 1, B], [0, 2 ** 31 - 1, B]):
        inp["group_start"] = torch.tensor(starts, dtype=torch.int32)
        out = shared.call(inp, tree(N), page)
        torch.cuda.synchronize()
        assert sv.sv_read_device_status() == sv.SV_DEV_BAD_GROUP, starts
        assert torch.equal(out, want)


@pytest.mark.parametrize("sizes,lens,own,N,Hq,Hkv,D", SIZES)
def test_shared_lengths_that_are_none_are_reported(cuda_ok, sizes, lens, own, N, Hq, Hkv, D):
    inp = shared.shared_inputs(sizes, lens, own, N, Hq, Hkv, D, dtype=F32, seed=2)
    want = shared.call(inp, tree(N))
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0
    cap = inp["block_table"].shape[1] * 16
    last = int(inp["prefix_len"][-1])
    for length in ([lens[0], -5], [cap + 1, lens[1]], [lens[0], last + 1]):  # below, beyond the cache, beyond a member's prefix
        inp["shared_len"] = torch.tensor(length, dtype=torch.int32)
        out = shared.call(inp, tree(N))
        torch.cuda.synchronize()
        assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX, length
        assert torch.equal(out, want)  # (every sequence's own rows)
    # an empty group's length is beyond nobody's prefix
    inp["shared_len"] = torch.tensor([lens[0], cap], dtype=torch.int32)
    inp["group_start"] = torch.tensor([0, sizes[0], sizes[0]], dtype=torch.int32)
    assert torch.equal(shared.call(inp, tree(N)), want) and sv.sv_read_device_status() == 0


@pytest.mark.parametrize("N", [1, 5])
def test_windows_know_no_groups(cuda_ok, N):
    """The kernel is the sliding window's too, which has none to report."""
    inp = shared.shared_inputs([3], [70], [1, 2, 3], N, 8, 2, 64, dtype=F32, seed=3)
    g = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
    cache = sv.KVCache(g["cache_k"], g["cache_v"], g["prefix_len"], g["block_table"], 16)
    out = sv.sv_window_attention(g["q"], g["k_tree"], g["v_tree"], cache, tree(N), 0.1, 32, sinks=2)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0 and bool(out.isfinite().all())
