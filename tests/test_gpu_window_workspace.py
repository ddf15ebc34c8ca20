"""Workspaces of windowed attention that were sized for another call of the same layers."""
import pytest
import torch

import plain_ops
import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
N, HQ, HKV, D, ROOM, W = 16, 32, 8, 64, 4100, 4001
PAR = wl.chain_parent(N - 1)


def _size(B):
    return sv.sv_window_attention_workspace_size(BF, B, N, HQ, HKV, D, ROOM, W)


def _call(B, workspace):
    """The status of a call of B sequences with this workspace; a result has to be the definition's."""
    lens = [40 + 31 * b % 260 for b in range(B)]
    inp = wl.attention_inputs(B, N, HQ, HKV, D, lens, dtype=BF, seed=B)
    g = {k: inp[k].cuda() for k in ("q", "k_tree", "v_tree", "prefix_len")}
    k, v = (torch.zeros(B, ROOM, HKV, D, dtype=BF, device="cuda") for _ in "kv")  # longer than the prefixes: the size goes by it
    k[:, :inp["cache_k"].shape[1]], v[:, :inp["cache_v"].shape[1]] = inp["cache_k"].cuda(), inp["cache_v"].cuda()
    cache = sv.KVCache(k, v, g["prefix_len"])
    out = torch.full_like(g["q"], float("nan"))
    # (through the C ABI: the Python call makes a workspace where none is passed)
    parent, stride, _ = sv._tree_arg(PAR, B, N)
    code = sv.load_library().sv_window_attention(
        sv.SV_BF16, B, N, HQ, HKV, D, g["q"].data_ptr(), g["k_tree"].data_ptr(), g["v_tree"].data_ptr(), cache.c_struct(),
        parent, stride, D ** -0.5, W, 3, out.data_ptr(), workspace.data_ptr() if workspace.numel() else None, workspace.numel(),
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0
    if code != sv.SV_OK:
        assert torch.isnan(out).all()
        return code
    ref, spread = plain_ops.window_attention(inp["q"], inp["k_tree"], inp["v_tree"], inp["cache_k"], inp["cache_v"],
                                             inp["prefix_len"], PAR, D ** -0.5, W, 3)
    size = D ** -0.5 * inp["q"].float().norm(dim=-1).max().item() * max(inp[x].float().norm(dim=-1).max().item()
                                                                        for x in ("k_tree", "cache_k"))
    assert ((out.double().cpu() - ref).abs() <= plain_ops.attention_bound(ref, spread, BF, D, size, 300 + N)).all()
    return code


def _bytes(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def test_a_size_of_none_serves_every_smaller_batch(cuda_ok):
    """The largest batch asks for no workspace, some of the smaller ones would like one."""
    sizes = [_size(B) for B in range(1, 49)]
    largest = [B for B in range(2, 49) if sizes[B - 1] == 0 and max(sizes[:B - 1]) > 0]
    assert largest  # (of 152 SMs: 12, with 10 and 11 below it)
    for B in range(1, largest[0] + 1):
        for n in (0, 16, 255):  # none, or less than any call asks for
            assert _call(B, _bytes(n)) == sv.SV_OK


def test_a_larger_workspace_serves_and_a_short_one_is_refused(cuda_ok):
    some = max(B for B in range(1, 49) if _size(B) > 0)
    ws = _bytes(_size(some))
    for B in range(1, some + 1, 5):
        assert _size(B) <= ws.numel() and _call(B, ws) == sv.SV_OK
    for n in (256, 4096, ws.numel() - 1):
        assert _call(some, ws[:n]) == sv.SV_ERR_WORKSPACE
