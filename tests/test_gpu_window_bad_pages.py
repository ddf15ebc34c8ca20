"""Windowed attention with page ids outside the pool: their keys are left out, by every kernel."""
import math

import pytest
import torch

import plain_ops
import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _without(inp, b, parent, window, sinks, bs, gone):
    """Sequence b's result in 64 bits without the prefix positions `gone`, and sum(p |v|)."""
    L, table = int(inp["prefix_len"][b]), inp["block_table"]
    path = plain_ops.paths(parent)
    keep = [p for p in range(L) if (p < sinks or L - p < window) and p not in gone]
    at = [int(table[b, p // bs]) * bs + p % bs for p in keep]
    q = inp["q"][b].double()
    N, Hq, D = q.shape
    Hkv = inp["k_tree"].shape[2]
    k, v = (torch.cat([c.reshape(-1, Hkv, D)[at], t[b]]).double() for c, t in ((inp["cache_k"], inp["k_tree"]), (inp["cache_v"], inp["v_tree"])))
    out, spread = torch.zeros_like(q), torch.zeros_like(q)
    for n in range(N):
        P = L + len(path[n]) - 1
        see = [P - p < window or p < sinks for p in keep]
        see += [j in path[n] and (P - (L + len(path[j]) - 1) < window or L + len(path[j]) - 1 < sinks) for j in range(N)]
        for h in range(Hq):
            g = h * Hkv // Hq
            s = (k[:, g] @ q[n, h] * D ** -0.5).masked_fill(~torch.tensor(see), -math.inf)
            w = torch.softmax(s, 0)
            out[n, h], spread[n, h] = w @ v[:, g], w @ v[:, g].abs()
    return out, spread


# few rows, fp32, and the 128-row kernel with one and two tiles of rows, of both head dims
@pytest.mark.parametrize("dtype,B,N,Hq,Hkv,D,bs", [(BF, 3, 5, 8, 2, 128, 16), (F32, 3, 5, 8, 2, 64, 16),
                                                   (BF, 64, 26, 32, 8, 128, 16), (BF, 64, 26, 32, 8, 64, 64),
                                                   (BF, 64, 26, 64, 8, 128, 32), (BF, 64, 26, 64, 8, 64, 16),
                                                   (BF, 40, 16, 32, 8, 128, 128), (BF, 64, 26, 64, 8, 128, 256)])
def test_keys_of_bad_pages_are_left_out(cuda_ok, dtype, B, N, Hq, Hkv, D, bs):
    par = {5: wl.chain_parent(4), 26: wl.TREE_T26, 16: wl.chain_parent(15)}[N]
    window, sinks = (3500, 21) if N == 16 else (260, 21)
    lens = [700 - 13 * (b % 7) for b in range(B)]
    inp = wl.attention_inputs(B, N, Hq, Hkv, D, lens, dtype=dtype, paged=True, block_size=bs, seed=B + bs)
    if B > 3:
        limit = inp["block_table"].shape[1] * bs
        if not sv.sv_window_attention_workspace_size(dtype, B, N, Hq, Hkv, D, limit, window):
            pytest.skip("not a shape of the 128-row kernel on this device")

    def call(table):
        cache = sv.KVCache(inp["cache_k"].cuda(), inp["cache_v"].cuda(), inp["prefix_len"].cuda(), table.cuda(), bs)
        return sv.sv_window_attention(inp["q"].cuda(), inp["k_tree"].cuda(), inp["v_tree"].cuda(), cache, par, D ** -0.5,
                                      window, sinks=sinks).cpu()

    good = call(inp["block_table"])
    assert sv.sv_read_device_status() == 0
    blocks = inp["cache_k"].shape[0]
    L = lens[1]
    # a page in the window, the last one (partly filled), one of the sinks, and all of them
    every = list(range(-(-L // bs)))
    for pages in ([(L - 100) // bs], [(L - 1) // bs], [0], every):
        ref, spread = _without(inp, 1, par, window, sinks, bs, {p for p in range(L) if p // bs in pages})
        size = D ** -0.5 * inp["q"][1].float().norm(dim=-1).max().item() * max(
            inp["k_tree"][1].float().norm(dim=-1).max().item(), inp["cache_k"].float().norm(dim=-1).max().item())
        bound = plain_ops.attention_bound(ref, spread, dtype, D, size, 800)
        for bad in (-1, blocks, 2 ** 31 - 1, -2 ** 31):
            table = inp["block_table"].clone()
            table[1, pages] = bad
            out = call(table)
            assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
            rest = [0] + list(range(2, B))
            assert torch.equal(out[rest], good[rest])
            assert torch.isfinite(out[1]).all() and ((out[1].double() - ref).abs() <= bound).all(), (pages, bad)
