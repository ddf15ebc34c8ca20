"""The 128-row attention kernel's bounded waits, made to run out where warps hold real rows beside
padding: every lane leaves together, the call returns and says so, and the next one is right.  (The
waits are bounded, the test shortens their bound.)"""
import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


# 20, 104 and 208 rows: row copies, one M tile, two of them; units cut over several CTAs
@pytest.mark.parametrize("B,N,Hq,Hkv,window", [(1, 5, 4, 1, 0), (3, 26, 32, 8, 0), (3, 26, 64, 8, 0), (16, 26, 32, 8, 0),
                                               (16, 26, 64, 8, 0), (16, 26, 32, 8, 2048), (16, 26, 64, 8, 2048)])
def test_padding_rows_leave_with_the_others(cuda_ok, B, N, Hq, Hkv, window):
    D, L = 128, 9000 if B == 1 else 3000
    par = wl.chain_parent(4) if N == 5 else wl.TREE_T26
    g = torch.Generator(device="cuda").manual_seed(B + N)
    q, kt, vt = (torch.randn(B, N, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    k, v = (torch.randn(B, L + 8, Hkv, D, generator=g, device="cuda").to(BF) for _ in "kv")
    cache = sv.KVCache(k, v, torch.full((B,), L, dtype=torch.int32, device="cuda"))
    if window:
        size = sv.sv_window_attention_workspace_size(BF, B, N, Hq, Hkv, D, L + 8, window)
        assert size > 0
    else:
        assert sv.sv_tree_attention_path(BF, N, Hq, Hkv, D) == 1
        size = sv.sv_tree_attention_workspace_size(BF, B, N, Hq, Hkv, D, L + 8)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def call():
        out = (sv.sv_window_attention(q, kt, vt, cache, par, D ** -0.5, window, sinks=4, workspace=ws) if window else
               sv.sv_tree_attention(q, kt, vt, cache, par, D ** -0.5, workspace=ws))
        torch.cuda.synchronize()
        return out

    want = call()
    assert sv.sv_read_device_status() == 0
    for limit in (1, 1000):
        try:
            sv.sv_set_wait_limit_ns(limit)
            call()
            status = sv.sv_read_device_status()
        finally:
            sv.sv_set_wait_limit_ns(0)
        assert status & ~sv.SV_DEV_TIMEOUT == 0 and (status or limit > 1)
        assert torch.equal(call(), want) and sv.sv_read_device_status() == 0
