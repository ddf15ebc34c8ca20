"""The waits of windowed attention's few-row kernel, made to run out: a limit far below a copy's time is
reached in every call, the call ends soon, says so, and the next one is right.  (Nothing hangs: the
waits are bounded, the test shortens their bound.)"""
import time

import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


# one warp per slice in a cluster and without one, two warps per slice with held and with loaded rows
@pytest.mark.parametrize("B,N,Hq,Hkv,window", [(1, 1, 8, 1, 1024), (64, 1, 32, 8, 100), (64, 5, 32, 8, 700), (2, 16, 64, 2, 1024),
                                               (64, 5, 64, 8, 513), (8, 64, 32, 32, 513)])
@pytest.mark.parametrize("paged", [False, True])
def test_a_wait_that_runs_out_is_reported(cuda_ok, B, N, Hq, Hkv, window, paged):
    D, L, bs = 128, 1600, 16
    par = wl.TREE_T64 if N == 64 else wl.chain_parent(N - 1)
    g = torch.Generator(device="cuda").manual_seed(B + N)
    q, kt, vt = (torch.randn(B, N, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    shape, table = (B, L, Hkv, D), None
    if paged:
        shape = (B * L // bs, bs, Hkv, D)
        table = torch.randperm(shape[0], generator=g, device="cuda").to(torch.int32).view(B, L // bs)
    k, v = (torch.randn(*shape, generator=g, device="cuda").to(BF) for _ in "kv")
    length = torch.randint(L // 2, L - 70, (B,), generator=g, device="cuda").to(torch.int32)
    cache = sv.KVCache(k, v, length, table, bs)
    assert sv.sv_window_attention_workspace_size(BF, B, N, Hq, Hkv, D, cache.max_prefix, window) == 0

    def call():
        out = sv.sv_window_attention(q, kt, vt, cache, par, D ** -0.5, window, sinks=4)
        torch.cuda.synchronize()
        return out

    want = call()
    assert sv.sv_read_device_status() == 0
    for _ in range(3):
        try:
            sv.sv_set_wait_limit_ns(1)
            begin = time.perf_counter()
            call()
            took = time.perf_counter() - begin
            status = sv.sv_read_device_status()
        finally:
            sv.sv_set_wait_limit_ns(0)
        assert status == sv.SV_DEV_TIMEOUT
        assert took < 1.0  # (nobody waits two seconds for a copy that was never made)
        assert torch.equal(call(), want) and sv.sv_read_device_status() == 0
