"""The waits of windowed attention's few-row kernel, made to run out: with a limit far below a copy's
time calls end soon and say so, and the next one is right.  (Nothing hangs: the
waits are bounded, the test shortens their bound.)"""
import time

import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


# clusters, one warp per slice without one, two warps per slice (held and loaded rows): enough memory
# traffic that copies are waited for
@pytest.mark.parametrize("B,N,Hq,Hkv,L,window", [(4, 1, 32, 8, 20000, 16384), (64, 1, 32, 8, 9000, 8192), (256, 5, 32, 8, 2000, 1024),
                                                 (64, 5, 64, 8, 2000, 513), (64, 16, 32, 8, 2000, 513)])
@pytest.mark.parametrize("paged", [False, True])
def test_a_wait_that_runs_out_is_reported(cuda_ok, B, N, Hq, Hkv, L, window, paged):
    D, bs = 128, 16
    par = wl.chain_parent(N - 1)
    g = torch.Generator(device="cuda").manual_seed(B + N)
    q, kt, vt = (torch.randn(B, N, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    rows = L // bs * bs
    shape, table = (B, rows, Hkv, D), None
    if paged:
        shape = (B * rows // bs, bs, Hkv, D)
        table = torch.randperm(shape[0], generator=g, device="cuda").to(torch.int32).view(B, rows // bs)
    k, v = (torch.empty(*shape, dtype=BF, device="cuda").normal_(generator=g) for _ in "kv")
    length = torch.randint(rows - 400, rows - 70, (B,), generator=g, device="cuda").to(torch.int32)
    cache = sv.KVCache(k, v, length, table, bs)
    if sv.sv_window_attention_workspace_size(BF, B, N, Hq, Hkv, D, cache.max_prefix, window):
        pytest.skip("not a shape of the few-row kernel on this device")
    out = torch.empty_like(q)

    def call():
        sv.sv_window_attention(q, kt, vt, cache, par, D ** -0.5, window, sinks=4, out=out)
        torch.cuda.synchronize()
        return sv.sv_read_device_status()

    assert call() == 0
    want, found = out.clone(), []
    for _ in range(12):
        try:
            sv.sv_set_wait_limit_ns(1)
            begin = time.perf_counter()
            found.append(call())
            took = time.perf_counter() - begin
        finally:
            sv.sv_set_wait_limit_ns(0)
        assert took < 1.0  # (nobody waits two seconds for a copy that was never made)
        assert call() == 0 and torch.equal(out, want)
    # (a call whose copies all land before they are waited for is right and says nothing)
    assert set(found) <= {0, sv.SV_DEV_TIMEOUT} and sv.SV_DEV_TIMEOUT in found
