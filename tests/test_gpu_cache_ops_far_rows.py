"""The operators around the KV cache past 2^31 elements: the same bits as on a small pool."""
import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _randn(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


# few rows, fp32, the 128-row kernel
@pytest.mark.parametrize("dtype,B,N,Hq", [(BF, 3, 5, 32), (F32, 2, 5, 32), (BF, 32, 26, 64)])
@pytest.mark.parametrize("paged", [True, False])
def test_windowed_attention_of_far_rows(cuda_ok, dtype, B, N, Hq, paged):
    Hkv, D, bs, window = 8, 128, 16, 700
    par = wl.chain_parent(4) if N == 5 else wl.TREE_T26
    need = B * 50  # pages of 800 positions each
    k, v = _randn(1, need, bs, Hkv, D, dtype=dtype), _randn(2, need, bs, Hkv, D, dtype=dtype)
    q, kt, vt = (_randn(3 + i, B, N, h, D, dtype=dtype) for i, h in enumerate((Hq, Hkv, Hkv)))
    length = torch.tensor([790 - 31 * (b % 9) for b in range(B)], dtype=torch.int32, device="cuda")
    table = torch.randperm(need, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(B, 50).cuda()
    if N == 26:
        assert sv.sv_window_attention_workspace_size(dtype, B, N, Hq, Hkv, D, 800, window) > 0

    def call(k, v, table):
        return sv.sv_window_attention(q, kt, vt, sv.KVCache(k, v, length, table, bs), par, D ** -0.5, window, sinks=5)

    if paged:
        want = call(k, v, table)
        blocks = (2 ** 31 + 2 ** 26) // (bs * Hkv * D) + need
        far_k, far_v = (torch.zeros(blocks, bs, Hkv, D, dtype=dtype, device="cuda") for _ in "kv")
        far_k[-need:], far_v[-need:] = k, v
        got = call(far_k, far_v, table + (blocks - need))
    else:
        # the last sequence of a contiguous cache ends past 2^31 elements
        rows = (2 ** 31 + 2 ** 26) // (B * Hkv * D) + 800
        dense = torch.stack([x[table.long()].reshape(B, 800, Hkv, D) for x in (k, v)])
        want = call(dense[0], dense[1], None)
        far_k, far_v = (torch.zeros(B, rows, Hkv, D, dtype=dtype, device="cuda") for _ in "kv")
        far_k[:, :800], far_v[:, :800] = dense[0], dense[1]
        got = call(far_k, far_v, None)
        size = sv.sv_window_attention_workspace_size(dtype, B, N, Hq, Hkv, D, 800, window)
        assert size == sv.sv_window_attention_workspace_size(dtype, B, N, Hq, Hkv, D, rows, window)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotation_from_and_to_far_rows(cuda_ok, dtype):
    Hq, Hkv, D, T = 32, 8, 128, 64
    width = (Hq + 2 * Hkv) * D
    w = torch.ones(D, device="cuda")
    freq = torch.tensor([10000.0 ** (-i / 64) for i in range(64)], dtype=torch.float64, device="cuda")
    many = (2 ** 31 + 2 ** 26) // width + T  # tokens of qkv
    far = torch.zeros(many, width, dtype=dtype, device="cuda")
    few = _randn(8, T, width, dtype=dtype)
    far[-T:] = few
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    want = sv.sv_qk_norm_rope(few, Hq, Hkv, w, w, freq, pos)
    # all but the last tokens are padding; K and V go to the end of a pool past 2^31 elements
    rows = (2 ** 31 + 2 ** 26) // (Hkv * D)
    k, v = (torch.zeros(rows, Hkv, D, dtype=dtype, device="cuda") for _ in "kv")
    slots, far_pos = (torch.full((many,), -1, dtype=torch.int32, device="cuda") for _ in "sp")
    slots[-T:], far_pos[-T:] = torch.arange(rows - T, rows, dtype=torch.int32, device="cuda"), pos
    q, _, _ = sv.sv_qk_norm_rope(far, Hq, Hkv, w, w, freq, far_pos, slots=slots, k_out=k, v_out=v)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0
    assert torch.equal(q[-T:], want[0]) and torch.equal(k[-T:], want[1]) and torch.equal(v[-T:], want[2])
    assert not k[:-T].any() and not v[:-T].any()
