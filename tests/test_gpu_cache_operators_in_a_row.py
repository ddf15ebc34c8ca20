"""The operators around the KV cache right behind one another on a stream, each reading what the one
before wrote: the same bits as with a synchronisation after every call."""
import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv

pytestmark = pytest.mark.gpu

B, N, HQ, HKV, D, BS, BLOCKS, COLUMNS = 24, 5, 8, 2, 64, 16, 700, 24


def _rounds(dtype, rounds, settle):
    """Tables, slots, K/V into the pages, lengths, per-sequence trees and windowed attention, from inputs
    that change every round."""
    g = torch.Generator(device="cuda").manual_seed(7)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda").to(torch.int32)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    weight = torch.ones(D, device="cuda")
    freq = torch.tensor([10000.0 ** (-2 * i / D) for i in range(D // 2)], dtype=torch.float64, device="cuda")
    k, v = randn(BLOCKS, BS, HKV, D), randn(BLOCKS, BS, HKV, D)
    table = torch.zeros(B, COLUMNS, dtype=torch.int32, device="cuda")
    length, parents = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, N, dtype=torch.int32, device="cuda")
    new, free = torch.zeros_like(length), torch.zeros(BLOCKS, dtype=torch.int32, device="cuda")
    cache = sv.KVCache(k, v, length, table, BS)
    found = []
    for _ in range(rounds):
        held, added = ints(0, 180, B), ints(0, 150, B)
        order = torch.randperm(BLOCKS, generator=g, device="cuda").to(torch.int32)
        qkv, tree = randn(B * 152, (HQ + 2 * HKV) * D), randn(B, N, (HQ + 2 * HKV) * D)
        up = torch.stack([torch.full_like(held, -1)] + [ints(0, n, B) for n in range(1, N)], 1)
        torch.cuda.synchronize()
        steps = [lambda: (length.copy_(held), new.copy_(added), free.copy_(order), parents.copy_(up),
                          table[:, :12].copy_(order[:B * 12].view(B, 12)), table[:, 12:].fill_(-1))]
        r = {}
        steps.append(lambda: r.update(sv.sv_block_tables(length, new, table, free[B * 12:], BS, BLOCKS, B * 152)))
        steps.append(lambda: r.update(qkv=sv.sv_qk_norm_rope(qkv, HQ, HKV, weight, weight, freq, r["positions"],
                                                             slots=r["slots"], k_out=k, v_out=v, q_out=torch.zeros(B * 152, HQ, D, dtype=dtype, device="cuda"))))
        steps.append(lambda: length.add_(new))
        steps.append(lambda: r.update(tree=sv.sv_tree_qk_norm_rope(tree, HQ, HKV, weight, weight, freq, length, parents)))
        for window in (60, 300, 1):
            steps.append(lambda w=window: r.update({w: sv.sv_window_attention(*r["tree"], cache, parents, D ** -0.5, w, sinks=3)}))
        for step in steps:
            step()
            if settle:
                torch.cuda.synchronize()
        found.append([table.clone(), k.clone(), v.clone(), length.clone(), r["slots"], r["qkv"][0], *r["tree"], r[60], r[300], r[1]])
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0
    return found


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_calls_in_a_row_read_what_the_one_before_wrote(cuda_ok, dtype):
    want, got = _rounds(dtype, 40, True), _rounds(dtype, 40, False)
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
