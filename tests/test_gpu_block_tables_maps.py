"""Block tables whose slot map is too short for the batch, and long prompts mixed with everything else:
every entry equals the definition's."""
import numpy as np
import pytest
import torch

import plain_ops
import speculative_decoding_verify_sv_gb300 as sv

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _check(length, new, block_size, num_slots, seed=0):
    """A batch against the definition; entries that the call does not write keep what they held."""
    rng = np.random.RandomState(seed)
    length, new = np.asarray(length), np.asarray(new)
    held, need = -(-length // block_size), -(-(length + new) // block_size)
    blocks = int(need.sum()) + 9
    ids = rng.permutation(blocks)
    table = np.full((len(length), int(need.max()) + 2), -7)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    free = np.concatenate([np.full(4, -9), ids[at:]])
    want = plain_ops.block_tables(length, new, table, free, 4, block_size, max(num_slots, int(new.sum())))
    t = _dev(table)
    r = sv.sv_block_tables(_dev(length), _dev(new), t, _dev(free), block_size, blocks, num_slots, free_head=_dev([4]))
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == (sv.SV_DEV_BAD_PREFIX if new.sum() > num_slots else 0)
    assert np.array_equal(t.cpu().numpy(), want["block_table"])
    for k in ("token_start", "free_head"):
        assert np.array_equal(r[k].cpu().numpy(), want[k]), k
    for k in ("slots", "positions"):
        assert np.array_equal(r[k].cpu().numpy(), want[k][:num_slots]), k


@pytest.mark.parametrize("B,block_size", [(1, 16), (2, 1), (37, 16), (300, 3), (2500, 16), (8192, 2)])
def test_short_maps_give_every_page_out(cuda_ok, B, block_size):
    rng = np.random.RandomState(B)
    length, new = rng.randint(0, 50, B), rng.randint(0, 40, B)
    new[rng.rand(B) < 0.3] = 0
    new[0] = 33
    total = int(new.sum())
    for T in sorted({0, 1, 15, 16, 17, total // 3, total // 2 + 1, total - 1, total}):
        _check(length, new, block_size, T, seed=B + T)


def test_short_maps_of_long_prompts(cuda_ok):
    rng = np.random.RandomState(1)
    new = rng.randint(3000, 9000, 6)
    for T in (6 * 256, 6 * 256 + 3, 20001, int(new.sum()) - 2):
        _check(rng.randint(0, 40, 6), new, 16, T, seed=T)


@pytest.mark.parametrize("block_size", [1, 3, 16, 48, 4096])
def test_long_prompts_between_empty_and_short_requests(cuda_ok, block_size):
    """Four neighbouring places per thread: held pages that are partly filled, requests without tokens
    between long ones, several short requests within one group of four, maps of any length."""
    length = [5, 0, 17, 31, 0, 1, 2, 3, 4, 700, 16, 0, 9]
    new = [4097, 0, 0, 3, 1, 1, 0, 1, 2, 5000, 0, 7, 3001]
    total = sum(new)
    for T in (total - 3, total, total + 1, total + 2, total + 3, total + 4, total + 2050):
        assert T // len(new) >= 256
        _check(length, new, block_size, T, seed=T)


def test_bad_ids_among_long_prompts(cuda_ok):
    """A held and a free id outside the pool, and a free list that ends: exactly their tokens get none."""
    bs, length, new = 16, [5, 40, 0], [2000, 1500, 900]
    table = np.full((3, 130), -7)
    table[0, 0], table[1, :3] = 3, [4, 10 ** 6, -2]
    need = [-(-(a + b) // bs) - -(-a // bs) for a, b in zip(length, new)]
    free = np.arange(10, 10 + sum(need) - 5)  # five pages short
    free[7] = 400
    t = _dev(table)
    r = sv.sv_block_tables(_dev(length), _dev(new), t, _dev(free), bs, 400, 4402)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
    assert r["free_head"].tolist() == [sum(need)]
    ids = np.concatenate([free, [-1] * 5])
    ids[7] = -1
    want, at = table.copy(), 0
    for b in range(3):
        first = -(-length[b] // bs)
        want[b, first:first + need[b]] = ids[at:at + need[b]]
        at += need[b]
    assert np.array_equal(t.cpu().numpy(), want)
    good = np.where((want >= 0) & (want < 400), want, -1)
    slots = []
    for b in range(3):
        for p in range(length[b], length[b] + new[b]):
            slots.append(good[b, p // bs] * bs + p % bs if good[b, p // bs] >= 0 else -1)
    assert r["slots"].tolist() == slots + [-1] * 2


def test_pages_of_tokens_past_32_bits(cuda_ok):
    """Three requests of 2^30 new tokens and a map of 100 places: all 3072 pages are given out, in
    milliseconds (a walk over 2^31 tokens takes seconds on the one CTA that such a map needs)."""
    bs, columns, blocks = 2 ** 20, 1024, 2047
    free = np.arange(3 * columns) % blocks
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    for T in (100, 0):
        t = torch.full((3, columns), -7, dtype=torch.int32, device="cuda")
        args = (zero, zero + 2 ** 30, t, _dev(free), bs, blocks, T)
        sv.sv_block_tables(*args)
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        r = sv.sv_block_tables(*args)
        end.record()
        torch.cuda.synchronize()
        assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
        assert np.array_equal(t.cpu().numpy().reshape(-1), free)
        assert r["free_head"].tolist() == [3 * columns] and r["slots"].tolist() == list(range(T))
        assert begin.elapsed_time(end) < 20


def test_a_refused_empty_batch_writes_nothing(cuda_ok):
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    outs = {k: torch.full((n,), 7, dtype=torch.int32, device="cuda")
            for k, n in (("token_start", 1), ("slots", 4), ("positions", 4), ("free_head", 1))}
    for kw in (dict(block_size=0), dict(num_blocks=0), dict(num_blocks=2 ** 30)):
        with pytest.raises(sv.SVError):
            sv.sv_block_tables(none, none, none.view(0, 3), _dev([1]), **{**dict(block_size=4, num_blocks=8), **kw}, num_slots=4, outs=outs)
        assert all((t == 7).all() for t in outs.values())
    sv.sv_block_tables(none, none, none.view(0, 3), _dev([1]), 4, 8, 4, outs=outs)
    assert [outs[k].tolist() for k in ("token_start", "slots", "positions", "free_head")] == [[0], [-1] * 4, [-1] * 4, [0]]
