"""Block tables of requests that hold more pages than their lengths reach: rounds that ask for the
longest path's tokens and keep those of the accepted one."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv

gpu = pytest.mark.gpu


def _dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _plain(length, new, held, table, free, head, bs, num_slots):
    table, out = table.copy(), []
    slots, positions, start = [], [], [0]
    for b in range(len(length)):
        have = max(-(-int(length[b]) // bs), int(held[b]))
        total = -(-(int(length[b]) + int(new[b])) // bs)
        for j in range(have, total):
            table[b, j] = free[head]
            head += 1
        out.append(max(have, total))
        for p in range(int(length[b]), int(length[b]) + int(new[b])):
            slots.append(int(table[b, p // bs]) * bs + p % bs)
            positions.append(p)
        start.append(len(slots))
    pad = [-1] * (num_slots - len(slots))
    return dict(block_table=table, held=np.array(out), free_head=np.array([head]), token_start=np.array(start),
                slots=np.array(slots + pad)[:num_slots], positions=np.array(positions + pad)[:num_slots])


@gpu
@pytest.mark.parametrize("bs", [1, 3, 16, 64])
@pytest.mark.parametrize("B,most", [(1, 40), (7, 3000), (300, 9), (2500, 5), (8192, 3)])
def test_held_pages(cuda_ok, B, most, bs):
    """Rows that hold fewer pages than their length needs, as many, and up to many more."""
    rng = np.random.RandomState(B + bs)
    length, new = rng.randint(0, 60, B), rng.randint(0, most, B)
    new[0] = most - 1
    reach = -(-length // bs)
    held = np.maximum(reach + rng.randint(-1, 6, B), 0)
    have = np.maximum(held, reach)
    total = int(new.sum())
    columns = int(np.maximum(have, -(-(length + new) // bs)).max()) + 1
    blocks = int(have.sum()) + total + 5
    ids = rng.permutation(blocks)
    table, at = np.full((B, columns), -7), 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = np.concatenate([[-9] * 2, ids[at:]])
    for T in sorted({total, total + 5, max(0, total - 2), total // 2}):
        want = _plain(length, new, held, table, free, 2, bs, T)
        t = _dev(table)
        r = sv.sv_block_tables(_dev(length), _dev(new), t, _dev(free), bs, blocks, T, free_head=_dev([2]), held=_dev(held))
        torch.cuda.synchronize()
        assert sv.sv_read_device_status() == (sv.SV_DEV_BAD_PREFIX if T < total else 0)
        assert sorted(r) == ["free_head", "held", "positions", "slots", "token_start"]
        for k, v in dict(r, block_table=t).items():
            assert np.array_equal(v.cpu().numpy(), want[k]), k


@gpu
@pytest.mark.parametrize("graph", [False, True])
def test_rounds_lose_no_page(cuda_ok, graph):
    """Forty rounds without a look at the device: no page stands in two rows, none is lost, and the
    rows' pages are those that the free list gave out."""
    B, bs, columns, blocks, ask = 6, 4, 80, 400, 7
    rng = np.random.RandomState(3)
    free = rng.permutation(blocks)
    table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
    length, held, head = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, B, 1))
    new, kept, ids = torch.full((B,), ask, dtype=torch.int32, device="cuda"), torch.zeros_like(length), _dev(free)
    outs = sv.sv_block_tables(length, new, table.clone(), ids, bs, blocks, B * ask, free_head=head, held=held)

    def one_round():
        sv.sv_block_tables(length, new, table, ids, bs, blocks, B * ask, free_head=head, held=held, outs=outs)
        length.add_(kept)  # what the accepted paths commit
        head.copy_(outs["free_head"])
        held.copy_(outs["held"])

    captured = torch.cuda.CUDAGraph()
    if graph:
        with torch.cuda.graph(captured):
            one_round()
    at, most = np.zeros(B, int), np.zeros(B, int)
    for _ in range(40):
        keep = rng.randint(1, ask + 1, B)
        kept.copy_(_dev(keep))
        if graph:
            captured.replay()
        else:
            one_round()
        most = np.maximum(most, -(-(at + ask) // bs))
        at += keep
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0
    t = table.cpu().numpy()
    assert held.tolist() == most.tolist() and length.tolist() == at.tolist()
    rows = [t[b, :most[b]].tolist() for b in range(B)]
    assert all((t[b, most[b]:] == -1).all() for b in range(B))
    given = sorted(x for row in rows for x in row)
    assert given == sorted(free[:int(head)].tolist()) and int(head) == most.sum()


@gpu
def test_odd_counts_are_clamped_and_reported(cuda_ok):
    bs = 4
    length, new, free = _dev([5, 5]), _dev([3, 3]), _dev([7, 8])
    for bad in (-1, 9, 2 ** 31 - 1, -2 ** 31):
        table = _dev([[1, 2, -1, -1], [3, 4, -1, -1]])
        r = sv.sv_block_tables(length, new, table, free, bs, 10, 6, held=_dev([bad, 2]))
        torch.cuda.synchronize()
        assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
        assert r["held"].tolist() == [4 if bad > 0 else 2, 2] and r["free_head"].tolist() == [0]
        assert r["slots"].tolist() == [9, 10, 11, 17, 18, 19]


@gpu
def test_empty_batch_and_wrong_tensors(cuda_ok):
    none = _dev([])
    r = sv.sv_block_tables(none, none, none.view(0, 3), _dev([1]), 4, 8, 2, held=none)
    assert r["held"].shape == (0,) and r["slots"].tolist() == [-1, -1]
    length, table = _dev([5, 5]), _dev([[1, 2], [3, 4]])
    for held, kind in ((_dev([1]), ValueError), (_dev([1, 2]).long(), TypeError)):
        with pytest.raises(kind):
            sv.sv_block_tables(length, length, table, _dev([1]), 4, 8, 2, held=held)
    held = _dev([2, 2])
    with pytest.raises(sv.SVError) as e:
        sv.sv_block_tables(length, length, table, _dev([1]), 4, 8, 2, held=held, outs=dict(held=held))
    assert e.value.code == sv.SV_ERR_INVALID_ARG


def test_refusals_before_launch():
    from speculative_decoding_verify_sv_gb300 import build as svbuild
    svbuild.build()
    lib, at = sv.load_library(), lambda n: ctypes.c_void_p(n << 20)

    def call(held=at(7), out=at(8), B=2, bs=16):
        return lib.sv_block_tables_held(B, at(1), at(2), bs, 4, 64, at(3), 8, at(4), held, at(5), 8, at(6), at(9), at(10), at(11),
                                        out, None)
    bad = sv.SV_ERR_INVALID_ARG
    assert call(held=None) == bad and call(out=None) == bad and call(out=at(7)) == bad and call(bs=0) == bad
    assert call(out=ctypes.c_void_p((7 << 20) + 4)) == bad and b"out_held" in lib.sv_last_error()
    assert call(B=0, held=None, out=None) == sv.SV_OK


def test_overlaps_are_refused():
    """The table and every output against one another and against every input (host addresses only)."""
    from speculative_decoding_verify_sv_gb300 import build as svbuild
    svbuild.build()
    lib, bad = sv.load_library(), sv.SV_ERR_INVALID_ARG
    B, mb, T, num_free = 5, 6, 8, 9
    names = ["length", "new", "free", "head", "held", "table", "start", "slots", "positions", "out_head", "out_held"]
    words = dict(length=B, new=B, free=num_free, head=1, held=B, table=B * mb, start=B + 1, slots=T, positions=T, out_head=1, out_held=B)

    def call(with_held, **over):
        at = {n: (i + 1) << 20 for i, n in enumerate(names)}
        at.update(over)
        p = {n: ctypes.c_void_p(x) for n, x in at.items()}
        if with_held:
            return lib.sv_block_tables_held(B, p["length"], p["new"], 16, mb, 64, p["free"], num_free, p["head"], p["held"], p["table"],
                                            T, p["start"], p["slots"], p["positions"], p["out_head"], p["out_held"], None)
        return lib.sv_block_tables(B, p["length"], p["new"], 16, mb, 64, p["free"], num_free, p["head"], p["table"], T, p["start"],
                                   p["slots"], p["positions"], p["out_head"], None)
    for with_held in (False, True):
        for w in names[5:]:
            for o in names:
                if o == w or (not with_held and "held" in w + o):
                    continue
                base = (names.index(o) + 1) << 20
                # the first and the last word that they share (slots and positions stay 16-byte aligned)
                step = 16 if w in ("slots", "positions") else 4
                for at in (base, base + 4 * (words[o] - 1) // step * step):
                    assert call(with_held, **{w: at}) == bad, (w, o)
                    assert b"overlap" in lib.sv_last_error() or {w, o} == {"out_head", "head"}
