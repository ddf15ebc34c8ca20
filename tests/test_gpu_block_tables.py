"""Block tables and slot maps from request lengths: every entry equals the definition's."""
import numpy as np
import pytest
import torch

import plain_ops
import speculative_decoding_verify_sv_gb300 as sv

pytestmark = pytest.mark.gpu


def _case(length, new, block_size, seed=0, spare=3, head=5, columns=None):
    """A pool in random order: the pages held, `head` taken ids, then the free ones."""
    rng = np.random.RandomState(seed)
    length, new = np.asarray(length), np.asarray(new)
    held = -(-length // block_size)
    total = -(-(length + new) // block_size)
    num_blocks = int(total.sum()) + spare + head
    ids = rng.permutation(num_blocks)
    table = np.full((len(length), columns or max(1, int(total.max()) + 1)), -7)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    free = np.concatenate([np.full(head, -9), ids[at:]])
    return dict(length=length, new=new, table=table, free=free, head=head, num_blocks=num_blocks, block_size=block_size)


def _dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _call(c, num_slots, head=True, **kw):
    table = _dev(c["table"])
    r = sv.sv_block_tables(_dev(c["length"]), _dev(c["new"]), table, _dev(c["free"]), c["block_size"], c["num_blocks"],
                           num_slots, free_head=_dev([c["head"]]) if head else None, **kw)
    return dict(r, block_table=table)


def _check(c, num_slots):
    r = _call(c, num_slots)
    want = plain_ops.block_tables(c["length"], c["new"], c["table"], c["free"], c["head"], c["block_size"], num_slots)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == 0
    for k, v in want.items():
        assert np.array_equal(r[k].cpu().numpy(), v), k


@pytest.mark.parametrize("block_size", [1, 3, 16, 128])
@pytest.mark.parametrize("B", [1, 2, 33, 513, 1537])
def test_ragged_batches(cuda_ok, B, block_size):
    rng = np.random.RandomState(B)
    length, new = rng.randint(0, 70, B), rng.randint(0, 9, B)
    length[0] = 0
    new[B // 2] = 0
    for extra in (0, 1, 7):
        _check(_case(length, new, block_size, seed=B + extra), int(new.sum()) + extra)


def test_edges_of_pages(cuda_ok):
    bs = 16
    length = [0, 0, 0, 15, 16, 17, 15, 16, 31, 32, 1]
    new = [0, 1, 16, 1, 1, 1, 0, 0, 2, 17, 100]
    _check(_case(length, new, bs), sum(new))
    _check(_case(length, new, bs), sum(new) + 2050)


def test_no_new_tokens_and_runs_of_empty_requests(cuda_ok):
    _check(_case([5, 0, 16], [0, 0, 0], 16), 9)
    _check(_case([5, 0, 16], [0, 0, 0], 16), 0)
    _check(_case([3] * 700 + [0], [0] * 700 + [5], 4), 5)
    _check(_case([3] * 700, [2] + [0] * 699, 4), 64)


def test_long_prompts_and_the_largest_batch(cuda_ok):
    rng = np.random.RandomState(3)
    _check(_case(np.zeros(7, int), rng.randint(5000, 40000, 7), 16), 300000)
    _check(_case(rng.randint(0, 40, sv.SV_MAX_TABLE_BATCH), rng.randint(0, 6, sv.SV_MAX_TABLE_BATCH), 8), 50000)


def test_head_defaults_to_the_list_start_and_calls_chain(cuda_ok):
    c = _case([0, 3], [20, 4], 4, head=0)
    r = _call(c, 24, head=False)
    assert int(r["free_head"]) == 5 + 1
    # the next step from the advanced lengths and head
    c2 = dict(c, length=c["length"] + c["new"], new=np.array([3, 9]), table=r["block_table"].cpu().numpy(),
              head=int(r["free_head"]), free=np.concatenate([c["free"], np.arange(100, 120)]), num_blocks=200)
    want = plain_ops.block_tables(c2["length"], c2["new"], np.pad(c2["table"], ((0, 0), (0, 4))), c2["free"], c2["head"],
                                  4, 12)
    c2["table"] = np.pad(c2["table"], ((0, 0), (0, 4)))
    r2 = _call(c2, 12)
    for k, v in want.items():
        assert np.array_equal(r2[k].cpu().numpy(), v), k


def test_shortages_and_bad_ids_are_reported(cuda_ok):
    c = _case([0, 0, 0], [16, 40, 16], 16, head=0, spare=0)
    short = dict(c, free=c["free"][:3])
    r = _call(short, 72)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
    assert int(r["free_head"]) == 5  # two more than there are
    t, s = r["block_table"].cpu().numpy(), r["slots"].cpu().numpy()
    assert t[0, 0] == c["free"][0] and list(t[1, :3]) == [c["free"][1], c["free"][2], -1] and t[2, 0] == -1
    assert (s[:48] >= 0).all() and (s[48:] == -1).all()
    bad = dict(c, free=np.where(np.arange(len(c["free"])) == 0, 10 ** 6, c["free"]))
    r = _call(bad, 72)
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
    assert int(r["block_table"][0, 0]) == -1 and (r["slots"][:16] == -1).all() and (r["slots"][16:] >= 0).all()
    held = _case([5], [3], 16, head=0)
    held["table"][0, 0] = -1
    r = _call(held, 3)
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK and (r["slots"] == -1).all()
    assert r["positions"].tolist() == [5, 6, 7]
    neg = dict(c, head=-1)
    r = _call(neg, 72)
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK and (r["slots"] == -1).all()


def test_lengths_out_of_range_are_clamped_and_reported(cuda_ok):
    c = _case([4, 4, 4], [3, 3, 3], 4, head=0, columns=2)
    cases = (([4, 4, 4], [3, 9, 3]),      # past the table: the part that fits gets slots
             ([4, -2, 4], [3, 3, 3]), ([4, 4, 4], [3, -1, 3]), ([4, 4, 2 ** 31 - 1], [3, 3, 2 ** 31 - 1]))
    for length, new in cases:
        r = _call(dict(c, length=np.array(length), new=np.array(new)), 16)
        torch.cuda.synchronize()
        assert sv.sv_read_device_status() & sv.SV_DEV_BAD_PREFIX
        assert r["slots"][:3].tolist() == [int(r["block_table"][0, 1]) * 4 + i for i in range(3)]
    # a slot map that is too short: its entries are right, and every page is given out
    r = _call(c, 5)
    full = _call(c, 9)
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX
    assert torch.equal(r["slots"], full["slots"][:5]) and torch.equal(r["block_table"], full["block_table"])
    assert torch.equal(r["free_head"], full["free_head"])


def test_graph_replay(cuda_ok):
    c = _case([10, 0, 33, 5], [3, 20, 0, 9], 8, columns=9)
    length, new, table, free = (_dev(c[k]) for k in ("length", "new", "table", "free"))
    head = _dev([c["head"]])
    outs = sv.sv_block_tables(length, new, table, free, 8, c["num_blocks"], 40, free_head=head)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sv_block_tables(length, new, table, free, 8, c["num_blocks"], 40, free_head=head, outs=outs)
    new.copy_(_dev([1, 2, 3, 4]))
    graph.replay()
    torch.cuda.synchronize()
    want = plain_ops.block_tables(c["length"], [1, 2, 3, 4], c["table"], c["free"], c["head"], 8, 40)
    for k in ("token_start", "slots", "positions", "free_head"):
        assert np.array_equal(outs[k].cpu().numpy(), want[k]), k


def test_refusals_and_empty_batch(cuda_ok):
    c = _case([3, 4], [2, 2], 4)
    t = {k: _dev(c[k]) for k in ("length", "new", "table", "free")}
    ok = dict(length=t["length"], new_tokens=t["new"], block_table=t["table"], free_blocks=t["free"], block_size=4,
              num_blocks=c["num_blocks"], num_slots=4)
    call = lambda **kw: sv.sv_block_tables(**{**ok, **kw})  # noqa: E731
    head = _dev([0])
    for bad, code in ((dict(block_size=0), sv.SV_ERR_INVALID_ARG), (dict(num_blocks=0), sv.SV_ERR_INVALID_ARG),
                      (dict(num_blocks=2 ** 30), sv.SV_ERR_UNSUPPORTED),
                      (dict(free_head=head, outs=dict(free_head=head)), sv.SV_ERR_INVALID_ARG)):
        with pytest.raises(sv.SVError) as e:
            call(**bad)
        assert e.value.code == code
    big = torch.zeros(sv.SV_MAX_TABLE_BATCH + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(sv.SVError) as e:
        call(length=big, new_tokens=big, block_table=big.view(-1, 1))
    assert e.value.code == sv.SV_ERR_UNSUPPORTED
    for bad, kind in ((dict(num_slots=-1), ValueError), (dict(new_tokens=t["new"][:1]), ValueError),
                      (dict(length=t["length"].long()), TypeError), (dict(block_table=t["table"][:1]), ValueError),
                      (dict(outs=dict(slots=torch.empty(5, dtype=torch.int32, device="cuda"))), ValueError)):
        with pytest.raises(kind):
            call(**bad)
    n0 = sv.sv_kernel_launches()
    call(length=t["length"][:0], new_tokens=t["new"][:0], block_table=t["table"][:0])
    assert sv.sv_kernel_launches() == n0 and sv.sv_read_device_status() == 0
    # the Python call fills the outputs of a batch without requests: no tokens, the head as it was
    for head, want in ((None, 0), (_dev([7]), 7)):
        r = call(length=t["length"][:0], new_tokens=t["new"][:0], block_table=t["table"][:0], num_slots=6, free_head=head)
        assert r["token_start"].tolist() == [0] and r["free_head"].tolist() == [want]
        assert r["slots"].tolist() == [-1] * 6 and r["positions"].tolist() == [-1] * 6


def test_totals_past_32_bits_end_and_are_reported(cuda_ok):
    """8192 requests of 2^30 new tokens: what the slot map holds is right, the call ends soon."""
    B, bs, columns = sv.SV_MAX_TABLE_BATCH, 2 ** 20, 1024
    table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(1000, -1, -1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    for T in (100, 2 ** 21):
        r = sv.sv_block_tables(zero, zero + 2 ** 30, table, free, bs, 1001, T)
        torch.cuda.synchronize()
        assert sv.sv_read_device_status() == sv.SV_DEV_BAD_PREFIX | sv.SV_DEV_BAD_BLOCK
        at = torch.arange(T, dtype=torch.int64, device="cuda")
        assert torch.equal(r["positions"].long(), at)
        assert torch.equal(r["slots"].long(), (1000 - at // bs) * bs + at % bs)
        assert r["token_start"][:4].tolist() == [0, 2 ** 30, 2 ** 31 - 1, 2 ** 31 - 1]
