"""Per-head norms with the position rotation against the definition in 64 bits."""
import pytest
import torch

import plain_ops
import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _inputs(T, Hq, Hkv, D, rot, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(T, (Hq + 2 * Hkv) * D + pad, generator=g).to(dtype)
    return dict(qkv=wide[:, pad:], qw=1 + 0.3 * torch.randn(D, generator=g), kw=1 + 0.3 * torch.randn(D, generator=g),
                inv=torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64))


def _compare(got, inp, positions, Hq, Hkv, eps, interleaved):
    D = inp["qw"].numel()
    (q, k, v), sizes = plain_ops.qk_norm_rope(inp["qkv"], Hq, Hkv, inp["qw"], inp["kw"], inp["inv"], positions, eps,
                                              interleaved)
    for x, ref, size in ((got[0], q, sizes[0]), (got[1], k, sizes[1])):
        over = ((x.double().cpu().reshape(ref.shape) - ref).abs() /
                plain_ops.rope_bound(ref, size, x.dtype, D).clamp(min=1e-30)).max().item()
        assert over <= 1.0, over
    assert torch.equal(got[2].cpu().reshape(v.shape).double(), v)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_rotations_and_slices(cuda_ok, dtype, D, rot, interleaved):
    for Hq, Hkv, T, pad in ((4, 4, 1, 0), (32, 4, 3, 16), (5, 1, 9, 8), (7, 7, 2, 0)):
        inp = _inputs(T, Hq, Hkv, D, rot, dtype, seed=T + D + rot, pad=pad)
        positions = torch.tensor([0, 1, 131071, 7, 2 ** 31 - 1, 511, 4096, 65536, 12345][:T], dtype=torch.int32)
        dev = {k: v.cuda() for k, v in inp.items()}
        wide = torch.zeros(T, inp["qkv"].shape[1] + pad, dtype=dtype, device="cuda")
        wide[:, pad:] = dev["qkv"]
        got = sv.sv_qk_norm_rope(wide[:, pad:], Hq, Hkv, dev["qw"], dev["kw"], dev["inv"], positions.cuda(), eps=1e-5,
                                 interleaved=interleaved)
        _compare(got, inp, positions, Hq, Hkv, 1e-5, interleaved)
    assert sv.sv_read_device_status() == 0


@pytest.mark.parametrize("T", [1, 2, 151, 1216, 3000])
def test_many_tokens(cuda_ok, T):
    """Every division of a token's heads over warps, and several tokens per warp."""
    inp = _inputs(T, 8, 2, 64, 32, BF, seed=T)
    positions = torch.arange(T, dtype=torch.int32) * 7
    dev = {k: v.cuda() for k, v in inp.items()}
    got = sv.sv_qk_norm_rope(dev["qkv"], 8, 2, dev["qw"], dev["kw"], dev["inv"], positions.cuda())
    _compare(got, inp, positions, 8, 2, 1e-6, False)


def test_frequencies_of_all_sizes_and_signs(cuda_ok):
    """Turns per position from double frequencies: zero, subnormal, whole turns, negative, and up to
    2^30 (the positions are powers of two, so that the definition's products are exact)."""
    inp = _inputs(4, 3, 2, 64, 64, F32, seed=21)
    special = [0.0, -0.0, 5e-324, 1e-310, 2.0 ** -1022, 1e-20, -1e-20, 2.0 ** -64, -2.0 ** -63, -1e-3, 0.5, -0.5, 1.0, -1.0,
               6.283185307179586, -6.283185307179586, 0.7853981633974483, 1.5707963267948966, 3.0, 100.25, -1234.5678,
               2.0 ** 20 + 0.1, 2.0 ** 30 + 0.3, -2.0 ** 30 - 0.7]
    inp["inv"] = torch.tensor(special + [0.1 * (i + 1) for i in range(32 - len(special))], dtype=torch.float64)
    positions = torch.tensor([0, 1, 2, 4], dtype=torch.int32)
    dev = {k: v.cuda() for k, v in inp.items()}
    for interleaved in (False, True):
        got = sv.sv_qk_norm_rope(dev["qkv"], 3, 2, dev["qw"], dev["kw"], dev["inv"], positions.cuda(), interleaved=interleaved)
        _compare(got, inp, positions, 3, 2, 1e-6, interleaved)


def test_slots_and_padding(cuda_ok):
    """K/V go to their slots and nowhere else; padding tokens and negative slots write nothing."""
    T, Hq, Hkv, D, rows = 12, 8, 2, 128, 64
    inp = _inputs(T, Hq, Hkv, D, 128, BF, seed=3)
    positions = torch.arange(100, 100 + T, dtype=torch.int32)
    positions[[4, 11]] = -1
    slots = torch.randperm(rows, generator=torch.Generator().manual_seed(4))[:T].to(torch.int32)
    slots[7] = -1
    inp["qkv"][4] = float("nan")
    dev = {k: v.cuda() for k, v in inp.items()}
    kc = torch.full((4, 16, Hkv, D), 3.0, dtype=BF, device="cuda")
    vc = torch.full_like(kc, -3.0)
    qo = torch.full((T, Hq, D), 9.0, dtype=BF, device="cuda")
    q, k, v = sv.sv_qk_norm_rope(dev["qkv"], Hq, Hkv, dev["qw"], dev["kw"], dev["inv"], positions.cuda(),
                                 slots=slots.cuda(), q_out=qo, k_out=kc, v_out=vc)
    assert q is qo and k is kc and v is vc
    full = sv.sv_qk_norm_rope(dev["qkv"], Hq, Hkv, dev["qw"], dev["kw"], dev["inv"], positions.abs().cuda())
    expect_k, expect_v = torch.full_like(kc, 3.0).view(rows, Hkv, D), torch.full_like(vc, -3.0).view(rows, Hkv, D)
    live = [t for t in range(T) if positions[t] >= 0]
    for t in live:
        assert torch.equal(qo[t], full[0][t])
        if slots[t] >= 0:
            expect_k[slots[t]], expect_v[slots[t]] = full[1][t], full[2][t]
    assert (qo[[4, 11]] == 9.0).all()
    assert torch.equal(kc.view(rows, Hkv, D), expect_k) and torch.equal(vc.view(rows, Hkv, D), expect_v)
    assert sv.sv_read_device_status() == 0
    slots[0] = rows  # beyond the pool: skipped and reported
    sv.sv_qk_norm_rope(dev["qkv"], Hq, Hkv, dev["qw"], dev["kw"], dev["inv"], positions.cuda(), slots=slots.cuda(),
                       q_out=qo, k_out=kc, v_out=vc)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_BLOCK
    assert torch.equal(kc.view(rows, Hkv, D), expect_k)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_rows(cuda_ok, dtype):
    """Positions from the prefix lengths and the depths of a shared or of each sequence's tree."""
    B, Hq, Hkv, D = 3, 8, 2, 128
    lens = torch.tensor([0, 777, 32768], dtype=torch.int32)
    g = torch.Generator().manual_seed(8)
    own = [[-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, 64)] for _ in range(B)]
    own[1] = wl.chain_parent(63)
    for parent in (wl.TREE_T26, wl.TREE_T64, [-1], own):
        rows = parent if parent is own else [parent] * B
        N = len(rows[0])
        inp = _inputs(B * N, Hq, Hkv, D, 128, dtype, seed=N)
        dev = {k: v.cuda() for k, v in inp.items()}
        arg = torch.tensor(own, dtype=torch.int32, device="cuda") if parent is own else parent
        got = sv.sv_tree_qk_norm_rope(dev["qkv"].view(B, N, -1), Hq, Hkv, dev["qw"], dev["kw"], dev["inv"],
                                      lens.cuda(), arg)
        assert got[0].shape == (B, N, Hq, D) and got[1].shape == got[2].shape == (B, N, Hkv, D)
        positions = torch.tensor([[int(L) + d for d in wl.depths(r)] for L, r in zip(lens, rows)])
        _compare(got, inp, positions, Hq, Hkv, 1e-6, False)
    assert sv.sv_read_device_status() == 0
    bad = torch.tensor([wl.chain_parent(4), [-1, 0, 3, 1, 2], wl.chain_parent(4)], dtype=torch.int32, device="cuda")
    inp = {k: v.cuda() for k, v in _inputs(15, Hq, Hkv, D, 128, dtype, seed=5).items()}
    sv.sv_tree_qk_norm_rope(inp["qkv"].view(3, 5, -1), Hq, Hkv, inp["qw"], inp["kw"], inp["inv"], lens.cuda(), bad)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status() == sv.SV_DEV_BAD_TREE


def test_norm_of_extreme_rows(cuda_ok):
    """A row of zeros stays zero; eps counts; a large common factor changes the result by
    roundings only."""
    Hq, Hkv, D = 2, 1, 64
    inp = {k: v.cuda() for k, v in _inputs(2, Hq, Hkv, D, 64, F32, seed=6).items()}
    pos = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    args = (Hq, Hkv, inp["qw"], inp["kw"], inp["inv"], pos)
    zero = sv.sv_qk_norm_rope(torch.zeros_like(inp["qkv"]), *args)
    assert all((x == 0).all() for x in zero)
    one = sv.sv_qk_norm_rope(inp["qkv"], *args, eps=0.0)
    big = sv.sv_qk_norm_rope(inp["qkv"] * 2.0 ** 40, *args, eps=0.0)
    for a, b in zip(one[:2], big[:2]):
        assert (a - b).abs().max().item() <= 2.0 ** -20 * a.abs().max().item()


def test_graph_and_stream(cuda_ok):
    inp = {k: v.cuda() for k, v in _inputs(40, 8, 2, 128, 128, BF, seed=9).items()}
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    call = lambda **kw: sv.sv_qk_norm_rope(inp["qkv"], 8, 2, inp["qw"], inp["kw"], inp["inv"], pos, **kw)  # noqa: E731
    outs = [torch.empty_like(x) for x in call()]
    names = dict(zip(("q_out", "k_out", "v_out"), outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(**names)
    pos.add_(1000)
    inp["qkv"].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, call()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pos.add_(1)
    want = call()
    s.wait_stream(torch.cuda.current_stream())
    call(stream=s, **names)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals_and_empty_calls(cuda_ok):
    inp = {k: v.cuda() for k, v in _inputs(4, 8, 2, 64, 64, BF, seed=1).items()}
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    ok = dict(qkv=inp["qkv"], Hq=8, Hkv=2, q_weight=inp["qw"], k_weight=inp["kw"], inv_freq=inp["inv"], positions=pos)
    call = lambda **kw: sv.sv_qk_norm_rope(**{**ok, **kw})  # noqa: E731
    call()
    for bad, kind in ((dict(qkv=inp["qkv"].half()), TypeError), (dict(Hq=9), ValueError),
                      (dict(q_weight=inp["qw"].to(BF)), TypeError), (dict(inv_freq=inp["inv"].float()), TypeError),
                      (dict(k_weight=inp["kw"][:32]), ValueError), (dict(positions=pos[:3]), ValueError),
                      (dict(positions=pos.long()), TypeError), (dict(slots=pos), ValueError),
                      (dict(qkv=inp["qkv"].t().contiguous().t()), ValueError),
                      (dict(k_out=torch.empty(4, 2, 32, dtype=BF, device="cuda")), ValueError)):
        with pytest.raises(kind):
            call(**bad)
    for bad, code in ((dict(inv_freq=inp["inv"][:4]), sv.SV_ERR_UNSUPPORTED),
                      (dict(inv_freq=torch.ones(40, dtype=torch.float64, device="cuda")), sv.SV_ERR_UNSUPPORTED),
                      (dict(eps=-1.0), sv.SV_ERR_INVALID_ARG), (dict(eps=float("nan")), sv.SV_ERR_INVALID_ARG),
                      (dict(q_out=inp["qkv"].reshape(-1)[:4 * 512].view(4, 8, 64)), sv.SV_ERR_INVALID_ARG)):
        with pytest.raises(sv.SVError) as e:
            call(**bad)
        assert e.value.code == code
    with pytest.raises(sv.SVError):  # no slots: a row for every token
        call(k_out=torch.empty(3, 2, 64, dtype=BF, device="cuda"), v_out=torch.empty(3, 2, 64, dtype=BF, device="cuda"))
    n0 = sv.sv_kernel_launches()
    q, k, v = call(qkv=inp["qkv"][:0], positions=pos[:0])
    assert q.shape == (0, 8, 64) and k.shape == v.shape == (0, 2, 64)
    q, k, v = sv.sv_tree_qk_norm_rope(inp["qkv"][:0].view(0, 5, 768), 8, 2, inp["qw"], inp["kw"], inp["inv"], pos[:0],
                                      wl.chain_parent(4))
    assert q.shape == (0, 5, 8, 64)
    assert sv.sv_kernel_launches() == n0 and sv.sv_read_device_status() == 0
