"""The compiled calls of the operators around the KV cache beside other threads of the process."""
import threading
import time

import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rope(T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(T, 12 * 64, generator=g, device="cuda").to(BF)
    w = torch.ones(64, device="cuda")
    freq = torch.tensor([10000.0 ** (-i / 32) for i in range(32)], dtype=torch.float64, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + seed
    outs = [torch.zeros(T, h, 64, dtype=BF, device="cuda") for h in (8, 2, 2)]
    return lambda stream=None: sv.sv_qk_norm_rope(qkv, 8, 2, w, w, freq, pos, q_out=outs[0], k_out=outs[1], v_out=outs[2], stream=stream)


def test_a_waiting_launch_does_not_hold_the_other_threads(cuda_ok):
    """Launches behind a long kernel wait once the queue of launches is full; other threads go on."""
    call = _rope(1, 0)
    call()
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)

    other = threading.Thread(target=tick)
    other.start()
    try:
        torch.cuda._sleep(2_000_000_000)  # about a second
        longest = (0.0, 0.0, 0.0)
        for _ in range(6000):
            t0 = time.perf_counter()
            call()
            t1 = time.perf_counter()
            longest = max(longest, (t1 - t0, t0, t1))
        torch.cuda.synchronize()
    finally:
        stop.set()
        other.join()
    took, t0, t1 = longest
    if took < 0.2:
        pytest.skip("no launch had to wait")
    assert sum(t0 <= t <= t1 for t in ticks) >= took / 0.02  # a tick per 20 ms at least, of one per 2


def test_two_threads_at_once(cuda_ok):
    """Calls of two threads, each on a stream of its own: the results of calls one after another."""
    inp = wl.attention_inputs(3, 5, 8, 2, 64, [300, 40, 129], dtype=BF, seed=4)
    g = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
    cache = sv.KVCache(g["cache_k"], g["cache_v"], g["prefix_len"])

    def work(i, stream, found):
        rope, par = _rope(50 + i, i), wl.chain_parent(4)
        new = torch.arange(9, dtype=torch.int32, device="cuda") * (i + 1)
        length = torch.zeros_like(new)
        table, free = torch.full((9, 40), -1, dtype=torch.int32, device="cuda"), torch.arange(400, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        for n in range(200):
            a = sv.sv_window_attention(g["q"], g["k_tree"], g["v_tree"], cache, par, 0.125, 17 + 40 * i + n % 3, sinks=2, stream=stream)
            b = rope(stream)
            c = sv.sv_block_tables(length, new, table, free, 8, 400, 400, stream=stream) if n == 0 else c
            with pytest.raises(sv.SVError) as e:
                sv.sv_window_attention(g["q"], g["k_tree"], g["v_tree"], cache, par, 0.125, -1 - i, stream=stream)
            assert f"window = {-1 - i} " in str(e.value)  # (each thread has its own last error)
        stream.synchronize()
        found[i] = [a, *b, *c.values()]

    streams = [torch.cuda.Stream() for _ in range(2)]
    want, got, failed = {}, {}, []
    for i in range(2):
        work(i, streams[i], want)

    def run(i):
        try:
            work(i, streams[i], got)
        except BaseException as e:  # noqa: BLE001 (shown by the assertion below)
            failed.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(want[i], got[i]))
    assert sv.sv_read_device_status() == 0
