"""Host-side refusals of the operators around the KV cache, through the C ABI and the compiled
Python calls, before anything is launched (CPU only; no call needs a device)."""
import ctypes

import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import build as svbuild

P = ctypes.c_void_p(1 << 20)
FAR, FAR2, FAR3 = (ctypes.c_void_p(k << 40) for k in (1, 2, 3))


@pytest.fixture(scope="module")
def lib():
    svbuild.build()
    return sv.load_library()


def _cache(**kw):
    c = sv._KVCacheC()
    c.k = c.v = c.prefix_len = 1 << 20
    c.Lmax = 128
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _window(lib, dt=1, B=1, N=1, Hq=4, Hkv=4, D=128, q=P, cache=None, scale=0.1, window=16, sinks=0, out=P):
    par = (ctypes.c_int32 * max(N, 1))(*range(-1, max(N, 1) - 1))
    return lib.sv_window_attention(dt, B, N, Hq, Hkv, D, q, P, P, cache or _cache(), par, 0, scale, window, sinks, out,
                                   None, 0, None)


def test_window_attention_rejects_before_launch(lib):
    bad, no = sv.SV_ERR_INVALID_ARG, sv.SV_ERR_UNSUPPORTED
    paged = dict(block_table=1 << 20, block_size=16, max_blocks=8, num_blocks=8)
    for code, kw in ((bad, dict(window=0)), (bad, dict(window=-5)), (bad, dict(sinks=-1)), (no, dict(sinks=65)),
                     (bad, dict(scale=0.0)), (bad, dict(scale=-1.0)), (bad, dict(scale=float("nan"))),
                     (bad, dict(scale=float("inf"))), (no, dict(D=96)), (no, dict(dt=2)), (bad, dict(Hq=6)),
                     (bad, dict(Hkv=0)), (bad, dict(B=-1)), (bad, dict(N=0)), (no, dict(N=65)), (bad, dict(q=None)),
                     (bad, dict(q=ctypes.c_void_p(18))), (bad, dict(out=None)), (bad, dict(cache=_cache(k=None))),
                     (bad, dict(cache=_cache(Lmax=-1))), (no, dict(cache=_cache(**dict(paged, block_size=24)))),
                     (bad, dict(cache=_cache(**dict(paged, block_size=0)))),
                     (no, dict(cache=_cache(Lmax=2 ** 31 - 1))), (no, dict(B=2 ** 20, cache=_cache(Lmax=4096))),
                     (no, dict(cache=_cache(**dict(paged, num_blocks=2 ** 28))))):
        assert _window(lib, **kw) == code, kw
        assert lib.sv_last_error() != b""
    # an output on top of an input
    far = dict(cache=_cache(k=1 << 40, v=1 << 41), q=FAR3)
    for out in (3 << 40, (3 << 40) + 1008, 1 << 20, (1 << 40) + 1024, (1 << 41) + 128 * 4 * 128 * 2 - 16):
        assert _window(lib, out=ctypes.c_void_p(out), **far) == bad and b"overlaps" in lib.sv_last_error(), out
    # a workspace for the 128-row kernel; sizes that need none, and sizes that are none
    assert lib.sv_window_attention_workspace_size(1, 64, 26, 64, 8, 128, 4096, 2048) > 0
    assert lib.sv_window_attention_workspace_size(1, 256, 5, 32, 8, 128, 8192, 1024) == 0
    assert lib.sv_window_attention_workspace_size(0, 64, 26, 64, 8, 128, 4096, 2048) == 0
    assert lib.sv_window_attention_workspace_size(1, 64, 26, 64, 8, 128, 4096, 0) == 0
    assert lib.sv_window_attention_workspace_size(1, 64, 26, 63, 8, 128, 4096, 2048) == 0
    # an empty batch needs no device and no tensors
    assert _window(lib, B=0, q=None, out=None, cache=_cache(k=None, v=None, prefix_len=None)) == sv.SV_OK


def _tables(lib, B=2, length=P, new=P, bs=16, mb=4, nb=64, free=P, num_free=8, head=P, table=P, T=8, start=P, slots=P,
            positions=P, out_head=FAR):
    return lib.sv_block_tables(B, length, new, bs, mb, nb, free, num_free, head, table, T, start, slots, positions,
                               out_head, None)


def test_block_tables_rejects_before_launch(lib):
    bad, no = sv.SV_ERR_INVALID_ARG, sv.SV_ERR_UNSUPPORTED
    for code, kw in ((bad, dict(B=-1)), (bad, dict(T=-1)), (bad, dict(num_free=-1)), (no, dict(B=8193)),
                     (bad, dict(bs=0)), (bad, dict(mb=0)), (bad, dict(nb=0)), (no, dict(nb=2 ** 27)),
                     (bad, dict(length=None)), (bad, dict(new=None)), (bad, dict(table=None)), (bad, dict(start=None)),
                     (bad, dict(slots=None)), (bad, dict(positions=None)), (bad, dict(out_head=None)),
                     (bad, dict(free=None)), (bad, dict(slots=ctypes.c_void_p(8))),
                     (bad, dict(positions=ctypes.c_void_p(4))), (bad, dict(out_head=P))):
        assert _tables(lib, **kw) == code, kw
    assert _tables(lib, B=0, length=None, new=None, table=None, start=None, slots=None, positions=None, out_head=None,
                   free=None, head=None) == sv.SV_OK


def _rope(lib, dt=1, T=4, Hq=8, Hkv=2, D=128, rot=128, qkv=P, ld=1536, qw=P, kw=P, eps=1e-6, freq=P, positions=P,
          slots=None, rows=4, q=FAR, k=FAR2, v=FAR3):
    return lib.sv_qk_norm_rope(dt, T, Hq, Hkv, D, rot, 0, qkv, ld, qw, kw, eps, freq, positions, slots, rows, q, k, v, None)


def test_qk_norm_rope_rejects_before_launch(lib):
    bad, no = sv.SV_ERR_INVALID_ARG, sv.SV_ERR_UNSUPPORTED
    inside = ctypes.c_void_p((1 << 20) + 4 * 1536 * 2 - 16)  # the last bytes of qkv
    for code, kw in ((bad, dict(T=-1)), (no, dict(dt=5)), (bad, dict(Hq=0)), (bad, dict(Hkv=0)), (no, dict(D=80)),
                     (no, dict(rot=0)), (no, dict(rot=24)), (no, dict(rot=144)), (bad, dict(ld=1535)),
                     (bad, dict(ld=1540)), (bad, dict(eps=-1.0)), (bad, dict(eps=float("nan"))), (bad, dict(qkv=None)),
                     (bad, dict(qw=None)), (bad, dict(kw=None)), (bad, dict(freq=None)), (bad, dict(positions=None)),
                     (bad, dict(q=None)), (bad, dict(k=None)), (bad, dict(v=None)), (bad, dict(q=ctypes.c_void_p(8))),
                     (bad, dict(rows=3)), (bad, dict(rows=-1)), (bad, dict(q=inside)), (bad, dict(k=inside)),
                     (bad, dict(v=P)), (bad, dict(k=FAR)), (bad, dict(v=FAR2)), (no, dict(rows=2 ** 41)), (no, dict(Hq=2 ** 25, ld=2 ** 40))):
        assert _rope(lib, **kw) == code, kw
    # row distances and row counts whose bytes pass 64 bits
    assert _rope(lib, T=2 ** 31 - 1, ld=2 ** 45, rows=2 ** 31) == no and _rope(lib, ld=2 ** 62) == no
    assert _rope(lib, Hkv=2 ** 23, ld=2 ** 33, Hq=1, D=64, rot=64, rows=2 ** 33) == no
    assert _rope(lib, T=0, qkv=None, qw=None, kw=None, freq=None, positions=None, q=None, k=None, v=None, rows=0) == sv.SV_OK
    par = (ctypes.c_int32 * 3)(-1, 0, 0)

    def tree(B=2, N=3, parent=par, prefix=P, rot=64):
        return lib.sv_tree_qk_norm_rope(1, B, N, 8, 2, 128, rot, 0, P, 1536, P, P, 1e-6, P, prefix, parent, 0, FAR, FAR2, FAR3,
                                        None)
    assert tree(B=-1) == bad and tree(N=0) == bad and tree(N=65) == no and tree(prefix=None) == bad
    assert tree(parent=(ctypes.c_int32 * 3)(-1, 2, 0)) == bad and tree(parent=None) == bad and tree(rot=12) == no
    assert tree(B=0, prefix=None) == sv.SV_OK


def test_python_calls_refuse_what_is_no_cuda_tensor(lib):
    t = torch.zeros(2, 1, 4, 64)
    i = torch.zeros(2, dtype=torch.int32)
    cache = sv.KVCache(t, t, i)
    for call in (lambda: sv.sv_window_attention(t, t, t, cache, [-1], 1.0, 4),
                 lambda: sv.sv_window_attention(None, t, t, cache, [-1], 1.0, 4),
                 lambda: sv.sv_block_tables(i, i, i.view(2, 1), i, 16, 4, 8),
                 lambda: sv.sv_block_tables([1, 2], i, i.view(2, 1), i, 16, 4, 8),
                 lambda: sv.sv_qk_norm_rope(t.view(2, -1), 2, 1, t, t, t, i),
                 lambda: sv.sv_tree_qk_norm_rope(t.view(2, 1, -1), 2, 1, t, t, t, i, [-1])):
        with pytest.raises(TypeError):
            call()
