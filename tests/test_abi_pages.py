"""Host-side refusals of the operators for shared prefixes and selected pages, through the C ABI and the
compiled Python calls, before anything is launched (CPU only; no call needs a device)."""
import ctypes

import pytest
import torch

import speculative_decoding_verify_sv_gb300 as sv
from speculative_decoding_verify_sv_gb300 import build as svbuild

P = ctypes.c_void_p(1 << 20)
FAR, FAR2, FAR3 = (ctypes.c_void_p(k << 40) for k in (1, 2, 3))
BAD, NO, SMALL = sv.SV_ERR_INVALID_ARG, sv.SV_ERR_UNSUPPORTED, sv.SV_ERR_WORKSPACE
PAGED = dict(block_table=1 << 20, block_size=16, max_blocks=8, num_blocks=8)


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


def _parent(N):
    return (ctypes.c_int32 * max(N, 1))(*range(-1, max(N, 1) - 1))


def _shared(lib, dt=1, B=1, N=1, Hq=4, Hkv=4, D=128, q=P, cache=None, parent="chain", scale=0.1, start=P, length=P, groups=1, out=FAR,
            ws=FAR2, ws_bytes=1 << 40):
    return lib.sv_shared_attention(dt, B, N, Hq, Hkv, D, q, P, P, cache or _cache(), _parent(N) if parent == "chain" else parent, 0,
                                   scale, start, length, groups, out, ws, ws_bytes, None)


def _sparse(lib, dt=1, B=1, N=1, Hq=4, Hkv=4, D=128, q=P, cache=None, parent="chain", scale=0.1, pages=P, sets=1, K=4, page=16, out=FAR,
            ws=FAR2, ws_bytes=1 << 40):
    return lib.sv_sparse_attention(dt, B, N, Hq, Hkv, D, q, P, P, cache or _cache(), _parent(N) if parent == "chain" else parent, 0,
                                   scale, pages, sets, K, page, out, ws, ws_bytes, None)


def test_both_attentions_reject_before_launch(lib):
    for code, kw in ((BAD, dict(scale=0.0)), (BAD, dict(scale=-1.0)), (BAD, dict(scale=float("nan"))), (BAD, dict(scale=float("inf"))),
                     (NO, dict(D=96)), (NO, dict(dt=2)), (BAD, dict(Hq=6)), (BAD, dict(Hkv=0)), (BAD, dict(B=-1)), (BAD, dict(N=0)),
                     (NO, dict(N=65)), (NO, dict(Hq=129, Hkv=1)), (BAD, dict(q=None)), (BAD, dict(q=ctypes.c_void_p(18))),
                     (BAD, dict(out=None)), (BAD, dict(out=ctypes.c_void_p((1 << 40) + 8))), (BAD, dict(parent=None)),
                     (BAD, dict(N=3, parent=(ctypes.c_int32 * 3)(-1, 2, 0))), (BAD, dict(cache=_cache(k=None))),
                     (BAD, dict(cache=_cache(Lmax=-1))), (NO, dict(cache=_cache(**dict(PAGED, block_size=24)))),
                     (BAD, dict(cache=_cache(**dict(PAGED, block_size=0)))), (NO, dict(cache=_cache(Lmax=2 ** 31 - 1))),
                     (NO, dict(B=2 ** 20, cache=_cache(Lmax=4096))), (NO, dict(cache=_cache(**dict(PAGED, num_blocks=2 ** 28))))):
        for call in (_shared, _sparse):
            assert call(lib, **kw) == code, (call, kw)
            assert lib.sv_last_error() != b""
    far = dict(cache=_cache(k=4 << 40, v=5 << 40), q=FAR3)
    for out in (3 << 40, (3 << 40) + 1008, 1 << 20, (4 << 40) + 1024, (5 << 40) + 128 * 4 * 128 * 2 - 16):
        for call in (_shared, _sparse):
            assert call(lib, out=ctypes.c_void_p(out), **far) == BAD and b"overlaps" in lib.sv_last_error(), out
    for call in (_shared, _sparse):  # an empty batch needs no device and no tensors
        assert call(lib, B=0, q=None, out=None, cache=_cache(k=None, v=None, prefix_len=None), ws=None, ws_bytes=0) == sv.SV_OK
    assert _shared(lib, B=0, q=None, out=None, start=None, length=None, cache=_cache(k=None, v=None, prefix_len=None)) == sv.SV_OK
    assert _sparse(lib, B=0, q=None, out=None, pages=None, cache=_cache(k=None, v=None, prefix_len=None)) == sv.SV_OK


def test_shared_attention_rejects_its_own(lib):
    need = lib.sv_shared_attention_workspace_size(1, 1, 1, 4, 4, 128, 1 << 20, 1)
    assert need > 0 and lib.sv_shared_attention_workspace_size(1, 1, 1, 4, 4, 128, 128, 1) == 0
    big = dict(cache=_cache(Lmax=1 << 20))
    for code, kw in ((BAD, dict(groups=0)), (BAD, dict(groups=-1)), (NO, dict(groups=129)), (BAD, dict(start=None)), (BAD, dict(length=None)),
                     (SMALL, dict(big, ws=None)), (SMALL, dict(big, ws_bytes=need - 1)), (BAD, dict(big, ws=ctypes.c_void_p((2 << 40) + 8)))):
        assert _shared(lib, **kw) == code, kw
    sizes = lib.sv_shared_attention_workspace_size
    assert sizes(1, 64, 5, 32, 8, 128, 4096, 128) > sizes(1, 64, 5, 32, 8, 128, 4096, 1) > 0
    for args in ((0, 64, 5, 32, 8, 128, 4096, 1), (1, 0, 5, 32, 8, 128, 4096, 1), (1, 64, 65, 32, 8, 128, 4096, 1), (1, 64, 5, 31, 8, 128, 4096, 1),
                 (1, 64, 5, 32, 8, 96, 4096, 1), (1, 64, 5, 32, 8, 128, -1, 1), (1, 64, 5, 32, 8, 128, 4096, 0), (1, 64, 5, 32, 8, 128, 4096, 129)):
        assert sizes(*args) == 0, args


def test_sparse_attention_rejects_its_own(lib):
    sizes = lib.sv_sparse_attention_workspace_size
    big = dict(N=26, Hq=64, Hkv=8, K=4096)
    need = sizes(1, 1, 26, 64, 8, 128, 16, 4096, 1)
    assert need > 0 and sizes(1, 1, 1, 4, 4, 128, 16, 4, 1) == 0
    for code, kw in ((BAD, dict(K=0)), (BAD, dict(K=-1)), (BAD, dict(sets=2)), (BAD, dict(sets=0)), (BAD, dict(N=3, sets=2)), (BAD, dict(page=0)),
                     (NO, dict(page=24)), (BAD, dict(page=32, cache=_cache(**PAGED))), (NO, dict(K=2 ** 28, page=16)), (BAD, dict(pages=None)),
                     (NO, dict(B=2 ** 15, N=32, sets=32, Hq=32, Hkv=32, cache=_cache(Lmax=16))), (SMALL, dict(big, ws=None)),
                     (SMALL, dict(big, ws_bytes=need - 1)), (BAD, dict(big, ws=ctypes.c_void_p((2 << 40) + 4)))):
        assert _sparse(lib, **kw) == code, kw
    assert _sparse(lib, pages=ctypes.c_void_p((1 << 40) + 512)) == BAD and b"overlaps" in lib.sv_last_error()
    for args in ((0, 64, 26, 64, 8, 128, 16, 4096, 1), (1, 64, 26, 64, 8, 128, 16, 4096, 26), (1, 0, 26, 64, 8, 128, 16, 4096, 1),
                 (1, 64, 26, 64, 8, 128, 8, 4096, 1), (1, 64, 26, 64, 8, 128, 16, 0, 1), (1, 64, 26, 64, 8, 80, 16, 4096, 1),
                 (1, 64, 26, 64, 8, 128, 16, 4096, 2), (1, 64, 26, 63, 8, 128, 16, 4096, 1)):
        assert sizes(*args) == 0, args


def test_page_bounds_reject_before_launch(lib):
    def call(dt=1, B=2, Hkv=4, D=128, page=16, cache=None, start=None, bounds=FAR):
        return lib.sv_page_bounds(dt, B, Hkv, D, page, cache or _cache(), start, bounds, None)
    for code, kw in ((NO, dict(dt=2)), (BAD, dict(B=-1)), (BAD, dict(Hkv=0)), (NO, dict(D=96)), (BAD, dict(page=0)), (NO, dict(B=65536)),
                     (BAD, dict(page=32, cache=_cache(**PAGED))), (BAD, dict(cache=_cache(k=None))), (BAD, dict(cache=_cache(prefix_len=None))),
                     (BAD, dict(bounds=None)), (BAD, dict(bounds=ctypes.c_void_p((1 << 40) + 8))), (BAD, dict(bounds=P)),
                     (BAD, dict(cache=_cache(v=(1 << 40) + 64))), (NO, dict(cache=_cache(Lmax=2 ** 31 - 1))), (NO, dict(Hkv=2 ** 23)),
                     (BAD, dict(cache=_cache(k=(1 << 20) + 8)))):
        assert call(**kw) == code, kw
    assert call(B=0, bounds=None, cache=_cache(k=None, v=None, prefix_len=None)) == sv.SV_OK


def test_page_scores_reject_before_launch(lib):
    def call(dt=1, B=2, N=1, Hq=8, Hkv=4, D=128, q=P, bounds=FAR2, length=FAR3, page=16, pages=8, table=None, blocks=0, sets=1, out=FAR):
        return lib.sv_page_scores(dt, B, N, Hq, Hkv, D, q, bounds, length, page, pages, table, blocks, sets, out, None)
    for code, kw in ((NO, dict(dt=2)), (BAD, dict(B=-1)), (BAD, dict(Hq=6)), (BAD, dict(Hkv=0)), (NO, dict(D=80)), (NO, dict(Hq=129, Hkv=1)),
                     (BAD, dict(N=0)), (NO, dict(N=65)), (BAD, dict(page=0)), (BAD, dict(pages=0)), (BAD, dict(sets=2)),
                     (BAD, dict(table=P, blocks=0)), (NO, dict(B=2 ** 26, N=8)), (NO, dict(pages=2 ** 31 - 1, B=64)), (NO, dict(pages=2 ** 20, B=2 ** 13, Hq=1, Hkv=1)), (BAD, dict(q=None)),
                     (BAD, dict(bounds=None)), (BAD, dict(length=None)), (BAD, dict(out=None)), (BAD, dict(q=ctypes.c_void_p(20))),
                     (BAD, dict(out=ctypes.c_void_p((1 << 40) + 4))), (BAD, dict(out=P)), (BAD, dict(out=FAR2)), (BAD, dict(out=FAR3)),
                     (BAD, dict(bounds=ctypes.c_void_p((1 << 40) + 128))), (BAD, dict(table=FAR, blocks=4))):
        assert call(**kw) == code, kw
    assert call(B=0, q=None, bounds=None, length=None, out=None) == sv.SV_OK


def test_select_pages_reject_before_launch(lib):
    def call(B=2, lists=4, pages=64, scores=FAR, length=P, page=16, K=8, first=1, last=1, out=FAR2):
        return lib.sv_select_pages(B, lists, pages, scores, length, page, K, first, last, out, None)
    for code, kw in ((BAD, dict(B=-1)), (BAD, dict(lists=0)), (BAD, dict(pages=0)), (BAD, dict(page=0)), (NO, dict(pages=32769)), (BAD, dict(K=0)),
                     (BAD, dict(first=-1)), (BAD, dict(last=-1)), (BAD, dict(first=5, last=4)), (BAD, dict(first=2 ** 31 - 1, last=2 ** 31 - 1)),
                     (NO, dict(B=2 ** 16, lists=2 ** 16)), (BAD, dict(scores=None)), (BAD, dict(length=None)), (BAD, dict(out=None)),
                     (BAD, dict(out=ctypes.c_void_p((1 << 40) + 64))), (BAD, dict(out=P))):
        assert call(**kw) == code, kw
    assert call(B=0, scores=None, length=None, out=None) == sv.SV_OK


def test_python_calls_refuse_what_is_no_cuda_tensor(lib):
    t = torch.zeros(2, 1, 4, 64)
    i = torch.zeros(2, dtype=torch.int32)
    cache = sv.KVCache(t, t, i)
    for call in (lambda: sv.sv_shared_attention(t, t, t, cache, [-1], 1.0, i, i[:1]),
                 lambda: sv.sv_shared_attention(None, t, t, cache, [-1], 1.0, i, i[:1]),
                 lambda: sv.sv_sparse_attention(t, t, t, cache, [-1], 1.0, i.view(2, 1, 1, 1)),
                 lambda: sv.sv_sparse_attention(t, t, t, cache, [-1], 1.0, [[[[0]]]]),
                 lambda: sv.sv_page_bounds(cache),
                 lambda: sv.sv_page_scores(t, t, i, 16),
                 lambda: sv.sv_page_scores(t, None, i, 16),
                 lambda: sv.sv_select_pages(t, i, 16, 4),
                 lambda: sv.sv_select_pages(None, i, 16, 4)):
        with pytest.raises(TypeError):
            call()
