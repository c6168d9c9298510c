"""The windowed, grouped-head, 4-bit and norm entry points refuse bad arguments on the host,
before anything reaches a GPU, and size their workspaces.  No GPU needed."""
import ctypes

import pytest

import blockwise_attention_gb300 as ba
from blockwise_attention_gb300 import _lib
from blockwise_attention_gb300._lib import BA_ERR_ARG, BA_ERR_SHAPE, BA_ERR_UNSUPPORTED, BA_OK, ba_kv4, ba_tensor

NONE = ba_tensor(None, 0, 0, 0)
X = ba_tensor(1 << 20, 1 << 20, 1 << 14, 64)
P = ctypes.c_void_p(1 << 20)
BF, F32 = _lib.BA_BF16, _lib.BA_F32


def window_fwd(lib, q=X, k=X, B=1, Hq=4, Hkv=2, Lq=8, Lk=8, d=64, dt=BF, q_off=0, window=4, sinks=1, kpm=None, ld=0, out=P,
               odt=BF, lse=P):
    return lib.attn_window_fwd(q, k, k, B, Hq, Hkv, Lq, Lk, d, dt, q_off, window, sinks, kpm, ld, 0.0, out, odt, lse, None,
                               0, None)


@pytest.mark.parametrize("bad,code", [
    (dict(window=0), BA_ERR_ARG), (dict(sinks=-1), BA_ERR_ARG), (dict(q_off=-1), BA_ERR_ARG), (dict(B=-1), BA_ERR_ARG),
    (dict(Hq=3), BA_ERR_SHAPE), (dict(Hkv=0), BA_ERR_SHAPE), (dict(d=48), BA_ERR_SHAPE), (dict(dt=7), BA_ERR_ARG),
    (dict(q=NONE), BA_ERR_ARG), (dict(k=NONE), BA_ERR_ARG), (dict(out=None), BA_ERR_ARG), (dict(lse=None), BA_ERR_ARG),
    (dict(out=ctypes.c_void_p((1 << 20) + 8)), BA_ERR_ARG), (dict(dt=F32, odt=BF), BA_ERR_ARG),
    (dict(kpm=P, ld=7), BA_ERR_ARG), (dict(q_off=2 ** 31 - 1), BA_ERR_SHAPE), (dict(Lq=0), BA_OK), (dict(B=0), BA_OK)])
def test_window_forward(bad, code):
    assert window_fwd(ba.load(), **bad) == code


def test_window_backward():
    lib = ba.load()

    def run(Hq=4, Hkv=2, Lq=8, Lk=8, d=64, window=4, dq=P, gdt=BF, q=X, B=1):
        return lib.attn_window_bwd(q, X, X, X, X, P, B, Hq, Hkv, Lq, Lk, d, BF, 0, window, 1, None, 0, 0.0, dq, P, P, gdt,
                                   None, 0, None)
    assert run(window=0) == BA_ERR_ARG and run(Hq=5) == BA_ERR_SHAPE and run(d=80) == BA_ERR_SHAPE
    assert run(dq=None) == BA_ERR_ARG and run(gdt=5) == BA_ERR_ARG and run(q=NONE) == BA_ERR_ARG
    assert run(B=20000) == BA_ERR_SHAPE and run(B=0) == BA_OK


def test_window_backward_workspace():
    """D per row; partials only where a chunk of the queries is smaller than all of them, and then few."""
    size = ba.load().attn_window_bwd_workspace_size
    base = 256 + 4 * 32 * 8192
    assert size(1, 32, 8, 8192, 8192, 128, 0, 1024, 0) == base          # no sinks
    assert size(1, 32, 8, 8192, 8192, 128, 0, 8192, 4) == base          # the window covers them
    assert size(1, 32, 8, 1024, 1024, 128, 0, 1000, 4) == 256 + 4 * 32 * 1024   # one chunk
    tile = 2 * 128 * 128 * 4
    assert size(1, 32, 8, 8192, 8192, 128, 0, 1024, 4) == base + 8 * 8 * tile     # chunks of 1152 rows
    assert size(1, 1, 1, 1 << 20, 1 << 20, 128, 0, 16, 4) <= 256 + (4 << 20) + 32 * tile
    assert size(1, 1, 1, 1 << 20, 1 << 20, 128, 0, 16, 4000) <= 256 + (4 << 20) + 64 * tile
    assert size(-1, 1, 1, 8, 8, 128, 0, 16, 4) == 0 and size(1, 1, 1, 8, 8, 128, 0, 0, 4) == 0


def test_window_decode():
    lib = ba.load()

    def run(B=1, Hq=4, Hkv=2, S=8, d=64, dt=BF, window=4, sinks=1, q=X, k=X, out=P, odt=BF, scale=0.0):
        return lib.attn_window_decode_fwd(q, k, k, B, Hq, Hkv, S, d, dt, None, window, sinks, scale, out, odt, P, None, 0, None)
    assert run(window=0) == BA_ERR_ARG and run(sinks=-2) == BA_ERR_ARG and run(Hq=7) == BA_ERR_SHAPE
    assert run(d=40) == BA_ERR_SHAPE and run(q=NONE) == BA_ERR_ARG and run(k=NONE) == BA_ERR_ARG and run(out=None) == BA_ERR_ARG
    assert run(k=ba_tensor((1 << 20) + 2, 1 << 20, 1 << 14, 64)) == BA_ERR_ARG
    assert run(k=ba_tensor(1 << 20, 1 << 20, 1 << 14, 65)) == BA_ERR_ARG
    assert run(dt=F32, odt=BF) == BA_ERR_ARG and run(scale=float("nan")) == BA_ERR_ARG
    assert run(B=4000000) == BA_ERR_SHAPE and run(B=0) == BA_OK


def cache(**kw):
    f = dict(k_codes=1 << 20, k_scales=1 << 20, v_codes=1 << 20, v_scales=1 << 20, codes_sB=1 << 14, codes_sH=1 << 12,
             codes_sT=32, scales_sB=1 << 11, scales_sH=1 << 9, scales_sT=4, k_exp=0, v_exp=0)
    f.update(kw)
    return ba_kv4(*(f[n] for n, _ in ba_kv4._fields_))


@pytest.mark.parametrize("bad", [dict(k_codes=None), dict(v_scales=None), dict(k_codes=(1 << 20) + 8), dict(v_scales=(1 << 20) + 2),
                                 dict(codes_sT=36), dict(scales_sH=6), dict(codes_sB=24), dict(k_exp=101), dict(v_exp=-101)])
def test_kv4_cache_layout(bad):
    lib = ba.load()
    c = cache(**bad)
    assert lib.kv4_append(X, X, c, 2, 2, 1, 8, 64, BF, None, None, None) == BA_ERR_ARG
    assert lib.kv4_read(c, 2, 2, 8, 64, 0, 8, BF, P, P, None) == BA_ERR_ARG
    assert lib.attn_decode_kv4_fwd(X, c, 2, 4, 2, 8, 64, BF, None, 0, 0, 0.0, P, BF, P, None, 0, None) == BA_ERR_ARG


def test_kv4_arguments():
    lib = ba.load()
    c = cache()
    assert lib.kv4_append(X, X, c, 1, 1, 1, 8, 32, BF, None, None, None) == BA_ERR_SHAPE
    assert lib.kv4_append(NONE, X, c, 1, 1, 1, 8, 64, BF, None, None, None) == BA_ERR_ARG
    assert lib.kv4_append(ba_tensor((1 << 20) + 4, 0, 0, 64), X, c, 1, 1, 1, 8, 64, BF, None, None, None) == BA_ERR_ARG
    assert lib.kv4_append(X, X, c, 1, 1, 0, 8, 64, BF, None, None, None) == BA_OK
    assert lib.kv4_read(c, 1, 1, 8, 64, 4, 5, BF, P, P, None) == BA_ERR_ARG
    assert lib.kv4_read(c, 1, 1, 8, 64, -1, 5, BF, P, P, None) == BA_ERR_ARG
    assert lib.kv4_read(c, 1, 1, 8, 64, 0, 8, BF, ctypes.c_void_p((1 << 20) + 8), P, None) == BA_ERR_ARG

    def run(Hq=4, Hkv=2, d=64, dt=BF, window=0, odt=BF):
        return lib.attn_decode_kv4_fwd(X, c, 1, Hq, Hkv, 8, d, dt, None, window, 0, 0.0, P, odt, P, None, 0, None)
    assert run(dt=F32, odt=F32) == BA_ERR_UNSUPPORTED and run(d=32) == BA_ERR_SHAPE and run(Hq=3) == BA_ERR_SHAPE
    assert run(window=-1) == BA_ERR_ARG and run(odt=3) == BA_ERR_ARG


def test_decode_workspaces_go_by_the_gpu_not_the_cache():
    """One partial result for each CTA (a few waves of them) and one more for each key head."""
    lib = ba.load()
    for size in (lib.attn_window_decode_workspace_size, lib.attn_decode_kv4_workspace_size):
        n = size(1, 32, 8, 65536, 128, 1024, 4)
        assert 0 < n <= (8 * 152 * 6 + 8) * 4 * (128 * 4 + 8) + 512 and n == size(1, 32, 8, 1 << 30, 128, 1024, 4)
        assert size(1, 32, 8, 1 << 30, 128, 1 << 29, 4) <= (8 * 152 * 6 + 8) * 4 * (128 * 4 + 8) + 512
        assert size(1, 5, 2, 64, 128, 64, 0) == 0 and size(0, 8, 2, 64, 128, 64, 0) == 0
    assert lib.attn_window_decode_workspace_size(1, 8, 2, 4096, 128, 0, 0) == 0


def test_qk_norm():
    lib = ba.load()

    def run(q=X, k=X, w=P, wdt=BF, B=1, Hq=2, Hkv=2, T=4, d=64, dt=BF, eps=1e-6, ld=0, base=1e4, ps=1.0, y=P):
        return lib.qk_norm_rope_fwd(q, k, w, w, wdt, B, Hq, Hkv, T, d, dt, eps, None, ld, base, ps, y, y, None)
    nan = float("nan")
    for bad in (dict(q=NONE), dict(k=NONE), dict(w=None), dict(y=None), dict(y=ctypes.c_void_p((1 << 20) + 8)), dict(wdt=4),
                dict(dt=F32, wdt=BF), dict(eps=-1.0), dict(eps=nan), dict(base=0.0), dict(base=nan), dict(base=float("inf")), dict(ps=-1.0), dict(ps=float("inf")), dict(T=-1),
                dict(ld=-1)):
        assert run(**bad) == BA_ERR_ARG, bad
    assert run(d=96) == BA_ERR_SHAPE and run(T=0) == BA_OK and run(Hq=0, Hkv=0) == BA_OK

    def bwd(dwq=P, gdt=BF):
        return lib.qk_norm_rope_bwd(X, X, P, P, BF, X, X, gdt, 1, 2, 2, 4, 64, BF, 1e-6, None, 0, 1e4, 1.0, P, P, dwq, P, None,
                                    0, None)
    assert bwd(dwq=None) == BA_ERR_ARG and bwd(gdt=9) == BA_ERR_ARG
    assert 0 < lib.qk_norm_rope_bwd_workspace_size(2, 16, 4, 8192, 128, BF) <= 1 << 21


@pytest.mark.parametrize("stride", ["codes_sB", "codes_sH", "codes_sT", "scales_sB", "scales_sH", "scales_sT"])
def test_kv4_append_wants_rows_in_places_of_their_own(stride):
    lib = ba.load()
    c = cache(**{stride: 0})
    assert lib.kv4_append(X, X, c, 2, 2, 1, 8, 64, BF, None, None, None) == BA_ERR_ARG
