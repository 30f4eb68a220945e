"""Host-side checks of the layer-normed block's entry points and of the 8-bit
ones: bad calls return an error before any CUDA call, so this runs without a
GPU."""
import ctypes

import pytest

import combine_ep_get_04_gb300 as ep
from combine_ep_get_04_gb300 import _lib
from combine_ep_get_04_gb300 import build as epbuild

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: rejected on the host
OTHER = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10002)
INVALID, UNSUPPORTED = _lib.EP_ERR_INVALID_ARG, _lib.EP_ERR_UNSUPPORTED
NONE = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def lib():
    epbuild.build()
    return ep.load()


def test_dropout_arguments(lib):
    def call(T=4, H=10, type=0, x=FAKE, ld_x=10, res=None, ld_res=0, p=0.1, rng=FAKE, y=OTHER, ld_y=10):
        return lib.ep_dropout(T, H, type, x, ld_x, res, ld_res, p, rng, 0, y, ld_y, None)

    for bad in (dict(T=-1), dict(H=0), dict(type=2), dict(x=None), dict(y=None), dict(ld_x=9), dict(ld_y=9), dict(res=FAKE, ld_res=9),
                dict(p=-0.1), dict(p=1.5), dict(p=float("nan")), dict(rng=ctypes.c_void_p(0x10004)), dict(type=1, x=ODD),
                dict(x=ctypes.c_void_p(0x10001)), dict(type=1, y=ODD), dict(type=1, res=ODD, ld_res=10), dict(y=FAKE, ld_y=12),
                dict(res=OTHER, ld_res=12)):
        assert call(**bad) == INVALID, bad
        assert lib.ep_last_error()
    assert call(T=2 ** 31) == UNSUPPORTED and call(H=2 ** 31, ld_x=2 ** 31, ld_y=2 ** 31) == UNSUPPORTED
    assert call(T=2 ** 30, H=2 ** 30, ld_x=2 ** 30, ld_y=2 ** 30) == UNSUPPORTED
    assert call(T=0, x=None, y=None) == 0


@pytest.mark.parametrize("bad,status", [(dict(T=-1), 1), (dict(H=0), 1), (dict(H=12), 1), (dict(H=16392), 2), (dict(stream_type=2), 1),
                                        (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(p=-1.0), 1),
                                        (dict(p=1.01), 1), (dict(p=float("nan")), 1)])
def test_layer_norm_descriptions(lib, bad, status):
    f = dict(T=4, H=64, stream_type=0, eps=1e-5, p=0.0, site=0)
    f.update(bad)
    s = _lib.LayerNormDesc(**f)
    assert lib.ep_layer_norm_workspace_bytes(ctypes.byref(s)) == NONE
    assert lib.ep_layer_norm(ctypes.byref(s), FAKE, 64, FAKE, 64, FAKE, FAKE, None, OTHER, FAKE, None, None, None) == status
    assert lib.ep_layer_norm_backward(ctypes.byref(s), FAKE, 64, FAKE, None, FAKE, FAKE, FAKE, OTHER, FAKE, FAKE, FAKE, FAKE, 1 << 30,
                                      None, None) == status
    assert lib.ep_last_error()


def test_layer_norm_arguments(lib):
    s = _lib.LayerNormDesc(4, 64, 0, 1e-5, 0.1, 0)

    def fwd(h=FAKE, ld_h=64, y=FAKE, ld_y=64, w=FAKE, b=FAKE, rng=FAKE, h_out=OTHER, n=FAKE):
        return lib.ep_layer_norm(ctypes.byref(s), h, ld_h, y, ld_y, w, b, rng, h_out, n, None, None, None)

    for bad in (dict(h=None), dict(h=ODD), dict(y=ODD), dict(w=ODD), dict(b=ODD), dict(h_out=ODD), dict(n=ODD), dict(n=None),
                dict(y=None), dict(h_out=None), dict(ld_h=56), dict(ld_h=68), dict(ld_y=56), dict(ld_y=70), dict(rng=ODD),
                dict(h_out=FAKE, ld_h=72)):
        assert fwd(**bad) == INVALID, bad
    need = lib.ep_layer_norm_workspace_bytes(ctypes.byref(s))
    assert need >= 2 * 64 * 4

    def bwd(h=FAKE, ld_h=64, w=FAKE, rng=FAKE, stats=FAKE, dh=FAKE, dn=FAKE, d_h=OTHER, d_y=FAKE, ws=FAKE, nb=need):
        return lib.ep_layer_norm_backward(ctypes.byref(s), h, ld_h, w, rng, stats, dh, dn, d_h, d_y, FAKE, FAKE, ws, nb, None, None)

    for bad in (dict(h=None), dict(h=ODD), dict(ld_h=63), dict(w=ODD), dict(rng=ODD), dict(stats=None), dict(dh=ODD), dict(dn=None),
                dict(dn=ODD), dict(d_h=None), dict(d_h=ODD), dict(d_y=ODD), dict(ws=None), dict(ws=ODD), dict(nb=need - 1),
                dict(d_h=FAKE, ld_h=72)):
        assert bwd(**bad) == INVALID, bad
    none = _lib.LayerNormDesc(0, 64, 0, 1e-5, 0.0, 0)
    assert lib.ep_layer_norm(ctypes.byref(none), None, 0, None, 0, *([None] * 8)) == 0


def test_quant_arguments(lib):
    def call(E=4, K=64, mode=0, cap=0, R=8, counts=FAKE, offsets=FAKE, x=FAKE, ld=64, q=FAKE, scales=FAKE):
        return lib.ep_quant_i8(E, K, mode, cap, R, counts, offsets, x, ld, q, scales, None, None)

    for bad in (dict(E=0), dict(K=0), dict(K=24), dict(mode=2), dict(mode=1, cap=0), dict(mode=1, cap=3), dict(R=-1),
                dict(mode=1, cap=2, counts=None), dict(x=None), dict(x=ODD), dict(ld=56), dict(ld=68), dict(q=None), dict(q=ODD),
                dict(scales=None), dict(scales=ODD)):
        assert call(**bad) == INVALID, bad
    assert call(E=1025) == UNSUPPORTED and call(K=16400, ld=16400) == UNSUPPORTED and call(R=2 ** 31) == UNSUPPORTED
    assert call(R=0, x=None, q=None, scales=None) == 0


@pytest.mark.parametrize("bad,status", [(dict(E=0), 1), (dict(E=1025), 2), (dict(N=0), 1), (dict(N=12), 1), (dict(K=0), 1),
                                        (dict(K=24), 1), (dict(paired=2), 1), (dict(E=1024, N=1 << 20, K=1 << 20), 2), (dict(N=1 << 25), 2)])
def test_i8_descriptions(lib, bad, status):
    f = dict(E=4, N=16, K=128, paired=0)
    f.update(bad)
    s = _lib.I8(**f)
    assert lib.ep_i8_bytes(ctypes.byref(s)) == NONE
    assert lib.ep_i8_pack(ctypes.byref(s), FAKE, FAKE, FAKE, None) == status
    assert lib.ep_expert_i8(ctypes.byref(s), FAKE, 0, 0, 4, 4, FAKE, FAKE, FAKE, FAKE, FAKE, None, None) == status


def test_i8_arguments(lib):
    s = _lib.I8(4, 16, 128, 0)
    # one block of 128 rows and one of 128 channels an expert, then the rows' scales
    assert lib.ep_i8_bytes(ctypes.byref(s)) == 4 * (128 * 128 + 128 * 4)
    for args in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (ODD, FAKE, FAKE), (FAKE, ODD, FAKE), (FAKE, FAKE, ODD)):
        assert lib.ep_i8_pack(ctypes.byref(s), *args, None) == INVALID

    def call(packed=FAKE, mode=0, cap=0, R=8, rows=8, counts=FAKE, offsets=FAKE, x=FAKE, xs=FAKE, y=FAKE):
        return lib.ep_expert_i8(ctypes.byref(s), packed, mode, cap, R, rows, counts, offsets, x, xs, y, None, None)

    for bad in (dict(packed=None), dict(packed=ODD), dict(mode=2), dict(mode=1, cap=0), dict(mode=1, cap=3), dict(R=-1), dict(rows=-1),
                dict(offsets=None), dict(mode=1, cap=2, counts=None), dict(x=None), dict(x=ODD), dict(xs=None), dict(xs=ODD),
                dict(y=None), dict(y=ODD)):
        assert call(**bad) == INVALID, bad
    assert call(R=0) == 0 and call(rows=0) == 0
    assert call(R=2 ** 31) == UNSUPPORTED
