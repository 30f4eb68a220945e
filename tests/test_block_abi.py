"""Host-side checks of the block operators' entry points: bad calls return an
error before any CUDA call, so this runs without a GPU."""
import ctypes
import os
import subprocess
import sys

import pytest

import combine_ep_get_04_gb300 as ep
from combine_ep_get_04_gb300 import _lib
from combine_ep_get_04_gb300 import build as epbuild

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: rejected on the host
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    epbuild.build()
    return ep.load()


@pytest.mark.parametrize("bad,status", [(dict(T=-1), 1), (dict(H=0), 1), (dict(H=12), 1), (dict(H=16392), 2),
                                        (dict(stream_type=2), 1), (dict(gate_kind=3), 1), (dict(eps=0.0), 1),
                                        (dict(eps=float("nan")), 1)])
def test_norm_descriptions(lib, bad, status):
    f = dict(T=4, H=64, stream_type=0, gate_kind=0, eps=1e-6)
    f.update(bad)
    s = _lib.Norm(**f)
    assert lib.ep_block_norm_workspace_bytes(ctypes.byref(s)) == ctypes.c_size_t(-1).value
    assert lib.ep_block_norm(ctypes.byref(s), FAKE, 64, FAKE, 64, FAKE, None, None, FAKE, FAKE, FAKE, None, None) == status
    assert lib.ep_last_error()


def test_norm_arguments(lib):
    s = _lib.Norm(4, 64, 0, 0, 1e-6)
    gated = _lib.Norm(4, 64, 0, 1, 1e-6)

    def fwd(shape=s, h=FAKE, ld_h=64, y=FAKE, ld_y=64, w_post=FAKE, gate=None, a=None, w_pre=FAKE, h_out=ctypes.c_void_p(0x20000),
            n=FAKE):
        return lib.ep_block_norm(ctypes.byref(shape), h, ld_h, y, ld_y, w_post, gate, a, w_pre, h_out, n, None, None)

    for bad in (dict(h=None), dict(h=ODD), dict(y=ODD), dict(w_post=ODD), dict(w_pre=ODD), dict(h_out=ODD), dict(n=ODD),
                dict(ld_h=63), dict(ld_h=56), dict(ld_h=68), dict(ld_y=56), dict(ld_y=70), dict(y=None), dict(n=None),
                dict(w_pre=None), dict(gate=FAKE), dict(shape=gated), dict(shape=gated, gate=ODD),
                dict(w_pre=None, n=None, h_out=None), dict(h_out=FAKE, ld_h=72)):
        assert fwd(**bad) == _lib.EP_ERR_INVALID_ARG, bad
    assert lib.ep_block_norm(ctypes.byref(_lib.Norm(0, 64, 0, 0, 1e-6)), *([None, 0] * 2), *([None] * 8)) == 0

    need = lib.ep_block_norm_workspace_bytes(ctypes.byref(s))
    assert need >= 3 * 64 * 4

    def bwd(shape=s, w_post=FAKE, gate=None, a=None, w_pre=FAKE, rstd=FAKE, dho=FAKE, dn=FAKE, dh=FAKE, dy=FAKE, dwq=FAKE,
            dg=None, da=None, dwp=FAKE, ws=FAKE, nb=need):
        return lib.ep_block_norm_backward(ctypes.byref(shape), FAKE, 64, FAKE, 64, w_post, gate, a, w_pre, rstd, dho, dn, dh, dy,
                                          dwq, dg, da, dwp, ws, nb, None, None)

    for bad in (dict(rstd=None), dict(dh=None), dict(dy=None), dict(dn=None), dict(dwq=None), dict(dwp=None), dict(dg=FAKE),
                dict(da=FAKE), dict(a=FAKE), dict(ws=None), dict(nb=need - 1), dict(ws=ODD), dict(dho=ODD), dict(dn=ODD),
                dict(dh=ODD), dict(dy=ODD), dict(shape=gated, gate=FAKE), dict(w_pre=None, dwp=None, dn=None, dho=None)):
        assert bwd(**bad) == _lib.EP_ERR_INVALID_ARG, bad


@pytest.mark.parametrize("bad,status", [(dict(T=-1), 1), (dict(E=0), 1), (dict(E=1025), 2), (dict(k=0), 1), (dict(k=17), 1),
                                        (dict(E=64, k=33), 2), (dict(groups=3), 1), (dict(E=64, groups=64), 2), (dict(groups=0), 1),
                                        (dict(topk_groups=0), 1), (dict(topk_groups=2), 1), (dict(full_softmax=2), 1),
                                        (dict(logits_type=2), 1), (dict(num_seqs=0), 1), (dict(num_seqs=65536), 2),
                                        (dict(T=2 ** 30, k=8), 2)])
def test_route_descriptions(lib, bad, status):
    f = dict(T=4, E=16, k=4, groups=1, topk_groups=1, full_softmax=0, logits_type=1, num_seqs=1, balance_coef=0.0, z_coef=0.0)
    f.update(bad)
    s = _lib.Route(**f)
    assert lib.ep_route_workspace_bytes(ctypes.byref(s)) == ctypes.c_size_t(-1).value
    assert lib.ep_route(ctypes.byref(s), FAKE, 16, *([FAKE] * 11), 1 << 30, None, None) == status
    assert lib.ep_last_error()


def test_route_arguments(lib):
    s = _lib.Route(4, 16, 4, 1, 1, 0, 1, 1, 0.0, 0.0)
    two = _lib.Route(4, 16, 4, 1, 1, 0, 1, 2, 0.0, 0.0)
    need = lib.ep_route_workspace_bytes(ctypes.byref(s))

    def fwd(shape=s, logits=FAKE, ld=16, seq=None, idx=FAKE, w=FAKE, lse=FAKE, counts=FAKE, probs=FAKE, tokens=FAKE, losses=FAKE,
            ws=FAKE, nb=need):
        return lib.ep_route(ctypes.byref(shape), logits, ld, None, None, seq, idx, w, lse, counts, probs, tokens, losses, ws, nb,
                            None, None)

    for bad in (dict(logits=None), dict(logits=ODD), dict(ld=15), dict(idx=None), dict(w=None), dict(lse=None), dict(counts=None),
                dict(probs=None), dict(tokens=None), dict(losses=None), dict(ws=None), dict(nb=need - 1), dict(ws=ODD),
                dict(shape=two)):
        assert fwd(**bad) == _lib.EP_ERR_INVALID_ARG, bad
    none = _lib.Route(0, 16, 4, 1, 1, 0, 1, 1, 0.0, 0.0)
    assert lib.ep_route(ctypes.byref(none), None, 0, *([None] * 11), 0, None, None) == 0

    def bwd(shape=s, logits=FAKE, ld=16, idx=FAKE, w=FAKE, lse=FAKE, counts=FAKE, tokens=FAKE, d=FAKE):
        return lib.ep_route_backward(ctypes.byref(shape), logits, ld, None, idx, w, lse, counts, tokens, None, None, d, None)

    for bad in (dict(logits=None), dict(logits=ODD), dict(ld=15), dict(idx=None), dict(w=None), dict(lse=None), dict(counts=None),
                dict(tokens=None), dict(d=None), dict(d=ODD), dict(shape=two)):
        assert bwd(**bad) == _lib.EP_ERR_INVALID_ARG, bad
    assert lib.ep_route_backward(ctypes.byref(none), None, 0, *([None] * 10)) == 0


@pytest.mark.parametrize("bad,status", [(dict(E=0), 1), (dict(E=1025), 2), (dict(N=0), 1), (dict(N=12), 1), (dict(K=0), 1),
                                        (dict(K=12), 1), (dict(group=16), 1), (dict(group=256), 1), (dict(paired=2), 1),
                                        (dict(E=1024, N=1 << 20, K=1 << 20), 2), (dict(N=1 << 25), 2)])
def test_w4_descriptions(lib, bad, status):
    f = dict(E=4, N=16, K=128, group=128, paired=0)
    f.update(bad)
    s = _lib.W4(**f)
    assert lib.ep_w4_bytes(ctypes.byref(s)) == ctypes.c_size_t(-1).value
    assert lib.ep_w4_pack(ctypes.byref(s), FAKE, FAKE, FAKE, None) == status
    assert lib.ep_expert_w4(ctypes.byref(s), FAKE, 0, 0, 4, 4, FAKE, FAKE, FAKE, None, 0, FAKE, None, None) == status


def test_w4_arguments(lib):
    s = _lib.W4(4, 16, 128, 64, 0)
    # one row block, one step of K: eight tiles of 1024 bytes of codes and two groups of 16 scales
    assert lib.ep_w4_bytes(ctypes.byref(s)) == 4 * 8 * (1024 + 64)
    for args in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (ODD, FAKE, FAKE), (FAKE, FAKE, ODD)):
        assert lib.ep_w4_pack(ctypes.byref(s), *args, None) == _lib.EP_ERR_INVALID_ARG

    def call(shape=s, packed=FAKE, mode=0, cap=0, R=8, rows=8, counts=FAKE, offsets=FAKE, x=FAKE, xs=None, payload=0, y=FAKE):
        return lib.ep_expert_w4(ctypes.byref(shape), packed, mode, cap, R, rows, counts, offsets, x, xs, payload, y, None, None)

    odd_k = _lib.W4(4, 16, 120, 64, 0)
    for bad in (dict(packed=None), dict(packed=ODD), dict(mode=2), dict(mode=1, cap=0), dict(mode=1, cap=3), dict(R=-1), dict(rows=-1),
                dict(offsets=None), dict(mode=1, cap=2, counts=None), dict(x=None), dict(x=ODD), dict(y=None), dict(y=ODD),
                dict(payload=3), dict(payload=1), dict(payload=1, xs=ODD), dict(shape=odd_k, payload=1, xs=FAKE)):
        assert call(**bad) == _lib.EP_ERR_INVALID_ARG, bad
    assert call(R=0) == 0 and call(rows=0) == 0
    assert call(R=2 ** 31) == _lib.EP_ERR_UNSUPPORTED
    assert call(shape=_lib.W4(1, 16, 1 << 20, 128, 0), payload=1, xs=FAKE) == _lib.EP_ERR_UNSUPPORTED   # a row's scales do not fit


def test_import_on_a_torch_without_cuda(lib):
    """A CPU build of torch has no CUDA bindings; what needs no GPU works there."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(ep.__file__)))
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_get')]:\n"
            "    delattr(torch._C, name)\n"
            "import combine_ep_get_04_gb300 as ep\n"
            "assert ep.recv_rows(ep.make_shape(4, 64, 8, 2)) == 8\n")
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


@pytest.mark.parametrize("eps", [1e-45, 1e-38, 9e-31, 2e30, -1e-6, float("inf")])
def test_norm_refuses_an_eps_whose_roots_overflow(lib, eps):
    s = _lib.Norm(4, 64, 0, 0, eps)
    assert lib.ep_block_norm_workspace_bytes(ctypes.byref(s)) == ctypes.c_size_t(-1).value
    assert lib.ep_block_norm(ctypes.byref(s), FAKE, 64, FAKE, 64, FAKE, None, None, FAKE, FAKE, FAKE, None, None) == _lib.EP_ERR_INVALID_ARG
    assert lib.ep_block_norm_workspace_bytes(ctypes.byref(_lib.Norm(4, 64, 0, 0, 1e-30))) > 0
