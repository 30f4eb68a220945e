"""The wait of the 8-bit products' warps runs out by itself: flagged, within the
bound that it states, with the context usable afterwards."""
import os
import subprocess

import pytest

import combine_ep_get_04_gb300 as ep

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_phase_that_never_completes_is_given_up(tmp_path):
    from combine_ep_get_04_gb300 import build as B
    exe = tmp_path / "suspended_wait_timeout"
    subprocess.run([B.nvcc(), *B.ARCH, *B.NVCC_FLAGS, os.path.join(HERE, "suspended_wait_timeout.cu"), "-o", str(exe)], check=True,
                   capture_output=True, text=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=120).stdout
    print(out)
    f = dict(kv.split("=", 1) for kv in out.split())
    assert int(f["timeout_flag"]) == int(f["timeout_bit"]) == ep.ERRF_TIMEOUT, out
    # the limit, and 128 tries of a millisecond each (and as much again: the clock's step and the warp's way to its turn)
    assert 1000.0 <= float(f["least_ms"]) <= float(f["most_ms"]) <= 1256.0, out
    assert f["err1"] == f["err2"] == f["err3"] == "cudaSuccess", out
    assert int(f["completed_flag"]) == 0 and f["completed_ok"] == "1", out
    assert f["plain_ok"] == "1", out
