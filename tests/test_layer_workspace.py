"""Refusals of the workspace of the norm's backward, on the CPU: the pointers
are never read."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 40
WORKSPACE, ALIAS = -7, -5
NAMES = ("dout", "r", "weight", "rstd", "dresidual", "dx", "dr", "dweight", "ws")


def call(size=1 << 30, has=1, rows=4, dim=256, **o):
    from selective_state_space_52_amd import _lib
    from selective_state_space_52_amd._lib import NormDims
    p = {n: BASE + i * (1 << 36) for i, n in enumerate(NAMES)}
    p.update(o)
    return _lib.lib().mssm_rms_norm_bwd(*[p[n] for n in NAMES], size, NormDims(rows, dim, 0, 1, 0, 0.0, 0), has,
                                        None)


def needed(rows=4, dim=256):
    import ctypes
    from selective_state_space_52_amd import _lib
    from selective_state_space_52_amd._lib import NormDims
    n = ctypes.c_int64(0)
    assert _lib.lib().mssm_rms_norm_bwd_workspace(NormDims(rows, dim, 0, 1, 0, 0.0, 0), n) == 0
    return n.value


@pytest.mark.parametrize("rows,dim", [(1, 1), (4, 256), (5000, 2560), (70, 32768)])
def test_refused(rows, dim):
    need, ws = needed(rows, dim), BASE + 8 * (1 << 36)
    assert need >= 4 * dim
    assert call(rows=rows, dim=dim, ws=None) == WORKSPACE
    assert call(rows=rows, dim=dim, ws=ws + 128) == WORKSPACE
    for size in (need - 1, 0, -1):
        assert call(rows=rows, dim=dim, size=size) == WORKSPACE
    for n in NAMES[:-1]:        # an input's or output's last bytes in the workspace, or its first
        assert call(rows=rows, dim=dim, **{n: ws}) == ALIAS
        assert call(rows=rows, dim=dim, **{n: ws + (need - 4) // 4 * 4}) == ALIAS


def test_no_hip_call_before_it():
    """A workspace that is missing or misaligned is refused before the first HIP
    call; the runtime's own log of its calls shows them."""
    run = ("import tests.test_layer_workspace as t; "
           "assert t.call(ws=None) == t.call(ws=t.BASE + 64) == t.call(size=0) == t.WORKSPACE; "
           "print('refused')")
    out = subprocess.run([sys.executable, "-c", run], cwd=ROOT, capture_output=True, text=True,
                         env={**os.environ, "AMD_LOG_LEVEL": "4"}, timeout=300)
    assert "refused" in out.stdout, out.stderr[-2000:]
    assert "hipGetDevice" not in out.stderr and "hipDeviceGetAttribute" not in out.stderr
