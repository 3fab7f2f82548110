"""Calls whose checks find no host memory return an error (no GPU: a process of
its own with a limit on its memory; nothing is launched: with enough memory the
calls are refused as well, since two segments write the same buffer)."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import ctypes as ct, resource
from l2_row_b200 import ds

N, A, eps = ds.DS_MAX_SEGMENTS, 1 << 32, ct.c_float(1e-6)
near = lambda i: A + (i << 20)                 # buffers that do not meet, but for the last segment's
far = lambda i, j: A + ((j + 1) << 40) + (i %% (N - 1) << 20)
name = %r
if "embed" in name:
    segs = (ds.ds_eseg * N)(*(ds.ds_eseg(w=near(i), ids=far(i, 0), y=far(i, 1), dy=far(i, 2), grad_w=far(i, 3), tokens=2, vocab=2,
                                         cols=16, ld=16, ld_y=16, ld_g=16, radius=1.0) for i in range(N)))
    args = (ds.DS_F32, ds.DS_F32, eps) + ((A << 12, 1 << 30) if "backward" in name else ()) + (None,)
elif name == "ds_qk_norm_rows":
    segs = (ds.ds_qnseg * N)(*(ds.ds_qnseg(q=near(i), q_out=far(i, 0), rows=2, ld_q=16, ld_qo=16, head_dim=16, hq=1)
                               for i in range(N)))
    args = (ds.DS_F32, eps, None)
elif name == "ds_qk_norm_rows_backward":
    segs = (ds.ds_qngseg * N)(*(ds.ds_qngseg(q=near(i), dq_out=far(i, 0), dq=far(i, 1), rows=2, ld_q=16, ld_dqo=16, ld_dq=16,
                                             head_dim=16, hq=1) for i in range(N)))
    args = (ds.DS_F32, ds.DS_F32, eps, None, None, None, 0, None)
else:
    segs = (ds.ds_lseg * N)(*(ds.ds_lseg(x=near(i), lse=far(i, 0), dx=far(i, 1), rows=2, cols=16, ld=16, ld_d=16, scale=1.0)
                              for i in range(N)))
    args = (ds.DS_F32,) + ((ds.DS_F32,) if "backward" in name else ()) + (None,)
call = getattr(ds.lib(), name)
with open("/proc/self/statm") as f:
    used = int(f.read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (1 << 20), resource.RLIM_INFINITY))
status = call(segs, N, *args)
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
assert status == ds.DS_ERR_TOO_MANY_SEGMENTS, status
assert b"host memory" in ds.lib().ds_last_error()
assert call(segs, N, *args) == ds.DS_ERR_OVERLAP
"""


@pytest.mark.skipif(not os.path.exists("/proc/self/statm"), reason="needs /proc")
@pytest.mark.parametrize("name", ["ds_embed_rows", "ds_embed_rows_backward", "ds_qk_norm_rows", "ds_qk_norm_rows_backward",
                                  "ds_logp_rows", "ds_logp_rows_backward"])
def test_no_exception_leaves_a_call(name):
    r = subprocess.run([sys.executable, "-c", PROGRAM % name], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
