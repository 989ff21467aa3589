"""Errors of the dense-tower operators' launches."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

REFUSED = """
import torch
from recsys_sparse_embedding_gb300 import binding as B
x = torch.ones(40, 64, device="cuda")
y = torch.empty_like(x)
layer = B.DenseLayer(torch.ones(48, 64, device="cuda"))
big = torch.ones(16384, 64, device="cuda")
z = torch.empty(16384, 48, device="cuda")
ws = B.DenseWorkspace(layer, 16384)
calls = {"norm": lambda: B.ctr_rms_norm_fwd(x, y), "layer": lambda: B.ctr_dense_fwd(layer, big, z, ws),
         "few rows": lambda: B.ctr_dense_fwd(layer, x, z[:40], ws)}
for c in calls.values():
    c()
torch.cuda.synchronize()
for name, c in calls.items():
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.capture_begin()
        try:
            s.synchronize()  # not allowed while capturing: the capture is void
        except RuntimeError:
            pass
        try:
            c()
            print(name, "was not refused")
        except B.DsfError as e:
            assert e.code == B.DSF_ECUDA
        try:
            g.capture_end()
        except RuntimeError:
            pass
    B.HashTable(64, 16, B.DSF_F32, [0])  # raises if its launch seems to fail
torch.cuda.synchronize()
print("done")
"""


def test_a_refused_launch_does_not_fail_the_next_call():
    """A launch into a capture that is already void is refused by the runtime:
    the call says so, and calls after it are answered for themselves."""
    r = subprocess.run([sys.executable, "-c", REFUSED], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.stdout.split() == ["done"], r.stdout + r.stderr[-2000:]
