"""A call that fails on the host leaves no error behind for the next one."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# in a process of its own: a capture that the runtime has ended takes torch's pool with it
PROGRAM = """
import torch
import vocabulary_cross_entropy_pass_gb300 as pkg
w = torch.randn(50, 64, device="cuda")
t = torch.arange(20, device="cuda")
x, g, out = torch.randn(20, 64, device="cuda"), torch.ones(64, device="cuda"), torch.empty(20, 64, device="cuda")
ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
calls = [lambda: pkg.ce_embed_fwd(t, w, out=out), lambda: pkg.ce_rmsnorm_fwd(x, g, out=out),
         lambda: pkg.ce_embed_bwd(x, t, 50), lambda: pkg.ce_rmsnorm_bwd(x, x, g),
         lambda: pkg.ce_logits_process(x, out=out), lambda: pkg.ce_fwd_only(x, t)]
for call in calls:
    call()
torch.cuda.synchronize()
for call in calls:
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin()
        status, _ = pkg.ce_get_error(ws)  # waits, which a capture does not allow
        try:
            graph.capture_end()
            print("captured")
        except RuntimeError:
            pass
    assert status == pkg.CEError(5).status == 5, status
    call()
torch.cuda.synchronize()
print("done")
"""


def test_a_refused_wait_is_not_the_next_launch_s_failure():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), r.stdout + r.stderr[-2000:]
