"""FlashAttention.apply is flash_attention's node: what that refuses in a capture it refuses too."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


CAPTURE = """
import torch
from attention_fa_fwd_03_gb300.autograd import FlashAttention
q, k, v = (torch.randn(1, 2, 100, 64, device="cuda").half().requires_grad_() for _ in range(3))
do = torch.randn(1, 2, 100, 64, device="cuda").half()
def attend():
    return FlashAttention.apply(q, k, v, 0.125, True, 0)[0]
eager = attend()
side = torch.cuda.Stream()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
try:
    with torch.cuda.graph(g, stream=side):
        attend().backward(do)
    print("captured")
except RuntimeError as e:
    print("refused" if "eager graph" in str(e) else e)
want = torch.autograd.grad(eager, (q, k, v), do)
del eager
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=side):
    attend().backward(do)
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a.grad, b) for a, b in zip((q, k, v), want))
print("done")
"""


def test_function_captured_beside_an_eager_graph():
    """As flash_attention: refused while an eager graph of the same leaves from the default stream lives, with the process as
    it was, and captured afterwards."""
    r = subprocess.run([sys.executable, "-c", CAPTURE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["refused", "done"], (r.returncode, r.stdout, r.stderr[-2000:])
