"""The library's first call on a device may be one that is being captured."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROG = r"""
import sys
import torch
from atomistic_mlip_b200 import e2f

which = sys.argv[1]
g = torch.Generator(device="cuda")
g.manual_seed(1)
ids = torch.randint(0, 50, (3000,), generator=g, device="cuda")
x = torch.randn(3000, 64, generator=g, device="cuda")
W, dy = torch.randn(96, 64, generator=g, device="cuda"), torch.randn(3000, 96, generator=g, device="cuda")


def call():
    if which == "embed":
        return (e2f.embed_forward(ids, x[:50]), e2f.embed_backward(ids, x, 50))
    return (e2f.linear_forward(x, W, act="silu"), *e2f.linear_backward(x, W, dy, act="silu", need_bias=True))


graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
assert e2f.stream_status() == 0
want = call()
assert all(torch.equal(p, q) for p, q in zip(got, want))
x.mul_(0.5)
graph.replay()
assert all(torch.equal(p, q) for p, q in zip(got, call()))
print("ok")
"""


@pytest.mark.parametrize("which", ["embed", "linear"])
def test_first_call_in_a_capture(cuda_ok, which):
    r = subprocess.run([sys.executable, "-c", PROG, which], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split()[-1:] == ["ok"], r.stderr[-2000:]
