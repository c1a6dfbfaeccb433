"""A process whose first call of each operator is captured into a CUDA graph:
nothing in a call needs to have run eagerly before."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys
import torch
from combine_top_group_b200 import ep
which = sys.argv[1]
g = torch.Generator(device="cuda").manual_seed(0)
rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
if which == "norm":
    x, gamma, dy = rand(700, 1024).bfloat16(), rand(1024), rand(700, 1024).bfloat16()
    o = dict(h=torch.empty_like(x), y=torch.empty_like(x), rstd=torch.empty(700, device="cuda"))
    dx, dg = torch.empty_like(x), torch.empty(1024, device="cuda")
    ws = torch.empty(ep.ep_rmsnorm_backward_workspace_bytes(700, 1024), dtype=torch.uint8, device="cuda")
    def run():
        ep.ep_rmsnorm(x, gamma, 1e-6, residual=dy, **o)
        ep.ep_rmsnorm_backward(o["h"], o["rstd"], gamma, dy, dx, dg, ws)
    outs = [*o.values(), dx, dg]
elif which == "balance":
    z = rand(500, 96)
    idx = z.topk(4).indices.int()
    loss, counts, dz = torch.empty(1, device="cuda"), torch.empty(1, 96, dtype=torch.int32, device="cuda"), torch.empty_like(z)
    ws = torch.empty(ep.ep_balance_loss_workspace_bytes(500, 96), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    def run():
        ep.ep_balance_loss(z, idx, 1, 0.1, loss, counts, ws, err)
        ep.ep_balance_loss_backward(z, counts, 4, 1, 0.1, dz)
    outs = [loss, counts, dz]
else:
    rows = int(which)
    buf = ep.ep_buffer_create(ep.ep_default_config(1, 1, 128, 1, 1), device="cuda")
    x, w = rand(rows, 2048).bfloat16(), rand(1, 512, 2048).bfloat16()
    o = torch.empty(rows, 512, device="cuda")
    run = lambda: ep.ep_linear(buf, x, w, o)
    outs = [o]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
for t in outs:
    t.zero_()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs]
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs)) and all(t.any() for t in got)
print("same")
'''


@pytest.mark.parametrize("which", ["norm", "balance", "3", "200", "2000"])
def test_first_call_is_captured(which):
    r = subprocess.run([sys.executable, "-c", CHILD, which], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
