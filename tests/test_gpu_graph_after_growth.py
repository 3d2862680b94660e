"""A graph captured while the library's workspace was small is replayed after
a larger call made the workspace grow: it still owns the scratch it was
captured with.  In a process of its own, where the workspace starts empty."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
from exact_blocked_attention_gb300 import blkattn
torch.cuda.set_device(0)
def problem(B, H, T, K, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(s, generator=g).to(dtype).cuda() for s in ((B, H, T, d), (B, 2, K, d), (B, 2, K, d)))
    lens = torch.full((B,), K, dtype=torch.int32, device="cuda")
    return q, k, v, lens, (lens[:, None] - T + torch.arange(T, dtype=torch.int32, device="cuda")).contiguous()
small = [problem(1, 4, 1, 700, 128, torch.bfloat16, 1), problem(1, 4, 2, 900, 64, torch.float32, 2)]
graphs = []
for p in small:
    want = blkattn.attention(*p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = blkattn.attention(*p)
    graphs.append((graph, got, [t.clone() for t in want]))
for step in range(3):  # the workspace and the counters grow, more than once
    big = problem(8 << step, 64, 6, 600, 128, torch.bfloat16, 3)
    blkattn.attention(*big)
    torch.cuda.synchronize()
    for graph, got, want in graphs:
        for t in got:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
assert blkattn.check_device_error() == 0
print("same after growth")
"""


def test_graph_replays_after_the_workspace_grew():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "same after growth" in r.stdout
