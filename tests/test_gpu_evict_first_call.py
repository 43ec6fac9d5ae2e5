"""The first eviction of a process, captured into a graph: what the launch
asks the device about clusters once must not end the capture."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
import paged_kv_cache_44_gb300 as pkv
n = {n}
slots = torch.randperm(n, device="cuda").int()[None]
scores = torch.randperm(n, device="cuda").float()[None]
num = torch.tensor([n], dtype=torch.int32, device="cuda")
new, ns, nn = torch.zeros_like(slots), torch.zeros_like(scores), torch.zeros_like(num)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    pkv.evict_tokens(slots, scores, num, new, ns, nn, 1000)
graph.replay()
keep = scores[0].topk(1000).indices.sort().values
assert int(nn) == 1000 and torch.equal(new[0, :1000], slots[0, keep]) and torch.equal(ns[0, :1000], scores[0, keep])
print("same")
"""


@pytest.mark.parametrize("n", [140000, 300000])
def test_first_call_in_a_capture(n):
    """Sixteen blocks per cluster; the longer one's shares do not fit shared memory."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = subprocess.run([sys.executable, "-c", PROGRAM.format(n=n)], cwd=root, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "same" in got.stdout, got.stderr[-2000:]
