"""The first call of a process captured into a graph: what a call sets up once (the error word,
limits of shared memory, the question after room for large clusters) may come under capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = r"""
import sys
import torch
from block_sparse_attention_online_gb300 import binding as bs
from tests import pages_plain as plain
from tests.test_gpu_pages import host, i32, pools, same

which = sys.argv[1]
side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
if which == "reserve":
    n, n_pages = 8192, 70000
    R, T = torch.zeros(n_pages, dtype=torch.int32, device="cuda"), i32([[-1]] * n)
    a, b = i32([0] * n), i32([1] * n)
    out = [torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(3)]
    call = lambda: bs.attn_skip_pages_reserve(R, T, a, b, 16, out=out)
    def check():
        assert T[:, 0].tolist() == list(range(n)) and R.sum() == n and out[0].tolist() == [1] * n
elif which == "verify":
    p = torch.zeros(1, 100000, device="cuda")
    p[0, 77777] = 1.0
    x, cu, ua, us = i32([]), i32([0, 0]), torch.zeros(0, device="cuda"), torch.full((1,), 0.5, device="cuda")
    out = torch.full((1, 1), -7, dtype=torch.int32, device="cuda"), i32([-7])
    call = lambda: bs.attn_skip_verify_drafts(p, x, cu, 0, ua, us, out=out)
    def check():
        assert out[0].tolist() == [[77777]] and out[1].tolist() == [0]
else:
    L = 3000
    kv, parts = pools(which, 1, 188, 1, 16, 3)
    keep, cu, table = list(range(1, L)), [0, L - 1], [list(range(188))]
    before = host(parts)
    args = i32(keep), i32(cu), i32(table)
    call = lambda: bs.attn_skip_kv_compact(kv, *args)
    def check():
        same(parts, [{m: plain.compact(x, keep, cu, table, 16) for m, x in p.items()} for p in before])
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=side):
    call()
torch.cuda.synchronize()
graph.replay()
torch.cuda.synchronize()
check()
bs.attn_skip_last_device_error()
print("well")
"""


@pytest.mark.parametrize("which", ["reserve", "verify", "bf16", "nvfp4"])
def test_the_first_call_may_be_captured(which):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM, which], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "well", r.stderr[-2000:]
