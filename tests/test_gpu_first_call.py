"""The first paged calls of a process may come inside a graph capture: their kernels are set up then."""

from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

TESTS = os.path.dirname(os.path.abspath(__file__))
CODE = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import exact_attention_116_b200 as fa
from chunk_cases import Batch, assert_close, call
b = Batch([3, 1], [300, 200], 8, 2, 128, 16, {f8}, seed=1)
t = b.gpu()
x = torch.randn(1, 64, 2, 128, device="cuda").bfloat16()
if {forward}:
    fa.attention_fwd(x, x.clone(), x.clone())
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    k, v = fa.cache_read_paged(t["k"], t["v"], t["table"], t["lens"], t["cu"], b.total, t["ks"], t["vs"])
    fa.cache_write_paged(k, v, t["k"], t["v"], t["table"], t["lens"], t["cu"], t["ks"], t["vs"])
    o, lse = call(t)
graph.replay()
torch.cuda.synchronize()
fa.check()
assert_close(o, lse, b.reference(128 ** -0.5, True, (-1, -1), 0), 4, "first call")
"""


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("forward", [False, True])
def test_first_calls_in_a_capture(forward, f8):
    code = CODE.format(root=os.path.dirname(TESTS), tests=TESTS, f8=f8, forward=forward)
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)
