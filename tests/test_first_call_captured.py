"""A process's first call of a kernel may be one that a graph captures: what the
library sets up or asks of the device for it then happens under the capture."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch, pair_biased_attention_b200 as pba
q, k, v = (torch.randn((2, h, n, 64), device="cuda").to(torch.bfloat16) for h, n in ((8, {Nq}), (4, 700), (4, 700)))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out, lse = pba.pba_cross_attn_forward(q, k, v)
    grads = pba.pba_cross_attn_backward(q, k, v, out, lse, q)
graph.replay()
want, want_lse = pba.pba_cross_attn_forward(q, k, v)
more = pba.pba_cross_attn_backward(q, k, v, want, want_lse, q)
assert all(torch.equal(a, b) for a, b in zip((out, lse, *grads), (want, want_lse, *more)))
assert pba.pba_last_device_error() == pba.PBA_OK
print("same")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("Nq", [1, 300])  # few rows; tiles in clusters
def test_cross_attention(cuda_device, Nq):
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(Nq=Nq)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
