"""A process's first prompt calls inside a capture, with contexts that clusters share (whose room on the device is asked for
then)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import torch
from moe_decode_megakernel_02_gb300 import latent
g = torch.Generator(device="cuda").manual_seed(1)
rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(DTYPE)
q, k, r, v = rand(9, 2, 192), rand(9000, 2, 128), rand(9000, 64), rand(9000, 2, 128)
qa, ka = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (9, 9000))
call = lambda: latent.attend_prompt(q, k, r, v, qa, ka, 0.07, return_lse=True)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    a = call()
graph.replay()
b = call()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(a, b)) and bool(torch.isfinite(a[0].float()).all())
print("same")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["torch.bfloat16", "torch.float16"])
def test_the_first_clustered_call_of_a_process_may_be_captured(dtype):
    r = subprocess.run([sys.executable, "-c", FIRST.replace("DTYPE", dtype)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
