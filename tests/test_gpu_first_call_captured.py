"""The first call of a process may be the one that a graph captures: whatever an
operator asks about the device or sets up then is allowed in a capture."""

import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import sys
sys.path.insert(0, ".")
import torch
from w4a16_int4_moe_gb300 import ops
bf = torch.bfloat16
gen = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(TOKENS, 1024, generator=gen, device="cuda").to(bf)
w = (torch.randn(640, 1024, generator=gen, device="cuda") / 32).to(bf)
q = torch.randint(0, 256, (1, 640, 512), generator=gen, device="cuda", dtype=torch.uint8)
s = torch.rand(1, 640, 32, generator=gen, device="cuda").to(bf)
packed = ops.w4a16_prepack(q, s)

def calls():
    out = [ops.w4a16_dense(x, w), ops.w4a16_dense(x, w, gated=True),
           ops.w4a16_block_norm(x, w[0].contiguous(), post_weight=w[1].contiguous())[0]]
    if TOKENS <= 32:
        out.append(ops.w4a16_linear_few_tokens(x, packed, 640))
    return out

side = torch.cuda.Stream()
side.wait_stream(torch.cuda.current_stream())
graph = torch.cuda.CUDAGraph()
with torch.cuda.stream(side):
    with torch.cuda.graph(graph, stream=side):
        got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
print("same")
"""


@pytest.mark.parametrize("tokens", [3, 40, 300, 4000])
def test_the_first_call_is_captured(cuda_dev, tokens):
    r = subprocess.run([sys.executable, "-c", CODE.replace("TOKENS", str(tokens))],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
