"""The first call of a process may be a captured one: what the library makes once for itself (the pool that scratch
comes from) is no part of a graph and does not end its capture.  Each case is a process of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
import torch
import sinkhorn_point_cloud_gb300 as sot
g = torch.Generator(device="cuda").manual_seed(0)
r = lambda *n: torch.randn(*n, device="cuda", generator=g).bfloat16()
layer = r(20, 64), r(8, 64), r(8, 64, 64), r(8, 64, 32)
ids, many, scores = torch.arange(2000, device="cuda") % 50, r(2000, 64), r(9000, 64)
chosen = torch.arange(9000, dtype=torch.int32, device="cuda")[:, None] % 64
call = {
    "routed": lambda: sot.sot_routed_layer(*layer, 2),
    "embed_grad": lambda: (sot.sot_embed_grad(many, ids, 50),),
    "embed_grad_few": lambda: (sot.sot_embed_grad(many[:100], ids[:100], 50),),
    "topk": lambda: sot.sot_token_topk(scores, 30)[1:],
    "balance": lambda: sot.sot_balance_loss(scores, chosen),
}[sys.argv[1]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
for a, b in zip(got, call()):
    assert torch.equal(a, b)
print("same")
"""


@pytest.mark.parametrize("call", ["routed", "embed_grad", "embed_grad_few", "topk", "balance"])
def test_first_call_captured(call):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sinkhorn_point_cloud_gb300 import build
    build.build()
    p = subprocess.run([sys.executable, "-c", PROGRAM, call], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.split() == ["same"], p.stderr[-2000:]
