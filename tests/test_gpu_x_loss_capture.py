"""Loss calls whose first use in a process lies in a stream capture: what is asked of the device once is asked there."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
import overlapped_tensor_gemm_gb300 as fo
ctx = fo.Context(0)
g = torch.Generator(device="cuda").manual_seed(1)
z = [torch.randn((200, 40000), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
y = torch.randint(0, 80000, (200,), generator=g, device="cuda", dtype=torch.int32)
logp, lse, ent, stats = (torch.empty(n, device="cuda") for n in (200, 200, 200, 4))
d, d2, adv = [torch.empty_like(t) for t in z], [torch.empty_like(t) for t in z], torch.rand(200, device="cuda")

def step():
    ctx.token_logprobs(z, y, logp, lse=lse, entropy=ent)
    ctx.token_logprobs_backward(z, y, lse, adv, d)
    if len(sys.argv) > 2:
        ctx.policy_loss(z, y, adv, stats, dlogits=d2, entropy_coef=0.1)

if len(sys.argv) > 2:  # (the policy loss's workspace has to be there)
    few = [torch.zeros((0, 64), device="cuda", dtype=torch.bfloat16)]
    ctx.policy_loss(few, y[:0], adv[:0], stats)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
outs = [logp, lse, ent] + d + ([stats] + d2 if len(sys.argv) > 2 else [])
got = [t.clone() for t in outs]
for t in outs:
    t.zero_()
step()
torch.cuda.synchronize()
ctx.poll()
assert all(torch.equal(a, b) for a, b in zip(got, outs)) and logp.abs().sum() > 0
want = torch.log_softmax(torch.cat(z, 1).double(), 1).gather(1, y.long()[:, None])[:, 0]
assert (logp.double() - want).abs().max() < 1e-4
print("fine")
"""


@pytest.mark.parametrize("policy", [[], ["policy"]], ids=["logprobs", "with policy"])
def test_first_use_in_a_capture(repo_root, policy):
    out = subprocess.run([sys.executable, "-c", PROGRAM, repo_root, *policy], capture_output=True, text=True, timeout=300,
                         env=dict(os.environ))
    assert out.returncode == 0 and "fine" in out.stdout, out.stderr[-2000:]
