"""First calls of the head from several host threads at once, each with its own stream and workspace."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import sys, threading
sys.path.insert(0, sys.argv[1])
import torch
import token_routing_expert_router_gb300 as moe

T, H, V, N = 300, 256, 1000, 8
g = torch.Generator(device="cuda"); g.manual_seed(1)
x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
w = (torch.randn(V, H, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
target = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
cfg = moe.MoEHeadConfig.make(T=T, H=H, V=V)
size = moe.moe_head_workspace_size(cfg)
state = []
for _ in range(N):
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    f = lambda *s: torch.empty(*s, device="cuda")
    state.append((torch.cuda.Stream(), ws, f(T), f(T), f(2), torch.empty_like(x), f(V, H)))
torch.cuda.synchronize()
start, errors = threading.Barrier(N), []

def work(stream, ws, loss, lse, mean, dx, dw):
    try:
        start.wait()
        moe.moe_head_loss(cfg, x, w, target, loss, lse, mean, ws, stream=stream)
        moe.moe_head_loss_backward(cfg, x, w, target, lse, dx, dw, ws, mean=mean, stream=stream)
    except Exception as e:
        errors.append(e)

threads = [threading.Thread(target=work, args=s) for s in state]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
for s in state:
    assert moe.moe_read_status(s[1]) == moe.MOE_OK
    assert all(torch.equal(a, b) for a, b in zip(s[2:], state[0][2:]))
print("same bits in", N, "threads")
"""


def test_first_calls_from_many_threads(lib):
    r = subprocess.run([sys.executable, "-c", PROGRAM, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "same bits" in r.stdout
