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


ATTENTION = r"""
import sys, threading
sys.path.insert(0, sys.argv[1])
import torch
import token_routing_expert_router_gb300 as moe

N, Hq, Hkv, D = 8, 4, 2, 64
g = torch.Generator(device="cuda"); g.manual_seed(1)
i32 = lambda *v: torch.tensor(v, device="cuda", dtype=torch.int32)
jobs = []  # of every thread: (stream, calls, workspaces, outputs)
table = torch.empty(D // 2, device="cuda", dtype=torch.int64)
moe.moe_rope_table(moe.MoERopeFreq.make(rot=D), table)

# query rows, keys, dtype, with its backward: tiles of 256 rows, shares of the keys, 64 and 16 rows on the FMA
# units, parts of lines
SHAPES = [([300, 45, 700], [300, 45, 700], torch.bfloat16, True), ([1, 1], [900, 33], torch.bfloat16, False),
          ([900, 400, 700], [900, 400, 700], torch.float32, True), ([60, 30], [60, 30], torch.float32, True),
          ([1, 2], [700, 90], torch.float32, False)]
inputs = []
for new, keys, dt, train in SHAPES:
    T, K = sum(new), sum(keys)
    q, k, v = (torch.randn(r, h, D, generator=g, device="cuda").to(dt) for r, h in ((T, Hq), (K, Hkv), (K, Hkv)))
    ends = lambda n: [sum(n[:i]) for i in range(len(n) + 1)]
    inputs.append((q, k, v, i32(*ends(new)), i32(*ends(keys)[:-1]), i32(*keys), torch.arange(T, device="cuda", dtype=torch.int32)))
for _ in range(N):
    calls, spaces, outs, stream = [], [], [], torch.cuda.Stream()
    for (new, keys, dt, train), (q, k, v, q_start, k_start, k_len, pos) in zip(SHAPES, inputs):
        code, T = (moe.BF16 if dt == torch.bfloat16 else moe.F32), sum(new)
        cfg = moe.MoEAttnConfig.make(Tq=T, Tk=sum(keys), B=len(new), Hq=Hq, Hkv=Hkv, D=D, act_dtype=code, max_q=max(new))
        ws = torch.empty(max(moe.moe_attn_workspace_size(cfg), moe.moe_attn_backward_workspace_size(cfg)), dtype=torch.uint8, device="cuda")
        moe.moe_workspace_init(ws)
        rope = moe.MoERopeConfig.make(T=T, Hq=Hq, Hk=0, D=D, act_dtype=code)
        x, o, lse, dq, dk, dv = (torch.zeros_like(q), torch.zeros_like(q), torch.zeros(Hq, T, device="cuda"), torch.zeros_like(q),
                                 torch.zeros_like(k), torch.zeros_like(v))

        def call(a=(cfg, rope, q, k, v, q_start, k_start, k_len, pos, x, o, lse, dq, dk, dv, ws, train), s=stream):
            cfg, rope, q, k, v, q_start, k_start, k_len, pos, x, o, lse, dq, dk, dv, ws, train = a
            moe.moe_rope(rope, q, None, None, pos, None, table, x, None, None, stream=s)
            moe.moe_attn(cfg, x, k, v, q_start, k_start, k_len, o, lse, ws, stream=s)
            if train:
                moe.moe_attn_backward(cfg, x, k, v, q_start, k_start, k_len, o, lse, q, dq, dk, dv, ws, stream=s)

        calls.append(call), spaces.append(ws), outs.extend((x, o, lse, dq, dk, dv))
    jobs.append((calls, spaces, outs))
torch.cuda.synchronize()
start, errors = threading.Barrier(N), []

def work(calls):
    try:
        start.wait()
        for call in calls:
            call()
    except Exception as e:
        errors.append(e)

threads = [threading.Thread(target=work, args=(j[0],)) for j in jobs]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
for calls, spaces, outs in jobs:
    assert all(moe.moe_read_status(ws) == moe.MOE_OK for ws in spaces)
    assert all(torch.isfinite(x).all() and torch.equal(x, y) for x, y in zip(outs, jobs[0][2]))
assert all(x.any() for x in jobs[0][2][:6])
print("same bits in", N, "threads")
"""


def test_first_calls_of_attention_from_many_threads(lib):
    r = subprocess.run([sys.executable, "-c", ATTENTION, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "same bits" in r.stdout
