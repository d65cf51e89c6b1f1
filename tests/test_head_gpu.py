"""The vocabulary head where its arithmetic can go wrong: tokens that the model is sure of.

Bounds are by norm: a value rounded to bf16 is off by at most HALF of itself and, over many
values, by HALF / sqrt(3) of their norm.
"""
import math

import pytest
import torch

import token_routing_expert_router_gb300 as moe
from test_step_gpu import BF, CODE, FP, HALF, U, gen, normal, poisoned, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(lib):
    pass


def relative(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("dt,T,H,V,lean", [(BF, 512, 4096, 8000, 1.0), (BF, 512, 4096, 8000, 1.5), (BF, 512, 4096, 8000, 2.0),
                                           (BF, 100, 4096, 8000, 2.0), (BF, 200, 1021, 8000, 8.0), (FP, 256, 1024, 8000, 8.0)])
def test_gradients_of_tokens_that_are_nearly_certain(dt, T, H, V, lean):
    """The target's dz is p - 1 with p near 1: what is left is the error of z - lse, so the target's
    logit and lse have to be of one making."""
    g = gen(1)
    w, t = normal(g, V, H, dtype=dt, std=0.05), torch.randint(0, V, (T,), generator=g, device="cuda")
    x = (normal(g, T, H, std=0.3) + lean * w[t].float()).to(dt)
    target = t.to(torch.int32)
    cfg = moe.MoEHeadConfig.make(T=T, H=H, V=V, act_dtype=CODE[dt])
    ws = workspace(moe.moe_head_workspace_size(cfg))
    loss, lse, mean = poisoned(T, dtype=FP), poisoned(T, dtype=FP), poisoned(2, dtype=FP)
    dx, dw = poisoned(T, H, dtype=dt), poisoned(V, H, dtype=FP)
    moe.moe_head_loss(cfg, x, w, target, loss, lse, mean, ws)
    moe.moe_head_loss_backward(cfg, x, w, target, lse, dx, dw, ws, mean=mean)

    X, W = x.double(), w.double()
    z = X @ W.t()
    want = torch.logsumexp(z, 1)
    D = torch.exp(z - want[:, None])
    others = D.scatter(1, t[:, None], 0.0).sum(1)  # 1 - p of the target
    D.scatter_(1, t[:, None], -others[:, None])
    D /= T
    # z and lse are rounded to fp32 (two halves of U each in the last additions of the sum, and lse's own)
    sure = 4 * U * want.abs().max().item() / others.square().mean().sqrt().item()
    tc = HALF[BF] / math.sqrt(3) if dt == BF and H % 8 == 0 else 0.0  # dz as the next products' operand
    assert relative(dw, D.t() @ X) < tc + sure + 16 * U
    assert relative(dx, D @ W) < math.hypot(tc, HALF[dt] / math.sqrt(3)) + sure + 16 * U
    assert ((loss.double() - (want - z.gather(1, t[:, None])[:, 0])).abs() <= 8 * U * (1 + want.abs())).all()
