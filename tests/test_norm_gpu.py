"""The block norms' optional gradients, and calls of several widths in turn."""
import math
import time

import pytest
import torch

import token_routing_expert_router_gb300 as moe
from test_step_gpu import BF, CODE, EPS, FP, RES, gen, norm_inputs, normal, poisoned, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(lib):
    pass


SHAPES = [(1, 8, BF), (37, 264, BF), (300, 2048, BF), (9, 999, BF), (40, 1001, FP), (20, 7168, FP), (33, 8200, BF), (12, 16384, FP),
          (15, 5002, BF)]


@pytest.mark.parametrize("T,H,dt", SHAPES)
@pytest.mark.parametrize("post,gates", [(1, 1), (0, 0)])
def test_a_gradient_that_is_left_out_is_zero(T, H, dt, post, gates):
    """dr NULL (nothing but the next norm reads the residual) gives the bits of a dr of zeros; dx or dy
    NULL the bits of the other outputs; without a next norm likewise."""
    d = norm_inputs(T, H, dt, post, 1, gates, gates, seed=T)
    g = gen(7)
    dr, dn = normal(g, T, H, dtype=dt), normal(g, T, H, dtype=dt)
    zero = torch.zeros_like(dr)
    cfg = moe.MoENormConfig.make(T=T, H=H, act_dtype=CODE[dt], eps=EPS, res_scale=RES)
    ws = workspace(moe.moe_block_norm_workspace_size(cfg))

    def call(dr, dn, want_x=True, want_y=True):
        out = {"dx": poisoned(T, H, dtype=dt) if want_x else None, "dy": poisoned(T, H, dtype=dt) if want_y else None}
        grads = {"dgate": poisoned(H, dtype=FP), "dtoken_gate": poisoned(T, dtype=FP)}
        if post:
            grads["dw_post"] = poisoned(H, dtype=FP)
        if dn is not None:
            grads["dw_next"] = poisoned(H, dtype=FP)
        moe.moe_block_norm_backward(cfg, d["x"], d["y"], d["w_post"], d["w_next"] if dn is not None else None, dr, dn,
                                    out["dx"], out["dy"], grads, ws, gate=d["gate"], token_gate=d["token_gate"])
        return {**out, **grads}

    def same(a, b):
        for name in a:
            if a[name] is not None and b[name] is not None:
                assert torch.isfinite(a[name]).all() and torch.equal(a[name], b[name]), name

    same(call(None, dn), call(zero, dn))
    whole = call(dr, dn)
    for left_out in (dict(want_x=False), dict(want_y=False), dict(want_x=False, want_y=False)):
        same(whole, call(dr, dn, **left_out))
    same(call(dr, None), call(dr, None, want_x=False))


@pytest.mark.parametrize("T,H,dt", SHAPES)
def test_the_stream_alone(T, H, dt):
    """No block output: dx from dr and dn, and from dn alone, with the bits that a block output behind a
    token gate of zeros gives."""
    g = gen(T + H)
    r, y, dr, dn = (normal(g, T, H, dtype=dt) for _ in range(4))
    w, shut = normal(g, H, mean=1.0, std=0.2), torch.zeros(T, device="cuda")
    cfg = moe.MoENormConfig.make(T=T, H=H, act_dtype=CODE[dt], eps=EPS, res_scale=RES)
    ws = workspace(moe.moe_block_norm_workspace_size(cfg))
    for a in (dr, None):
        dx, dx2, dw, dw2 = poisoned(T, H, dtype=dt), poisoned(T, H, dtype=dt), poisoned(H, dtype=FP), poisoned(H, dtype=FP)
        moe.moe_block_norm_backward(cfg, r, None, None, w, a, dn, dx, None, {"dw_next": dw}, ws)
        moe.moe_block_norm_backward(cfg, r, y, None, w, a, dn, dx2, None, {"dw_next": dw2}, ws, token_gate=shut)
        assert torch.isfinite(dx).all() and torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("widths", [(1536, 2048), (12288, 16384)])
def test_widths_in_turn_cost_no_more_than_one(widths):
    """What a launch needs of the device is asked for once per width, not whenever the width changes."""
    g, calls = gen(3), {}
    for H in widths:
        r, dn, dx, w = normal(g, 1, H, dtype=BF), normal(g, 1, H, dtype=BF), poisoned(1, H, dtype=BF), normal(g, H, mean=1.0)
        cfg = moe.MoENormConfig.make(T=1, H=H)

        def call(cfg=cfg, r=r, dn=dn, w=w, dx=dx):
            moe.moe_block_norm_backward(cfg, r, None, None, w, None, dn, dx, None, {}, None)
        calls[H] = call

    def seconds(order):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for H in order:
            calls[H]()
        return time.perf_counter() - t0

    a, b = widths
    one = turn = math.inf
    for i in range(100):  # the least of each; more of them where the host is busy with other things
        one, turn = min(one, seconds([a] * 100 + [b] * 100)), min(turn, seconds([a, b] * 100))
        if i >= 15 and turn < 1.1 * one:
            break
    print(f"{one * 5e3:.2f} us a call of one width, {turn * 5e3:.2f} us in turn")
    assert turn < 1.1 * one
