"""The operators around the layer without a GPU: sizes, and the refusals that come before any
CUDA call."""
import ctypes

import pytest

import token_routing_expert_router_gb300 as moe

P = ctypes.c_void_p
A, ODD = P(4096), P(4096 + 4)
INVALID, UNSUPPORTED, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


def norm_cfg(**kw):
    return moe.MoENormConfig.make(**{**dict(T=4, H=64), **kw})


def head_cfg(**kw):
    return moe.MoEHeadConfig.make(**{**dict(T=4, H=64, V=100), **kw})


def embed_cfg(**kw):
    return moe.MoEEmbedConfig.make(**{**dict(T=4, H=64, V=100), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(act_dtype=moe.E4M3), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(res_scale=float("inf")), INVALID),
    (dict(H=16385), UNSUPPORTED), (dict(H=16384), OK), (dict(T=0), OK)])
def test_norm_config(L, kw, code):
    n = ctypes.c_size_t()
    assert L.moe_block_norm_workspace_size(ctypes.byref(norm_cfg(**kw)), ctypes.byref(n)) == code


def test_norm_arguments(L):
    c = ctypes.byref(norm_cfg())

    def fwd(x=A, y=A, w_post=A, w_next=A, gate=None, token_gate=None, r=A, n=A, cfg=c):
        return L.moe_block_norm(cfg, x, y, w_post, w_next, gate, token_gate, r, n, None)

    assert fwd(x=None) == INVALID and fwd(x=ODD) == INVALID and fwd(y=ODD) == INVALID
    assert fwd(r=None, n=None) == INVALID          # nothing to form
    assert fwd(w_next=None) == INVALID             # n needs its weight
    assert fwd(y=None) == INVALID                  # a post norm without a block output
    assert fwd(y=None, w_post=None, gate=A) == INVALID
    assert fwd(y=None, w_post=None, token_gate=A) == INVALID
    for name in ("w_post", "w_next", "gate", "token_gate", "r", "n"):
        assert fwd(**{name: ODD}) == INVALID, name
    assert fwd(cfg=None) == INVALID
    assert fwd(x=None, cfg=ctypes.byref(norm_cfg(T=0))) == OK  # no rows: no buffer is touched

    def bwd(r=A, y=A, w_post=A, w_next=A, gate=None, token_gate=None, dr=A, dn=A, dx=A, dy=A, ws=A, **g):
        gr = moe.MoENormGrads.from_tensors(g)
        return L.moe_block_norm_backward(c, r, y, w_post, w_next, gate, token_gate, dr, dn, dx, dy, ctypes.byref(gr),
                                         ws, None)

    assert bwd(r=None) == INVALID and bwd(dr=None, dn=None, w_next=None) == INVALID
    assert bwd(dn=None) == INVALID and bwd(w_next=None) == INVALID
    assert bwd(y=None, w_post=None) == INVALID     # dy without y
    assert bwd(y=None, w_post=None, dy=None, dgate=4096) == INVALID
    assert bwd(w_post=None, dw_post=4096) == INVALID and bwd(w_next=None, dn=None, dw_next=4096) == INVALID
    assert bwd(dw_next=4096, ws=None) == INVALID and bwd(dgate=4100) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(V=0), INVALID), (dict(piece=-1), INVALID),
    (dict(act_dtype=moe.E4M3), INVALID), (dict(grad_dtype=moe.MXE4M3), INVALID), (dict(V=1 << 24), UNSUPPORTED),
    (dict(T=1 << 30, V=1 << 23), UNSUPPORTED), (dict(T=0), OK), (dict(H=33), OK)])
def test_head_config(L, kw, code):
    n = ctypes.c_size_t()
    assert L.moe_head_workspace_size(ctypes.byref(head_cfg(**kw)), ctypes.byref(n)) == code


def test_head_workspace_does_not_hold_the_logits(L):
    """A vocabulary 16 times as large adds only the (max, sum) pairs and the 256 MB piece's share."""
    small = moe.moe_head_workspace_size(head_cfg(T=8192, H=512, V=16384))
    large = moe.moe_head_workspace_size(head_cfg(T=8192, H=512, V=262144))
    assert large - small < 8192 * (262144 - 16384) * 2 / 8
    piece = moe.moe_head_workspace_size(head_cfg(T=8192, H=512, V=262144, piece=1024))
    assert piece < large


def test_head_arguments(L):
    c = ctypes.byref(head_cfg())

    def fwd(x=A, w=A, target=A, loss=A, lse=A, mean=None, ws=A):
        return L.moe_head_loss(c, x, w, target, loss, lse, mean, ws, None)

    for name in ("x", "w", "target", "loss", "lse", "ws"):
        assert fwd(**{name: None}) == INVALID and fwd(**{name: ODD}) == INVALID, name
    assert fwd(mean=ODD) == INVALID

    def bwd(x=A, w=A, target=A, lse=A, dloss=A, mean=None, dx=A, dw=A, ws=A):
        return L.moe_head_loss_backward(c, x, w, target, lse, dloss, mean, dx, dw, ws, None)

    for name in ("x", "w", "target", "lse", "ws"):
        assert bwd(**{name: None}) == INVALID and bwd(**{name: ODD}) == INVALID, name
    assert bwd(dloss=None) == INVALID and bwd(mean=A) == INVALID   # exactly one of the two
    assert bwd(dx=None, dw=None) == INVALID and bwd(dx=ODD) == INVALID and bwd(dw=ODD) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(V=0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(act_dtype=5), INVALID), (dict(grad_dtype=-1), INVALID), (dict(V=(1 << 21)), UNSUPPORTED),
    (dict(V=(1 << 21) - 1), OK), (dict(T=0), OK)])
def test_embed_config(L, kw, code):
    n = ctypes.c_size_t()
    assert L.moe_embed_workspace_size(ctypes.byref(embed_cfg(**kw)), ctypes.byref(n)) == code


def test_embed_arguments(L):
    c = ctypes.byref(embed_cfg())
    fwd = lambda table=A, token=A, out=A, ws=A: L.moe_embed(c, table, token, out, ws, None)
    bwd = lambda token=A, dout=A, dtable=A, acc=0, ws=A: L.moe_embed_backward(c, token, dout, dtable, acc, ws, None)
    for name in ("table", "token", "out", "ws"):
        assert fwd(**{name: None}) == INVALID and fwd(**{name: ODD}) == INVALID, name
    for name in ("token", "dout", "dtable", "ws"):
        assert bwd(**{name: None}) == INVALID and bwd(**{name: ODD}) == INVALID, name
    assert bwd(acc=2) == INVALID


def test_grad_clip_arguments(L):
    def call(grads, max_norm=1.0, norm=A, ws=A, count=None):
        a = (moe.MoEGrad * max(1, len(grads)))(*grads)
        return L.moe_grad_clip(a, len(grads) if count is None else count, ctypes.c_float(max_norm), norm, ws, None)

    good = moe.MoEGrad(4096, None, 10, moe.F32)
    assert call([good], max_norm=0.0) == INVALID and call([good], max_norm=float("nan")) == INVALID
    assert call([good], max_norm=float("inf")) == INVALID
    assert call([good], norm=None) == INVALID and call([good], ws=ODD) == INVALID
    assert call([good], count=-1) == INVALID
    assert call([moe.MoEGrad(None, None, 10, moe.F32)]) == INVALID
    assert call([moe.MoEGrad(4096 + 2, None, 10, moe.F32)]) == INVALID      # fp32 on a 2-byte boundary
    assert call([moe.MoEGrad(4096 + 1, None, 10, moe.BF16)]) == INVALID
    assert call([moe.MoEGrad(4096, 4096 + 2, 10, moe.F32)]) == INVALID
    assert call([moe.MoEGrad(4096, None, -1, moe.F32)]) == INVALID
    assert call([moe.MoEGrad(4096, None, 10, moe.E4M3)]) == INVALID
    assert call([moe.MoEGrad(4096, None, 1 << 41, moe.F32)]) == UNSUPPORTED
    assert L.moe_grad_norm(None, 1, A, A, None) == INVALID
    n = ctypes.c_size_t()
    assert L.moe_grad_clip_workspace_size(-1, ctypes.byref(n)) == INVALID
    assert moe.moe_grad_clip_workspace_size([None] * 500) > moe.moe_grad_clip_workspace_size([None])


def test_python_side_refusals():
    import torch
    with pytest.raises(TypeError):
        moe.MoENormConfig.make(T=1, H=8, epsilon=1e-6)
    with pytest.raises(ValueError):
        moe.MoEGradList.from_tensors([torch.zeros(4)])                  # not on the GPU
    with pytest.raises(ValueError):
        moe.MoEGradList.from_tensors([torch.zeros(4)], [])
    with pytest.raises(ValueError):
        moe.MoEGradList.from_tensors([torch.zeros(4, dtype=torch.float16)])
