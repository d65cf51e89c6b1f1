"""Rotary positions and attention without a GPU: sizes, and the refusals that come before any CUDA call."""
import ctypes

import pytest
import torch

import token_routing_expert_router_gb300 as moe

P = ctypes.c_void_p
A, ODD, BYTE = P(4096), P(4096 + 4), P(4096 + 1)
INVALID, UNSUPPORTED, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


def rope_cfg(**kw):
    return moe.MoERopeConfig.make(**{**dict(T=4, Hq=4, Hk=2, D=64, slots=8), **kw})


def attn_cfg(**kw):
    return moe.MoEAttnConfig.make(**{**dict(Tq=10, Tk=20, B=2, Hq=4, Hkv=2, D=64), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(rot=3), INVALID), (dict(rot=-2), INVALID), (dict(scaling=3), INVALID), (dict(base=0.0), INVALID),
    (dict(base=float("nan")), INVALID), (dict(scaling=moe.ROPE_LINEAR, factor=0.0), INVALID),
    (dict(scaling=moe.ROPE_YARN, trained_len=0.0), INVALID), (dict(scaling=moe.ROPE_YARN, beta_fast=1.0), INVALID),
    (dict(scaling=moe.ROPE_YARN, factor=float("inf")), INVALID), (dict(rot=4098), UNSUPPORTED), (dict(rot=0), OK)])
def test_rope_table(L, kw, code):
    assert L.moe_rope_table(ctypes.byref(moe.MoERopeFreq.make(**{"rot": 64, **kw})), None if code == OK else A, None) == code


def test_rope_table_arguments(L):
    f = ctypes.byref(moe.MoERopeFreq.make(rot=64))
    assert L.moe_rope_table(None, A, None) == INVALID
    assert L.moe_rope_table(f, None, None) == INVALID and L.moe_rope_table(f, ODD, None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hq=0, Hk=0), INVALID), (dict(D=0, rot=0), INVALID),
    (dict(rot=3), INVALID), (dict(rot=66), INVALID), (dict(rot=32, first=33), INVALID), (dict(first=-1, rot=2), INVALID),
    (dict(first=2 ** 31 - 1, rot=2), INVALID), (dict(layout=2), INVALID), (dict(act_dtype=moe.E4M3), INVALID),
    (dict(slots=-1), INVALID), (dict(magnitude=float("nan")), INVALID), (dict(ld_q=255), INVALID), (dict(ld_k=-1), INVALID),
    (dict(ld_v_out=127), INVALID), (dict(ld_q=1 << 32), INVALID), (dict(D=4098), UNSUPPORTED), (dict(Hq=20000), UNSUPPORTED), (dict(Hk=2000, D=4096), UNSUPPORTED),
    (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(T=0), OK)])
def test_rope_config(L, kw, code):
    c = ctypes.byref(rope_cfg(**kw))
    none = [None] * 10
    assert L.moe_rope(c, *none, None) == code
    assert L.moe_rope_backward(c, *[None] * 6, None) == code


def test_rope_arguments(L):
    def fwd(cfg=rope_cfg(), q=A, k=A, v=A, pos=A, slot=A, table=A, q_out=A, k_out=A, v_out=A, ws=A):
        return L.moe_rope(ctypes.byref(cfg), q, k, v, pos, slot, table, q_out, k_out, v_out, ws, None)

    for name in ("q", "k", "v", "pos", "table", "q_out", "k_out", "v_out", "ws"):
        assert fwd(**{name: None}) == INVALID, name
    for name in ("q", "k", "v", "q_out", "k_out", "v_out", "pos", "slot", "table", "ws"):
        assert fwd(**{name: BYTE}) == INVALID, name
    for name in ("q", "k", "v", "q_out", "k_out", "v_out"):  # fp32 rows on a 2-byte boundary
        assert fwd(cfg=rope_cfg(act_dtype=moe.F32), **{name: P(4096 + 2)}) == INVALID, name
    assert fwd(table=ODD) == INVALID and fwd(ws=ODD) == INVALID

    def bwd(cfg=rope_cfg(), a=A, b=A, pos=A, table=A, dq=A, dk=A):
        return L.moe_rope_backward(ctypes.byref(cfg), a, b, pos, table, dq, dk, None)

    for name in ("a", "b", "pos", "table", "dq", "dk"):
        assert bwd(**{name: None}) == INVALID and bwd(**{name: BYTE}) == INVALID, name


@pytest.mark.parametrize("kw,code", [
    (dict(Tq=-1), INVALID), (dict(Tk=-1), INVALID), (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(Hq=5), INVALID), (dict(D=0, scale=1.0), INVALID), (dict(causal=2), INVALID), (dict(max_q=-1), INVALID),
    (dict(act_dtype=moe.MXE4M3), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=2.0 ** 101), INVALID), (dict(scale=2.0 ** -101), INVALID),
    (dict(scale=2.0 ** 100), OK), (dict(scale=2.0 ** -100), OK), (dict(scale=float("nan")), INVALID), (dict(ld_q=255), INVALID),
    (dict(ld_k=127), INVALID), (dict(ld_v=-128), INVALID), (dict(ld_o=100), INVALID), (dict(D=129), UNSUPPORTED),
    (dict(Hq=32768), UNSUPPORTED), (dict(B=(1 << 16) + 1), UNSUPPORTED), (dict(Tk=(1 << 30) + 1), UNSUPPORTED),
    (dict(D=128), OK), (dict(D=1), OK), (dict(Tq=0), OK), (dict(B=0), OK)])
def test_attn_config(L, kw, code):
    c, n = ctypes.byref(attn_cfg(**kw)), ctypes.c_size_t()
    assert L.moe_attn_workspace_size(c, ctypes.byref(n)) == code
    assert L.moe_attn_backward_workspace_size(c, ctypes.byref(n)) == code


def test_attn_arguments(L):
    def fwd(cfg=attn_cfg(), q=A, k=A, v=A, q_start=A, k_start=A, k_len=A, o=A, lse=A, ws=A):
        return L.moe_attn(ctypes.byref(cfg), q, k, v, q_start, k_start, k_len, o, lse, ws, None)

    names = ("q", "k", "v", "q_start", "k_start", "k_len", "o", "lse", "ws")
    for name in names:
        assert fwd(**{name: None}) == INVALID, name
        assert fwd(**{name: BYTE}) == INVALID, name
    assert fwd(ws=ODD) == INVALID
    assert fwd(cfg=attn_cfg(act_dtype=moe.F32), q=P(4096 + 2)) == INVALID
    assert fwd(cfg=attn_cfg(Tk=9), k_start=None, k_len=None) == INVALID   # the keys are the queries' rows
    assert fwd(cfg=attn_cfg(Tq=0), q=None, o=None, lse=None) == OK
    assert fwd(cfg=attn_cfg(B=0), q_start=None) == OK

    def bwd(cfg=attn_cfg(), q=A, k=A, v=A, q_start=A, k_start=A, k_len=A, o=A, lse=A, do=A, dq=A, dk=A, dv=A, ws=A):
        return L.moe_attn_backward(ctypes.byref(cfg), q, k, v, q_start, k_start, k_len, o, lse, do, dq, dk, dv, ws, None)

    for name in names + ("do", "dq", "dk", "dv"):
        assert bwd(**{name: None}) == INVALID, name
        assert bwd(**{name: BYTE}) == INVALID, name
    assert bwd(cfg=attn_cfg(Tk=9), k_start=None, k_len=None) == INVALID
    assert bwd(cfg=attn_cfg(B=0), q_start=None) == OK
    assert bwd(cfg=attn_cfg(Tq=0, Tk=0), q_start=None) == OK


def test_python_side_refusals():
    with pytest.raises(ValueError):
        moe._rows(torch.zeros(4, 8), 0, 8)           # not on the GPU
    with pytest.raises(TypeError):
        moe.MoEAttnConfig.make(Tq=1, Tk=1, B=1, Hq=1, Hkv=1, D=8, window=4)
    assert moe.MoEAttnConfig.make(Tq=1, Tk=1, B=1, Hq=1, Hkv=1, D=16).scale == 0.25
    assert moe.MoERopeConfig.make(T=1, Hq=1, Hk=1, D=48).rot == 48


class Fake:
    """A CUDA tensor as far as the binding looks at one."""

    is_cuda = True

    def __init__(self, t):
        self.t, self.shape = t, t.shape

    def stride(self, *a):
        return self.t.stride(*a)

    def dim(self):
        return self.t.dim()

    def data_ptr(self):
        return 4096


def test_rows_follow_the_configuration():
    row = torch.zeros(5, 8, 16)
    assert moe._rows(Fake(row[:, :2]), 128, 32) == 4096 and moe._rows(Fake(row.reshape(5, 128)[:, 32:64]), 128, 32) == 4096
    assert moe._rows(Fake(row[:1, :2]), 0, 32) == 4096          # one row has no stride
    assert moe._rows(Fake(row), 0, 128) == 4096 and moe._rows(None, 0, 128) is None and moe._rows(4096, 0, 1) == 4096
    for t, ld, width in ((row[:, :2], 0, 32), (row[:, :2], 128, 16), (row[:, ::2], 128, 64), (row[:, :, ::2], 128, 64),
                         (row.transpose(1, 2), 128, 128), (row[0, 0], 0, 16)):
        with pytest.raises(ValueError):
            moe._rows(Fake(t), ld, width)
