"""Rotary positions against complex numbers in 64 bits."""
import math

import pytest
import torch

import token_routing_expert_router_gb300 as moe
from test_step_gpu import BF, CODE, FP, HALF, U, gen, normal, poisoned, within, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(lib):
    pass


YARN = dict(scaling=moe.ROPE_YARN, factor=40.0, trained_len=4096.0)
SCALINGS = [dict(), dict(scaling=moe.ROPE_LINEAR, factor=4.0), YARN, dict(scaling=moe.ROPE_YARN, factor=8.0, trained_len=512.0,
                                                                            base=500000.0, beta_fast=16.0, beta_slow=2.0)]


def frequencies(rot, scaling=moe.ROPE_UNSCALED, base=10000.0, factor=1.0, trained_len=1.0, beta_fast=32.0, beta_slow=1.0):
    """Radians per position, in 64 bits on the host."""
    out = []
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(base))
        if scaling == moe.ROPE_LINEAR:
            f /= factor
        elif scaling == moe.ROPE_YARN:
            keep = min(1.0, max(0.0, (trained_len * f / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow)))
            f = f * keep + f / factor * (1 - keep)
        out.append(f)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def turned(x, pos, freq, first, layout, m, sign):
    """The rotation in 64 bits, and the bound on what the library's arithmetic may lose of it."""
    rot = 2 * freq.numel()
    y, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    part = x.double()[..., first:first + rot]
    a, b = (part[..., :rot // 2], part[..., rot // 2:]) if layout == moe.ROPE_HALF else (part[..., 0::2], part[..., 1::2])
    angle = pos.double()[:, None, None] * freq
    z = torch.complex(a, b) * torch.polar(torch.full_like(angle, m), sign * angle)
    # the eighth of a turn that goes to fp32 loses 2^-27 turns; the table and this reference's own
    # product lose 2^-50 of the whole angle each
    lost = 2 * math.pi * 2.0 ** -27 + angle.abs() * 2.0 ** -49
    # cos and sin within an ulp (2 U), their product with m, two products and a sum
    mag = (5 * U + lost) * m * (a.abs() + b.abs())
    cat = (lambda u, v: torch.cat([u, v], -1)) if layout == moe.ROPE_HALF else (lambda u, v: torch.stack([u, v], -1).flatten(-2))
    y[..., first:first + rot] = cat(z.real, z.imag)
    size[..., first:first + rot] = cat(mag, mag)
    return y, size + HALF[x.dtype] * (y.abs() + size) * (size > 0)


CASES = [
    # T, Hq, Hk, D, rot, first, layout, dtype, scaling
    (1, 32, 8, 128, 128, 0, moe.ROPE_HALF, BF, 0), (5, 3, 1, 64, 64, 0, moe.ROPE_INTERLEAVED, FP, 1),
    (1000, 16, 4, 128, 128, 0, moe.ROPE_HALF, BF, 2), (257, 4, 2, 192, 64, 128, moe.ROPE_INTERLEAVED, BF, 2),
    (33, 2, 2, 80, 72, 4, moe.ROPE_HALF, BF, 0), (33, 2, 2, 80, 72, 4, moe.ROPE_HALF, FP, 3),
    (17, 1, 1, 50, 50, 0, moe.ROPE_HALF, FP, 1), (17, 3, 1, 50, 26, 7, moe.ROPE_INTERLEAVED, BF, 0),
    (64, 5, 0, 24, 8, 16, moe.ROPE_HALF, BF, 0), (64, 0, 5, 24, 20, 2, moe.ROPE_INTERLEAVED, FP, 0),
    (9, 2, 1, 2, 2, 0, moe.ROPE_HALF, BF, 0), (300, 2, 1, 1, 0, 1, moe.ROPE_HALF, FP, 0),
    (3, 2, 1, 4096, 4096, 0, moe.ROPE_HALF, BF, 0), (12, 8, 8, 40, 0, 0, moe.ROPE_INTERLEAVED, BF, 0),
    (700, 64, 1, 576, 64, 512, moe.ROPE_INTERLEAVED, BF, 2), (4100, 4, 4, 36, 36, 0, moe.ROPE_INTERLEAVED, FP, 2),
    (50, 7, 7, 66, 12, 54, moe.ROPE_HALF, BF, 1)]


def inputs(T, Hq, Hk, D, dt, packed, seed=0):
    g = gen(seed)
    if packed:
        row = normal(g, T, Hq + 2 * Hk, D, dtype=dt)
        return row[:, :Hq], row[:, Hq:Hq + Hk], row[:, Hq + Hk:], (Hq + 2 * Hk) * D
    return normal(g, T, Hq, D, dtype=dt), normal(g, T, Hk, D, dtype=dt), normal(g, T, Hk, D, dtype=dt), 0


def table_of(rot, scaling):
    t = torch.empty(max(1, rot // 2), dtype=torch.int64, device="cuda")
    moe.moe_rope_table(moe.MoERopeFreq.make(rot=rot, **scaling), t)
    return t


@pytest.mark.parametrize("far", [100, 1 << 20, 2 ** 31 - 5000])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,first,layout,dt,scaling", CASES)
def test_rope_and_backward(T, Hq, Hk, D, rot, first, layout, dt, scaling, packed, far):
    q, k, v, ld = inputs(T, Hq, Hk, D, dt, packed)
    pos = (torch.arange(T, device="cuda") + far - 50).to(torch.int32)
    pos[0] = -far  # negative positions turn the other way
    m = 1.0 if scaling < 2 else 0.1 * math.log(40.0) + 1
    cfg = moe.MoERopeConfig.make(T=T, Hq=Hq, Hk=Hk, D=D, rot=rot, first=first, layout=layout, act_dtype=CODE[dt], magnitude=m,
                                 ld_q=ld, ld_k=ld, ld_v=ld)
    table = table_of(rot, SCALINGS[scaling])
    freq = frequencies(rot, **SCALINGS[scaling])
    qo, ko, vo = (poisoned(T, H, D, dtype=dt) for H in (Hq, Hk, Hk))
    moe.moe_rope(cfg, q, k, v, pos, None, table, qo, ko, vo)
    for got, x in ((qo, q), (ko, k)):
        want, bound = turned(x, pos, freq, first, layout, m, 1.0)
        if got.numel():
            within(got, want, bound)
    assert torch.equal(vo, v)
    # without v, in place, and the same bits
    q2, k2, _, _ = inputs(T, Hq, Hk, D, dt, packed)
    row = moe.MoERopeConfig.make(**{**cfg.as_dict(), "ld_q_out": ld, "ld_k_out": ld})
    moe.moe_rope(row, q2, k2, None, pos, None, table, q2, k2, None)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    # backward: by minus the angle; into the projection's rows, the value heads left alone
    gq, gk, gv, _ = inputs(T, Hq, Hk, D, dt, packed, seed=1)
    dq, dk, dv, _ = inputs(T, Hq, Hk, D, dt, packed, seed=2)
    dv0 = dv.clone()
    gqc, gkc = gq.contiguous(), gk.contiguous()
    moe.moe_rope_backward(cfg, gqc, gkc, pos, table, dq, dk)
    for got, x in ((dq, gqc), (dk, gkc)):
        want, bound = turned(x, pos, freq, first, layout, m, -1.0)
        if got.numel():
            within(got, want, bound)
    assert torch.equal(dv, dv0)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,Hk,D,rot", [(1, 8, 128, 128), (70, 2, 50, 20), (999, 1, 192, 64)])
def test_rope_into_a_cache(T, Hk, D, rot, dt):
    Hq, rows = 2 * Hk, T + 37
    q, k, v, ld = inputs(T, Hq, Hk, D, dt, True)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    slot = torch.randperm(rows, device="cuda", generator=gen(5))[:T].to(torch.int32)
    cfg = moe.MoERopeConfig.make(T=T, Hq=Hq, Hk=Hk, D=D, rot=rot, act_dtype=CODE[dt], slots=rows, ld_q=ld, ld_k=ld, ld_v=ld)
    table, ws = table_of(rot, {}), workspace(moe.WORKSPACE_HEAD)
    qo, ko = poisoned(T, Hq, D, dtype=dt), poisoned(T, Hk, D, dtype=dt)
    moe.moe_rope(cfg, q, k, None, pos, None, table, qo, ko, None)
    kc, vc = (torch.full((rows, Hk, D), 7.0, device="cuda", dtype=dt) for _ in range(2))
    q2 = poisoned(T, Hq, D, dtype=dt)
    moe.moe_rope(cfg, q, k, v, pos, slot, table, q2, kc, vc, ws)
    wantk, wantv = torch.full_like(kc, 7.0), torch.full_like(vc, 7.0)
    wantk[slot.long()], wantv[slot.long()] = ko, v
    assert torch.equal(kc, wantk) and torch.equal(vc, wantv) and torch.equal(q2, qo)
    assert moe.moe_read_status(ws) == moe.MOE_OK
    # a padded token is not stored, its q is rotated all the same
    slot2 = slot.clone()
    slot2[0] = -1
    kc.fill_(7.0), vc.fill_(7.0)
    moe.moe_rope(cfg, q, k, v, pos, slot2, table, q2, kc, vc, ws)
    wantk[slot[0]] = wantv[slot[0]] = 7.0
    assert torch.equal(kc, wantk) and torch.equal(vc, wantv) and torch.equal(q2, qo)
    assert moe.moe_read_status(ws) == moe.MOE_OK
    # a slot behind the cache is not stored either, and is reported
    slot2[0] = rows
    moe.moe_rope(cfg, q, k, v, pos, slot2, table, q2, kc, vc, ws)
    assert torch.equal(kc, wantk) and torch.equal(vc, wantv) and torch.equal(q2, qo)
    assert moe.moe_read_status(ws) == moe.MOE_ERR_DEVICE_BAD_INPUT
    assert moe.moe_read_status(ws) == moe.MOE_OK


def test_rope_cache_rows_beyond_32_bits_of_elements():
    """The last rows of a cache of more than 2^32 elements."""
    Hk, D, rows = 2, 128, (1 << 32) // 256 + 300
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * rows * Hk * D * 2:
        pytest.skip("needs 18 GB")
    kc = torch.empty(rows, Hk, D, device="cuda", dtype=BF)
    kc[-64:] = 0
    kc[:64] = 0
    q, k, _, _ = inputs(4, 2, Hk, D, BF, False)
    slot = torch.tensor([rows - 1, rows - 3, rows - 2, 5], device="cuda", dtype=torch.int32)
    cfg = moe.MoERopeConfig.make(T=4, Hq=2, Hk=Hk, D=D, slots=rows)
    pos, ko, qo = torch.arange(4, device="cuda", dtype=torch.int32), torch.empty_like(k), torch.empty_like(q)
    table, ws = table_of(D, {}), workspace(moe.WORKSPACE_HEAD)
    moe.moe_rope(cfg, q, k, None, pos, None, table, qo, ko, None)
    moe.moe_rope(cfg, q, k, None, pos, slot, table, qo, kc, None, ws)
    assert torch.equal(kc[slot.long()], ko)
    assert not kc[-64:-3].any() and not kc[:5].any() and not kc[6:64].any()
    assert moe.moe_read_status(ws) == moe.MOE_OK


def test_rope_by_differences():
    """The backward is the transpose of the forward: <rope(x), g> differentiated by x, channel by channel."""
    T, D = 3, 10
    x, g = normal(gen(1), T, 1, D), normal(gen(2), T, 1, D)
    cfg = moe.MoERopeConfig.make(T=T, Hq=1, Hk=0, D=D, rot=6, first=2, act_dtype=moe.F32, magnitude=1.25)
    pos = torch.tensor([0, 3, 70000], device="cuda", dtype=torch.int32)
    table, out, dx = table_of(6, {}), torch.empty_like(x), torch.empty_like(x)
    moe.moe_rope_backward(cfg, g, None, pos, table, dx, None)
    for c in range(D):
        hi, lo = x.clone(), x.clone()
        hi[..., c] += 0.5
        lo[..., c] -= 0.5
        moe.moe_rope(cfg, hi, None, None, pos, None, table, out, None, None)
        up = (out.double() * g.double()).sum((1, 2))
        moe.moe_rope(cfg, lo, None, None, pos, None, table, out, None, None)
        slope = up - (out.double() * g.double()).sum((1, 2))
        # linear: differences are exact but for the roundings of 2 x 10 products of size up to ~4 each
        assert (slope - dx[:, 0, c].double()).abs().max() < 40 * 8 * U * 4


@pytest.mark.parametrize("rot,D,layout,dt", [(64, 192, moe.ROPE_INTERLEAVED, BF), (128, 128, moe.ROPE_HALF, FP)])
def test_frequencies_of_the_callers_own(rot, D, layout, dt):
    """A table that the caller fills: YaRN mixed linearly in the pair's index, which is not moe_rope_table's."""
    base, L, factor, fast, slow = 10000.0, 4096, 40.0, 32.0, 1.0

    def at(turns):
        return rot * math.log(L / (2 * math.pi * turns)) / (2 * math.log(base))

    lo, hi = max(0, math.floor(at(fast))), min(rot // 2 - 1, math.ceil(at(slow)))
    ramp = [min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(rot // 2)]
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]
    f = [v * (1 - r) + v / factor * r for v, r in zip(plain, ramp)]
    entries = [round(v / (2 * math.pi) % 1 * 2.0 ** 64) % 2 ** 64 for v in f]
    table = torch.tensor([e - 2 ** 64 if e >= 2 ** 63 else e for e in entries], dtype=torch.int64, device="cuda")
    freq = torch.tensor(f, dtype=torch.float64, device="cuda")
    ratio = freq / frequencies(rot, **YARN)
    assert ratio.max() > 4 and (ratio > 1.05).sum() > rot // 8  # other frequencies than the listed scaling's
    T, m = 300, 0.1 * math.log(factor) + 1
    q, k, v, ld = inputs(T, 4, 2, D, dt, True)
    pos = (torch.arange(T, device="cuda") * 541).to(torch.int32)
    cfg = moe.MoERopeConfig.make(T=T, Hq=4, Hk=2, D=D, rot=rot, first=D - rot, layout=layout, act_dtype=CODE[dt], magnitude=m,
                                 ld_q=ld, ld_k=ld, ld_v=ld)
    qo, ko = poisoned(T, 4, D, dtype=dt), poisoned(T, 2, D, dtype=dt)
    moe.moe_rope(cfg, q, k, None, pos, None, table, qo, ko, None)
    for got, x in ((qo, q), (ko, k)):
        want, bound = turned(x, pos, freq, D - rot, layout, m, 1.0)
        within(got, want, bound)
