"""Attention and its gradients against the formulas in 64 bits, with bounds per element on what the
documented arithmetic may lose."""
import math

import pytest
import torch

import token_routing_expert_router_gb300 as moe
from test_step_gpu import BF, CODE, FP, HALF, U, gen, normal, poisoned, workspace
from test_step_gpu import within as within_all

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(lib):
    pass


# The exponentials and the packed fp32 operations flush results below fp32's smallest normal value,
# 2^-126, to zero: a probability is off by that much beside its relative error, and so is a product of it.
FTZ = 2.0 ** -126


def within(got, want, bound):
    if got.numel():
        within_all(got, want, bound)


class Batch:
    """q, k, v and where the sequences are. lens: (query rows, keys) of every sequence; place:
    "self" (keys beside the queries), "cache" (a region for each, with NaN around), "shared" (all
    on the same keys). NaN in every row that is in no sequence."""

    def __init__(self, lens, Hq, Hkv, D, dt, causal=1, place="self", packed=False, tail=3, scale=None, sharp=1.0, max_q=None,
                 seed=0):
        g = gen(seed)
        self.lens, self.Hq, self.Hkv, self.D, self.dt, self.causal = lens, Hq, Hkv, D, dt, causal
        B = len(lens)
        self.q_at, at = [], 0
        for n, _ in lens:
            self.q_at.append(at)
            at += n
        T = self.used = at
        self.Tq = T + tail
        self.q_start = torch.tensor(self.q_at + [T], dtype=torch.int32, device="cuda")
        if place == "self":
            assert all(n == m for n, m in lens)
            self.k_at, self.k_start, self.k_len, self.Tk = self.q_at, None, None, self.Tq
        else:
            if place == "cache":
                region = max([m for _, m in lens] + [0]) + 5
                self.k_at, self.Tk = [b * region + 2 for b in range(B)], B * region + 4
            else:
                self.k_at, self.Tk = [1] * B, max(m for _, m in lens) + 4
            self.k_start = torch.tensor(self.k_at, dtype=torch.int32, device="cuda")
            self.k_len = torch.tensor([m for _, m in lens], dtype=torch.int32, device="cuda")
        if packed:
            assert place == "self"
            row = poisoned(self.Tq, Hq + 2 * Hkv, D, dtype=dt)
            row[:T] = normal(g, T, Hq + 2 * Hkv, D, dtype=dt)
            row[:T, :Hq] *= sharp
            self.q, self.k, self.v = row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:]
        else:
            self.q, self.k, self.v = (poisoned(r, h, D, dtype=dt) for r, h in ((self.Tq, Hq), (self.Tk, Hkv), (self.Tk, Hkv)))
            self.q[:T] = normal(g, T, Hq, D, dtype=dt, std=sharp)
            for (_, m), a in zip(lens, self.k_at):
                self.k[a:a + m], self.v[a:a + m] = normal(g, m, Hkv, D, dtype=dt), normal(g, m, Hkv, D, dtype=dt)
        self.do = poisoned(self.Tq, Hq, D, dtype=dt)
        self.do[:T] = normal(g, T, Hq, D, dtype=dt)
        self.scale = 1 / math.sqrt(D) if scale is None else scale
        ld = (Hq + 2 * Hkv) * D if packed else 0
        self.packed = packed
        self.cfg = moe.MoEAttnConfig.make(Tq=self.Tq, Tk=self.Tk, B=B, Hq=Hq, Hkv=Hkv, D=D, causal=causal, act_dtype=CODE[dt],
                                          max_q=max([n for n, _ in lens] + [0]) if max_q is None else max_q,
                                          scale=self.scale, ld_q=ld, ld_k=ld, ld_v=ld)
        self.scale = self.cfg.scale  # as fp32 has it
        self.ws = workspace(moe.moe_attn_workspace_size(self.cfg))
        self.bws = workspace(moe.moe_attn_backward_workspace_size(self.cfg))

    def forward(self, stream=None):
        o, lse = torch.full((self.Tq, self.Hq, self.D), 7.0, dtype=self.dt, device="cuda"), torch.full((self.Hq, self.Tq), 7.0,
                                                                                                  device="cuda")
        moe.moe_attn(self.cfg, self.q, self.k, self.v, self.q_start, self.k_start, self.k_len, o, lse, self.ws, stream=stream)
        return o, lse

    def grads(self):
        """Buffers for the gradients, laid out as q, k and v, full of sevens."""
        if self.packed:
            row = torch.full((self.Tq, self.Hq + 2 * self.Hkv, self.D), 7.0, dtype=self.dt, device="cuda")
            return row[:, :self.Hq], row[:, self.Hq:self.Hq + self.Hkv], row[:, self.Hq + self.Hkv:]
        return tuple(torch.full_like(x, 7.0) for x in (self.q, self.k, self.v))

    def backward(self, o, lse, out=None):
        out = self.grads() if out is None else out
        moe.moe_attn_backward(self.cfg, self.q, self.k, self.v, self.q_start, self.k_start, self.k_len, o, lse, self.do, *out,
                              self.bws)
        return out

    def parts(self):
        """(b, query rows, key rows, mask of visible pairs) of every sequence."""
        for b, (n, m) in enumerate(self.lens):
            i, j = torch.arange(n, device="cuda")[:, None], torch.arange(m, device="cuda")[None, :]
            seen = (j <= i + m - n) if self.causal else torch.ones(n, m, dtype=torch.bool, device="cuda")
            yield b, slice(self.q_at[b], self.q_at[b] + n), slice(self.k_at[b], self.k_at[b] + m), seen

    def check_forward(self, o, lse):
        """Against the formula. With e_s the error of a score, a probability's is e_p = p (e_s + ...);
        o and lse follow by the sums of them."""
        assert (o[self.used:] == 7).all() and (lse[:, self.used:] == 7).all()
        G, bf = self.Hq // self.Hkv, self.dt == BF
        for b, rq, rk, seen in self.parts():
            n, m = seen.shape
            for h in range(self.Hq):
                q, k, v = self.q[rq, h].double(), self.k[rk, h // G].double(), self.v[rk, h // G].double()
                s, want, wlse, p, ep, el = self._scores(q, k, v, seen)
                empty = ~seen.any(1)
                got = lse[h, rq]
                assert torch.equal(got == -math.inf, empty)
                within(got[~empty], wlse[~empty], el[~empty])
                bound = self._o_bound(p, ep, el, v, want)
                assert not o[rq, h][empty].any()
                within(o[rq, h], want, bound)

    def _scores(self, q, k, v, seen):
        s = (q @ k.t()) * self.scale
        s = s.masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(s, 1) if s.shape[1] else torch.full((s.shape[0],), -math.inf, dtype=torch.float64, device="cuda")
        some = lse > -math.inf
        p = torch.where(some[:, None], (s - lse[:, None]).exp(), 0.0).nan_to_num(0.0)
        o = p @ v
        # D fp32 products summed in any order, a tensor core's truncating additions counted twice
        es = 2 * (self.D + 8) * U * self.scale * (q.abs() @ k.abs().t())
        # the exponent in base 2 and the exponential: 2^-22 of it, the argument's own roundings
        z = torch.where(seen, s, 0.0).abs() + torch.where(some, lse, 0.0).abs()[:, None] + 16
        ep = torch.where(seen, es + 8 * U * z + 2.0 ** -21, 0.0)  # relative
        m = s.shape[1]
        el = (p * ep).sum(1) + (2 * m + 32) * U + 8 * U * torch.where(some, lse, 0.0).abs()
        return s, o, lse, p, ep, el

    def _o_bound(self, p, ep, el, v, want):
        half = HALF[BF] if self.dt == BF else 0.0
        mag = p @ v.abs()
        lost = (p * (ep + half) + FTZ) @ v.abs() + (el[:, None] + (2 * p.shape[1] + 64) * U) * mag
        return lost + HALF[self.dt] * (want.abs() + lost) + FTZ

    def check_backward(self, dq, dk, dv):
        outside = [torch.ones(self.Tq if i == 0 else self.Tk, dtype=torch.bool, device="cuda") for i in range(3)]
        G = self.Hq // self.Hkv
        half = HALF[BF] if self.dt == BF else 0.0
        for b, rq, rk, seen in self.parts():
            n, m = seen.shape
            outside[0][rq] = False
            outside[1][rk] = False
            outside[2][rk] = False
            acc = 2 * U * (max(n * G, m) + 64)
            for hk in range(self.Hkv):
                k, v = self.k[rk, hk].double(), self.v[rk, hk].double()
                zero = torch.zeros_like(k)
                wk, wv, bk, bv = zero.clone(), zero.clone(), zero.clone(), zero.clone()
                for h in range(hk * G, (hk + 1) * G):
                    q, do = self.q[rq, h].double(), self.do[rq, h].double()
                    s, o, lse, p, ep, el = self._scores(q, k, v, seen)
                    eo = self._o_bound(p, ep, el, v, o)
                    ep = ep + el[:, None] + 2.0 ** -21  # exp(s - lse), lse from the forward
                    dp, delta = do @ v.t(), (do * o).sum(1, keepdim=True)
                    edp = 2 * (self.D + 8) * U * (do.abs() @ v.abs().t())
                    ed = (do.abs() * eo).sum(1, keepdim=True) + 2 * (self.D + 8) * U * (do * o).abs().sum(1, keepdim=True)
                    ds = p * (dp - delta)
                    first = ed
                    if self.dt == BF:
                        # the first delta is put right by the sum of a row's ds: what remains is the error of
                        # the sum of p dp, and nothing of o's rounding
                        ed = (p * (ep * dp.abs() + edp)).sum(1, keepdim=True) + acc * (p * dp.abs()).sum(1, keepdim=True)
                    eds = p * (edp + ed) + ds.abs() * (ep + half + 4 * U) + p * 4 * U * (dp.abs() + delta.abs())
                    # flushed: p (times dp - delta), and ds itself
                    eds = eds * (1 + half) + FTZ * (dp.abs() + delta.abs() + 1)
                    want = self.scale * ds @ k
                    # dq's own ds have the first delta, and are rounded with it; so is the mean key that takes it back
                    lost = self.scale * ((eds + acc * ds.abs() + 2 * (half + acc) * p * first) @ k.abs())
                    within(dq[rq, h], want, lost + HALF[self.dt] * (want.abs() + lost) + 4 * U * want.abs() + FTZ)
                    wv += p.t() @ do
                    bv += (p * (ep + half + acc) + FTZ).t() @ do.abs()
                    wk += self.scale * ds.t() @ q
                    bk += self.scale * (eds + acc * ds.abs()).t() @ q.abs()
                # fp32 scales q by the scores' scale first: one rounding more
                bk = bk + 4 * U * (bk + wk.abs())
                within(dk[rk, hk], wk, bk + HALF[self.dt] * (wk.abs() + bk) + FTZ)
                within(dv[rk, hk], wv, bv + HALF[self.dt] * (wv.abs() + bv) + FTZ)
        for rows, g in zip(outside, (dq, dk, dv)):
            assert (g[rows] == 7).all()

    def check_status(self, want=moe.MOE_OK):
        assert moe.moe_read_status(self.ws) == want


EDGES = [1, 0, 63, 64, 65, 127, 128, 129, 0, 200, 2]
same = lambda ns: [(n, n) for n in ns]  # noqa: E731

SELF = [
    # query rows (= keys) of the sequences, Hq, Hkv, D, dtype
    ([1], 1, 1, 1, FP), ([1], 2, 1, 8, BF), (EDGES, 4, 2, 64, BF), (EDGES, 4, 1, 128, BF), (EDGES, 2, 2, 50, FP),
    (EDGES, 3, 1, 36, BF), ([300], 6, 2, 80, BF), ([300], 2, 2, 128, FP), ([257, 255], 8, 1, 32, BF), ([513], 2, 1, 24, BF),
    ([700, 3, 401], 4, 4, 96, BF), ([1100], 2, 1, 128, BF), ([1100], 1, 1, 64, BF), ([5] * 300, 1, 1, 16, BF), ([], 2, 2, 64, BF),
    ([0, 0], 2, 2, 64, BF), ([384, 640], 2, 2, 120, BF), ([260], 2, 2, 127, BF), ([2] * 600 + [150], 1, 1, 8, FP)]


@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,D,dt", SELF)
def test_packed_sequences(lens, Hq, Hkv, D, dt, packed, causal):
    b = Batch(same(lens), Hq, Hkv, D, dt, causal=causal, packed=packed, seed=len(lens))
    o, lse = b.forward()
    b.check_forward(o, lse)
    grads = b.backward(o, lse)
    b.check_backward(*grads)
    b.check_status()
    assert moe.moe_read_status(b.bws) == moe.MOE_OK
    # the same bits again
    o2, lse2 = b.forward()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for x, y in zip(grads, b.backward(o, lse)):
        assert torch.equal(x, y)


OVER = [
    # (query rows, keys) of the sequences, Hq, Hkv, D, dtype
    ([(1, 700)], 8, 2, 128, BF), ([(1, 1)], 4, 1, 64, BF), ([(1, 0), (1, 5), (1, 64), (1, 2000), (1, 129)], 16, 2, 128, BF),
    ([(1, 33), (1, 0), (1, 900)], 4, 4, 64, FP), ([(1, 3000)] * 3, 32, 2, 128, BF), ([(1, 500), (1, 77)], 7, 1, 80, BF),
    ([(4, 600), (1, 9), (3, 64), (0, 50), (2, 1)], 8, 2, 128, BF), ([(5, 600), (2, 300)], 12, 1, 64, BF),
    ([(4, 2), (2, 1), (1, 0)], 4, 2, 64, BF), ([(200, 130), (64, 64), (10, 300)], 4, 2, 64, BF),
    ([(200, 130), (130, 0), (10, 300)], 4, 2, 128, BF), ([(150, 20), (7, 300), (3, 0)], 2, 1, 40, FP),
    ([(130, 1000), (300, 301), (1, 800)], 4, 2, 128, BF), ([(16, 400), (0, 9)], 2, 1, 36, BF), ([(2, 130)] * 40, 2, 2, 64, BF),
    ([(1, 40000)], 2, 1, 128, BF), ([(1, 9000), (1, 100)], 2, 2, 128, FP), ([(6, 700)], 128, 1, 64, BF),
    ([(1, 1 + 17 * i) for i in range(70)], 4, 1, 128, BF), ([(1, 260)] * 300, 2, 1, 32, BF), ([(8, 1111)] * 2, 6, 3, 104, BF)]


@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("place", ["cache", "shared"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,dt", OVER)
def test_over_a_cache(lens, Hq, Hkv, D, dt, place, causal):
    b = Batch(lens, Hq, Hkv, D, dt, causal=causal, place=place, seed=len(lens) + D)
    o, lse = b.forward()
    b.check_forward(o, lse)
    b.check_status()
    o2, lse2 = b.forward()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if place == "cache" and sum(n * m for n, m in lens) * Hq < 10 ** 7:
        grads = b.backward(o, lse)
        b.check_backward(*grads)
        assert moe.moe_read_status(b.bws) == moe.MOE_OK
        for x, y in zip(grads, b.backward(o, lse)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dt,D,n", [(BF, 128, 300), (BF, 64, 200), (FP, 64, 130), (BF, 36, 130)])
@pytest.mark.parametrize("m", [None, 2000])
def test_sharp_and_flat_scores(dt, D, n, m):
    """Rows whose maximum grows from tile to tile by hundreds, and rows that are all alike."""
    lens = [(n, n)] if m is None else [(2, m)]
    for sharp, scale in ((40.0, 1.0), (1e-3, 1e-3)):
        b = Batch(lens, 4, 2, D, dt, place="self" if m is None else "cache", sharp=sharp, scale=scale, seed=3)
        if sharp > 1:  # keys that lean towards the last queries, more and more
            for (_, mm), a in zip(b.lens, b.k_at):
                lean = b.q[b.used - 1, ::2].float() / (sharp * math.sqrt(D))
                ramp = torch.linspace(0, 3, mm, device="cuda")[:, None, None]
                b.k[a:a + mm] = (b.k[a:a + mm].float() * 0.2 + ramp * lean).to(dt)
        o, lse = b.forward()
        # scores of some hundreds are off by some 1e-4, which the bounds hold
        b.check_forward(o, lse)
        if m is None:
            b.check_backward(*b.backward(o, lse))


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("lens", [[(1, 300), (1, 40)], [(200, 300), (64, 64)]])
def test_sequences_out_of_range(dt, lens):
    """Rows or keys that are not there: reported, and nothing of them read or written."""
    b = Batch(lens, 4, 2, 64, dt, place="cache")
    o, lse = b.forward()
    for name, at, value, rows, keys in (("q_start", 0, -1, False, None), ("q_start", 2, b.Tq + 1, False, None),
                                        ("q_start", 1, -5, False, None), ("k_start", 1, b.Tk, True, False),
                                        ("k_start", 1, -3, True, False), ("k_len", 1, b.Tk, True, False),
                                        ("k_len", 1, -1, True, False)):
        t = getattr(b, name)
        old = t[at].clone()
        t[at] = value
        o2, lse2 = b.forward()
        b.check_status(moe.MOE_ERR_DEVICE_BAD_INPUT)
        b.check_status()
        if keys is False:  # the sequence has no keys
            r = slice(b.q_at[1], b.q_at[1] + lens[1][0])
            assert not o2[r].any() and (lse2[:, r] == -math.inf).all()
            assert torch.equal(o2[:b.q_at[1]], o[:b.q_at[1]])
        grads = b.backward(o, lse)
        assert moe.moe_read_status(b.bws) == moe.MOE_ERR_DEVICE_BAD_INPUT
        assert all((x[b.used if i == 0 else b.Tk - 2:] == 7).all() for i, x in enumerate(grads))
        t[at] = old
    # more query rows than announced
    cfg = moe.MoEAttnConfig.make(**{**b.cfg.as_dict(), "max_q": max(n for n, _ in lens) - 1 or 1})
    if cfg.max_q < max(n for n, _ in lens):
        b.cfg = cfg
        o2, _ = b.forward()
        b.check_status(moe.MOE_ERR_DEVICE_BAD_INPUT)
        assert (o2[:lens[0][0]] == 7).all()
    b = Batch(lens, 4, 2, 64, dt, place="shared")  # the backward would write the keys twice
    o, lse = b.forward()
    b.check_status()
    b.backward(o, lse)
    assert moe.moe_read_status(b.bws) == moe.MOE_ERR_DEVICE_BAD_INPUT


def test_gradients_by_differences():
    """The 64-bit formulas behind the bounds, and the kernels, against central differences."""
    b = Batch([(5, 9), (3, 2)], 2, 1, 8, FP, place="cache", seed=11)
    o, lse = b.forward()
    grads = b.backward(o, lse)

    def total(q, k, v):
        out = 0.0
        for _, rq, rk, seen in b.parts():
            for h in range(2):
                s = (q[rq, h] @ k[rk, 0].t() * b.scale).masked_fill(~seen, -1e30)
                p = torch.softmax(s, 1) * seen
                out = out + (p @ v[rk, 0] * b.do[rq, h].double()).sum()
        return out

    x = [t.double().nan_to_num(0.0) for t in (b.q, b.k, b.v)]
    g, h = gen(4), 1e-5
    for i in range(3):
        d = normal(g, *x[i].shape).double()
        hi, lo = list(x), list(x)
        hi[i], lo[i] = x[i] + h * d, x[i] - h * d
        slope = (total(*hi) - total(*lo)) / (2 * h)
        inside = torch.where(grads[i] == 7, 0.0, grads[i].double())
        # differences lose h^2 times a third derivative of order 10; fp32 gradients 1e-5 of some dozens
        assert abs(slope - (inside * d).sum()) < 1e-3


def test_positions_cache_and_attention_together():
    """A prompt and ten tokens behind it, as a server runs them: rotated into a cache of pages that are
    slots, one token a step - against the attention over the whole packed text at once."""
    n, new, Hq, Hkv, D = 70, 10, 8, 2, 64
    T, g = n + new, gen(21)
    row = normal(g, T, Hq + 2 * Hkv, D, dtype=BF)
    q, k, v = row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:]
    table = torch.empty(D // 2, dtype=torch.int64, device="cuda")
    moe.moe_rope_table(moe.MoERopeFreq.make(rot=D), table)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    ld = (Hq + 2 * Hkv) * D

    def turn(lo, hi, k_out, v_out, slot, slots, ws):
        cfg = moe.MoERopeConfig.make(T=hi - lo, Hq=Hq, Hk=Hkv, D=D, slots=slots, ld_q=ld, ld_k=ld, ld_v=ld)
        out = torch.empty(hi - lo, Hq, D, device="cuda", dtype=BF)
        moe.moe_rope(cfg, q[lo:hi], k[lo:hi], v[lo:hi], pos[lo:hi].clone(), slot, table, out, k_out, v_out, ws)
        return out

    # at once
    kk, vv = torch.empty(T, Hkv, D, device="cuda", dtype=BF), torch.empty(T, Hkv, D, device="cuda", dtype=BF)
    qq = turn(0, T, kk, vv, None, 0, None)
    cfg = moe.MoEAttnConfig.make(Tq=T, Tk=T, B=1, Hq=Hq, Hkv=Hkv, D=D)
    ws = workspace(moe.moe_attn_workspace_size(cfg))
    start = torch.tensor([0, T], device="cuda", dtype=torch.int32)
    o, lse = torch.empty_like(qq), torch.empty(Hq, T, device="cuda")
    moe.moe_attn(cfg, qq, kk, vv, start, None, None, o, lse, ws)
    # step by step: the text is the second of two slots regions
    slots = 200
    kc, vc = (poisoned(slots, Hkv, D, dtype=BF) for _ in range(2))
    first = 100
    for lo, hi in [(0, n)] + [(i, i + 1) for i in range(n, T)]:
        slot = (torch.arange(lo, hi, device="cuda") + first).to(torch.int32)
        qs = turn(lo, hi, kc, vc, slot, slots, ws)
        c = moe.MoEAttnConfig.make(Tq=hi - lo, Tk=slots, B=1, Hq=Hq, Hkv=Hkv, D=D, max_q=hi - lo)
        assert moe.moe_attn_workspace_size(c) <= ws.numel()
        os_, ls = torch.empty_like(qs), torch.empty(Hq, hi - lo, device="cuda")
        moe.moe_attn(c, qs, kc, vc, torch.tensor([0, hi - lo], device="cuda", dtype=torch.int32),
                     torch.tensor([first], device="cuda", dtype=torch.int32),
                     torch.tensor([hi], device="cuda", dtype=torch.int32), os_, ls, ws)
        assert torch.equal(qs, qq[lo:hi])
        # the same products and sums in another order: p rounded against another maximum, 2^-8 each
        within(os_, o[lo:hi].double(), 2 * HALF[BF] * o[lo:hi].double().abs() + 2 * HALF[BF] * vv[:hi].double().abs().max())
        within(ls, lse[:, lo:hi].double(), 2.0 ** -18 * (1 + lse[:, lo:hi].double().abs()))
    assert torch.equal(kc[first:first + T], kk) and torch.equal(vc[first:first + T], vv)
    assert moe.moe_read_status(ws) == moe.MOE_OK


RUNS = [([(300, 300), (77, 77), (129, 129)], "self", 8, 2, 64, BF), ([(1, 500), (1, 900), (1, 3)], "cache", 8, 2, 128, BF),
        ([(300, 300), (20, 20)], "self", 4, 2, 64, FP), ([(1, 500), (1, 900)], "cache", 8, 2, 128, FP)]


@pytest.mark.parametrize("lens,place,Hq,Hkv,D,dt", RUNS)
def test_captured_graphs_that_share_a_workspace(lens, place, Hq, Hkv, D, dt):
    """Two graphs over the same workspace, replayed in turn on another stream, give the bits of direct calls."""
    a, b = (Batch(lens, Hq, Hkv, D, dt, place=place, seed=s) for s in (1, 2))
    b.ws, b.bws = a.ws, a.bws
    want = [(x.forward(), x.backward(*x.forward())) for x in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for x in (a, b):
            graph = torch.cuda.CUDAGraph()
            o, lse = torch.empty_like(want[0][0][0]), torch.empty_like(want[0][0][1])
            grads = x.grads()
            side.synchronize()
            with torch.cuda.graph(graph, stream=side):
                moe.moe_attn(x.cfg, x.q, x.k, x.v, x.q_start, x.k_start, x.k_len, o, lse, x.ws)
                x.backward(o, lse, grads)
            graphs.append(graph)
            outs.append((o, lse, grads))
        for _ in range(3):
            for (o, lse, grads), graph in zip(outs, graphs):
                o.fill_(7.0), lse.fill_(7.0)
                for t in grads:
                    t.fill_(7.0)
                graph.replay()
    torch.cuda.synchronize()
    for (fwd, bwd), (o, lse, grads) in zip(want, outs):
        assert torch.equal(o, fwd[0]) and torch.equal(lse, fwd[1])
        assert all(torch.equal(x, y) for x, y in zip(grads, bwd))
    a.check_status()


@pytest.mark.parametrize("lens,place,Hq,Hkv,D,dt", RUNS)
def test_calls_at_once_on_two_streams(lens, place, Hq, Hkv, D, dt):
    """Calls that overlap, each with a stream and a workspace of its own."""
    parts = [Batch(lens, Hq, Hkv, D, dt, place=place, seed=s) for s in (1, 2, 3)]
    want = [(x.forward(), x.backward(*x.forward())) for x in parts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in parts]
    got = [None] * len(parts)
    for _ in range(5):
        for i, (x, s) in enumerate(zip(parts, streams)):
            with torch.cuda.stream(s):
                o, lse = x.forward()
                got[i] = (o, lse, x.backward(o, lse))
    torch.cuda.synchronize()
    for (fwd, bwd), (o, lse, grads) in zip(want, got):
        assert torch.equal(o, fwd[0]) and torch.equal(lse, fwd[1])
        assert all(torch.equal(x, y) for x, y in zip(grads, bwd))


@pytest.mark.parametrize("D,dt", [(64, BF), (128, BF), (128, FP)])
def test_long_offsets(D, dt):
    """Keys at the far end of a cache of more than 2^31 elements: the bits of the same keys in a small one."""
    Hkv, m = 2, 700
    rows = (1 << 31) // (Hkv * D) + 5000
    size = rows * Hkv * D * (2 if dt == BF else 4)
    if torch.cuda.mem_get_info()[0] < 3 * size:
        pytest.skip("needs 3 times the cache")
    b = Batch([(1, m), (3, m - 9)], 4, Hkv, D, dt, place="cache", seed=5)
    o, lse = b.forward()
    far = [torch.empty(rows, Hkv, D, device="cuda", dtype=dt) for _ in range(2)]
    at = rows - b.Tk
    far[0][at:], far[1][at:] = b.k, b.v
    cfg = moe.MoEAttnConfig.make(**{**b.cfg.as_dict(), "Tk": rows})
    o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    moe.moe_attn(cfg, b.q, far[0], far[1], b.q_start, b.k_start + at, b.k_len, o2, lse2, b.ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    b.check_status()


def test_many_sequences():
    """More sequences than threads, empty ones among them."""
    lens = [(i % 3, i % 3) for i in range(3000)] + [(200, 200)]
    for dt in (BF, FP):
        b = Batch(lens, 2, 1, 16, dt, place="self", seed=9)
        o, lse = b.forward()
        grads = b.backward(o, lse)
        b.check_status()
        # the last sequence by the formulas, the sequences of one row: one key, its value
        alone = Batch([(200, 200)], 2, 1, 16, dt, place="self", seed=9)
        at = slice(b.used - 200, b.used)
        for name in ("q", "k", "v", "do"):
            getattr(alone, name)[:200] = getattr(b, name)[at]
        o1, lse1 = torch.full((alone.Tq, 2, 16), 7.0, dtype=dt, device="cuda"), torch.full((2, alone.Tq), 7.0, device="cuda")
        o1[:200], lse1[:, :200] = o[at], lse[:, at]
        alone.check_forward(o1, lse1)
        mine = alone.grads()
        for x, y in zip(mine, grads):
            x[:200] = y[at]
        alone.check_backward(*mine)
        ones = torch.tensor([b.q_at[i] for i, (n, _) in enumerate(lens) if n == 1], device="cuda")
        assert torch.equal(o[ones], b.v[ones].expand(-1, 2, 16))


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_no_keys_at_all_and_no_queries(dt, n):
    """Tk = 0: zeros, -inf and zero gradients; Tq = 0: zero gradients of the keys."""
    Hq, Hkv, D = 4, 2, 64
    code, i32 = CODE[dt], dict(device="cuda", dtype=torch.int32)
    q, none = normal(gen(1), n, Hq, D, dtype=dt), torch.empty(0, Hkv, D, device="cuda", dtype=dt)
    cfg = moe.MoEAttnConfig.make(Tq=n, Tk=0, B=1, Hq=Hq, Hkv=Hkv, D=D, act_dtype=code, max_q=n)
    ws = workspace(max(moe.moe_attn_workspace_size(cfg), moe.moe_attn_backward_workspace_size(cfg)))
    start, zero = torch.tensor([0, n], **i32), torch.zeros(1, **i32)
    o, lse, dq = poisoned(n, Hq, D, dtype=dt), poisoned(Hq, n, dtype=FP), poisoned(n, Hq, D, dtype=dt)
    moe.moe_attn(cfg, q, none, none, start, zero, zero, o, lse, ws)
    assert not o.any() and (lse == -math.inf).all()
    moe.moe_attn_backward(cfg, q, none, none, start, zero, zero, o, lse, q, dq, none, none, ws)
    assert not dq.any() and moe.moe_read_status(ws) == moe.MOE_OK
    # keys, but no queries
    k = normal(gen(2), n, Hkv, D, dtype=dt)
    nq = torch.empty(0, Hq, D, device="cuda", dtype=dt)
    cfg = moe.MoEAttnConfig.make(Tq=0, Tk=n, B=1, Hq=Hq, Hkv=Hkv, D=D, act_dtype=code)
    ws = workspace(max(moe.moe_attn_workspace_size(cfg), moe.moe_attn_backward_workspace_size(cfg)))
    dk, dv = poisoned(n, Hkv, D, dtype=dt), poisoned(n, Hkv, D, dtype=dt)
    nl, start = torch.empty(Hq, 0, device="cuda"), torch.zeros(2, **i32)
    length = torch.tensor([n], **i32)
    moe.moe_attn(cfg, nq, k, k, start, zero, length, nq, nl, ws)
    moe.moe_attn_backward(cfg, nq, k, k, start, zero, length, nq, nl, nq, nq, dk, dv, ws)
    assert not dk.any() and not dv.any() and moe.moe_read_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("dt,D", [(BF, 64), (FP, 32)])
def test_on_the_stream_that_is_given(dt, D):
    """stream= another than the current one: ordered on it, with tensors made on the current one."""
    b = Batch([(200, 200), (1, 1), (90, 90)], 4, 2, D, dt, seed=6)
    o, lse = b.forward()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, lse2 = b.forward(stream=side)  # the outputs are filled on the current stream first
    side.synchronize()
    torch.cuda.synchronize()
    moe.moe_attn(b.cfg, b.q, b.k, b.v, b.q_start, b.k_start, b.k_len, o2, lse2, b.ws, stream=side)
    side.synchronize()
    assert torch.equal(o[:b.used], o2[:b.used]) and torch.equal(lse[:, :b.used], lse2[:, :b.used])


def test_rows_of_two_shapes():
    """[T, heads, D] and [T, heads * D] name the same rows."""
    b = Batch([(130, 130)], 4, 2, 64, BF, seed=8)
    o, lse = b.forward()
    flat = lambda t: t.reshape(len(t), -1)  # noqa: E731
    o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    moe.moe_attn(b.cfg, flat(b.q), flat(b.k), flat(b.v), b.q_start, None, None, flat(o2), lse2, b.ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_sequence_does_not_see_its_neighbours():
    """NaN in one sequence's rows stays there: the others' bits are those without it."""
    for dt, D in ((BF, 128), (BF, 64), (BF, 36), (FP, 64)):
        b = Batch([(100, 100), (70, 70), (300, 300)], 4, 2, D, dt, seed=4)
        o, lse = b.forward()
        grads = b.backward(o, lse)
        for t in (b.q, b.k, b.v, b.do):
            t[100:170] = float("nan")
        o2, lse2 = b.forward()
        grads2 = b.backward(o2, lse2)
        for lo, hi in ((0, 100), (170, 470)):
            assert torch.equal(o[lo:hi], o2[lo:hi]) and torch.equal(lse[:, lo:hi], lse2[:, lo:hi])
            assert all(torch.equal(x[lo:hi], y[lo:hi]) for x, y in zip(grads, grads2))


@pytest.mark.parametrize("dt,D,n,m", [(BF, 128, 300, 300), (BF, 64, 1, 5000), (BF, 36, 70, 70), (FP, 64, 100, 100), (FP, 32, 1, 40),
                                      (FP, 32, 1, 5000)])
def test_nan_stays_visible(dt, D, n, m):
    """NaN in a query is NaN in its own outputs alone; NaN in a key that all see is NaN in all of its head's."""
    Hq, Hkv = 4, 2
    b = Batch([(n, m)], Hq, Hkv, D, dt, place="cache", seed=5)
    o, lse = b.forward()
    b.q[n - 1, 1] = float("nan")
    o2, lse2 = b.forward()
    assert o2[n - 1, 1].isnan().all() and lse2[1, n - 1].isnan()
    same = torch.ones(n, Hq, dtype=torch.bool, device="cuda")
    same[n - 1, 1] = False
    assert torch.equal(o[:n][same], o2[:n][same]) and torch.equal(lse.T[:n][same], lse2.T[:n][same])
    b.k[b.k_at[0], 1] = float("nan")
    o3, lse3 = b.forward()
    assert o3[:n, 2:].isnan().all() and lse3[2:, :n].isnan().all()


@pytest.mark.parametrize("dt,D,n,m", [(BF, 64, 1, 700), (BF, 64, 300, 700), (BF, 36, 70, 90), (FP, 32, 1, 700), (FP, 32, 100, 200)])
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** 100])
def test_the_smallest_and_largest_scale(dt, D, n, m, scale):
    """2^-100: all scores round to 0 against 1, o is the mean of v and lse the logarithm of the count.
    2^100: the largest score has the weight 1."""
    b = Batch([(n, m)], 2, 1, D, dt, causal=0, place="cache", scale=scale, seed=9)
    o, lse = b.forward()
    at = b.k_at[0]
    k, v = b.k[at:at + m, 0].double(), b.v[at:at + m, 0].double()
    for h in range(2):
        s = b.q[:n, h].double() @ k.T
        if scale < 1:
            want, want_lse = v.mean(0).expand(n, D), torch.full((n,), math.log(m), device="cuda", dtype=torch.float64)
        else:
            top, best = s.max(1)
            want, want_lse = v[best], top * scale
        # o: one rounding of its type, fp32 sums of m terms below 6 (2^-24 m of them at most); lse: as many roundings
        eps = torch.finfo(dt).eps / 2
        assert ((o[:n, h].double() - want).abs() <= eps * want.abs() + 2.0 ** -24 * m * 6).all()
        assert ((lse[h, :n].double() - want_lse).abs() <= 2.0 ** -24 * m * want_lse.abs()).all()


@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("dt,D,packed", [(FP, 20, False), (FP, 64, True), (FP, 98, False), (FP, 128, False), (BF, 20, True), (BF, 50, False),
                                         (BF, 100, False)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (6, 1)])
def test_fma_units_with_many_and_few_heads(dt, D, packed, Hq, Hkv, causal):
    """Tiles of 64 rows (8 heads, both ways) and of 16 (one key head) over every edge."""
    b = Batch(same(EDGES), Hq, Hkv, D, dt, causal=causal, packed=packed, seed=D)
    o, lse = b.forward()
    b.check_forward(o, lse)
    b.check_backward(*b.backward(o, lse))
    b.check_status()


@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("D", [1, 32, 60, 128])
@pytest.mark.parametrize("lens,place", [(same([1, 0, 63, 64, 2, 17, 16]), "self"), ([(5, 40), (0, 9), (17, 3), (33, 0), (16, 129)], "cache")])
def test_small_fp32_batches(lens, place, D, causal):
    """dq beside dk and dv in one launch, captured and replayed behind other work too."""
    b = Batch(lens, 2, 1, D, FP, causal=causal, place=place, seed=D)
    o, lse = b.forward()
    b.check_forward(o, lse)
    grads = b.backward(o, lse)
    b.check_backward(*grads)
    b.check_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, lse2 = b.forward()
        grads2 = b.backward(o2, lse2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(x, y) for x, y in zip(grads, grads2))
