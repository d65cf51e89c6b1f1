"""Attention of batches with empty, refused and overlapping sequences, of very many sequences, of long
sums in fp32, and of every call on the stream that it is given."""
import pytest
import torch

import token_routing_expert_router_gb300 as moe
from test_attn_gpu import Batch
from test_step_gpu import BF, FP, U, gen, normal, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(lib):
    pass


# Hq, Hkv, D, dtype: the tensor cores, the FMA units with bf16, and with fp32 by tiles of 64 rows and of 16
KERNELS = [(4, 2, 64, BF), (4, 1, 128, BF), (2, 1, 36, BF), (32, 32, 32, FP), (2, 1, 64, FP)]


@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("Hq,Hkv,D,dt", KERNELS)
def test_backward_with_empty_places(Hq, Hkv, D, dt, causal):
    """Places of a batch without keys, with and without queries, whose start is any row: nothing to report, and
    the sequences around them have their gradients."""
    b = Batch([(70, 90), (0, 0), (130, 200), (5, 0), (33, 40), (0, 0), (64, 64)], Hq, Hkv, D, dt, causal=causal, place="cache",
              seed=D)
    for at, row in ((1, 0), (3, b.Tk), (5, 7)):
        b.k_start[at] = row
    o, lse = b.forward()
    b.check_forward(o, lse)
    b.check_status()
    grads = b.backward(o, lse)
    assert moe.moe_read_status(b.bws) == moe.MOE_OK
    b.check_backward(*grads)


@pytest.mark.parametrize("name,value", [("k_len", "Tk"), ("k_start", "Tk"), ("k_start", -3), ("k_len", -1)])
@pytest.mark.parametrize("Hq,Hkv,D,dt", KERNELS)
def test_backward_behind_keys_out_of_range(Hq, Hkv, D, dt, name, value):
    """A sequence whose keys are not there takes none from the ones behind it."""
    lens = [(20, 40), (30, 50), (60, 80)]
    b = Batch(lens, Hq, Hkv, D, dt, place="cache", seed=D)
    o, lse = b.forward()
    want = b.backward(o, lse)
    getattr(b, name)[1] = b.Tk if value == "Tk" else value
    got = b.backward(o, lse)
    assert moe.moe_read_status(b.bws) == moe.MOE_ERR_DEVICE_BAD_INPUT
    for i in (0, 2):
        q, k = slice(b.q_at[i], b.q_at[i] + lens[i][0]), slice(b.k_at[i], b.k_at[i] + lens[i][1])
        for x, y, rows in zip(got, want, (q, k, k)):
            assert torch.equal(x[rows], y[rows])
    assert not got[0][20:50].any()
    assert all((x[b.k_at[1]:b.k_at[1] + 50] == 7).all() for x in got[1:])


def _keys_apart(start, length, Tk):
    """Which sequences keep their keys in the backward: those in range that do not begin before one in front
    of them, in range too, ends."""
    end, keep = 0, []
    for k0, m in zip(start, length):
        inside = 0 <= k0 <= Tk and 0 <= m <= Tk - k0
        keep.append(inside and (m == 0 or k0 >= end))
        if inside and m:
            end = max(end, k0 + m)
    return keep


OVERLAPS = [[(0, 100), (0, 50), (60, 40)], [(0, 100), (0, 50), (60, 40), (100, 30)], [(50, 30), (0, 60), (10, 20), (80, 0), (80, 40)],
            [(0, 90), (40, 400), (60, 20), (90, 30)], [(10, 5)] * 4]


@pytest.mark.parametrize("Hq,Hkv,D,dt", KERNELS)
@pytest.mark.parametrize("keys", OVERLAPS + ["many"])
def test_backward_of_overlapping_keys(keys, Hq, Hkv, D, dt):
    """Every key's gradient is written by one sequence: the others have no keys, and are reported."""
    if keys == "many":  # several sequences to a thread
        g = torch.Generator()
        g.manual_seed(3)
        keys, at = [], 0
        for i in range(700):
            m = int(torch.randint(0, 6, (1,), generator=g))
            back = int(torch.randint(0, 4, (1,), generator=g)) if i % 5 == 4 else 0
            keys.append((max(0, at - back), m))
            at = max(at, keys[-1][0] + m)
        Hq, Hkv = Hq // Hkv, 1
    Tk = max(k0 + m for k0, m in keys) + 3
    n = 2 if len(keys) > 100 else 40
    b = Batch([(n, 1)] * len(keys), Hq, Hkv, D, dt, place="cache", seed=7)
    b.cfg = moe.MoEAttnConfig.make(**{**b.cfg.as_dict(), "Tk": Tk})
    b.Tk = Tk
    b.k, b.v = normal(gen(1), Tk, Hkv, D, dtype=dt), normal(gen(2), Tk, Hkv, D, dtype=dt)
    b.k_start.copy_(torch.tensor([k for k, _ in keys], dtype=torch.int32))
    b.k_len.copy_(torch.tensor([m for _, m in keys], dtype=torch.int32))
    b.bws = torch.empty(moe.moe_attn_backward_workspace_size(b.cfg), dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(b.bws)
    keep = _keys_apart([k for k, _ in keys], [m for _, m in keys], Tk)
    assert not all(keep)
    o, lse = b.forward()
    got = b.backward(o, lse)
    assert moe.moe_read_status(b.bws) == moe.MOE_ERR_DEVICE_BAD_INPUT
    b.lens = [(n, m if ok else 0) for (_, m), ok in zip(keys, keep)]
    b.k_at = [k for k, _ in keys]
    b.check_backward(*got)
    for x, y in zip(got, b.backward(o, lse)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("rows,Hq,D,dt", [(140000, 128, 8, BF), (4300001, 1, 1, FP)])
def test_rows_that_come_back_65536_times(rows, Hq, D, dt):
    """A q_start that goes back to 0 for every second sequence: reported, also where the sequences' tiles
    together are more than 32 bits count, and nothing outside the rows is written."""
    B, code = 65536, moe.BF16 if dt == BF else moe.F32
    q, o = (torch.zeros(rows + 2, Hq, D, device="cuda", dtype=dt) for _ in range(2))
    o[0], o[-1] = 7, 7
    lse = torch.full((Hq + 2, rows), 7.0, device="cuda")
    q_start = torch.zeros(B + 1, device="cuda", dtype=torch.int32)
    q_start[1::2] = rows
    k, v = torch.ones(1, 1, D, device="cuda", dtype=dt), torch.full((1, 1, D), 3.0, device="cuda", dtype=dt)
    k_start, k_len = torch.zeros(B, device="cuda", dtype=torch.int32), torch.ones(B, device="cuda", dtype=torch.int32)
    cfg = moe.MoEAttnConfig.make(Tq=rows, Tk=1, B=B, Hq=Hq, Hkv=1, D=D, causal=0, act_dtype=code)
    ws = torch.empty(max(moe.moe_attn_workspace_size(cfg), moe.moe_attn_backward_workspace_size(cfg)), dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    moe.moe_attn(cfg, q[1:-1], k, v, q_start, k_start, k_len, o[1:-1], lse[1:-1], ws)
    assert moe.moe_read_status(ws) == moe.MOE_ERR_DEVICE_BAD_INPUT
    # every row's only key has the score 0
    assert ((o[1:-1] == 3) | (o[1:-1] == 0)).all() and ((lse[1:-1] == 0) | (lse[1:-1] == 7)).all()
    assert (o[0] == 7).all() and (o[-1] == 7).all() and (lse[0] == 7).all() and (lse[-1] == 7).all()
    dq, dkv = torch.zeros_like(q), torch.zeros(2, 3, 1, D, device="cuda", dtype=dt)
    dq[0], dq[-1] = 7, 7
    moe.moe_attn_backward(cfg, q[1:-1], k, v, q_start, k_start, k_len, o[1:-1], lse[1:-1], q[1:-1], dq[1:-1], dkv[0, 1:2], dkv[1, 1:2], ws)
    assert moe.moe_read_status(ws) == moe.MOE_ERR_DEVICE_BAD_INPUT
    assert not dq[1:-1].any() and (dq[0] == 7).all() and (dq[-1] == 7).all()
    assert not dkv[:, 0].any() and not dkv[:, 2].any()


def _uniform(n, m, Hq, Hkv, D, seed):
    """A batch whose scores are all 0 (every probability 1 / m) and whose rows are all alike."""
    b = Batch([(n, m)], Hq, Hkv, D, FP, causal=0, place="cache", seed=seed)
    g = gen(seed + 1)
    row = torch.rand(2, Hq, D, generator=g, device="cuda") + 1.0
    b.q[:n], b.do[:n] = row[0], row[1]
    return b


@pytest.mark.parametrize("D", [16, 128])
@pytest.mark.parametrize("Hkv", [1, 32])
def test_long_sums_of_key_gradients_in_fp32(Hkv, D):
    """dk and dv over 32768 equal terms: an accumulator that takes them one after the other rounds every one
    the same way."""
    n, m, G = 8192, 64, 4
    b = _uniform(n, m, Hkv * G, Hkv, D, 5)
    at = slice(b.k_at[0], b.k_at[0] + m)
    b.k[at] = 0
    o, lse = b.forward()
    _, dk, dv = b.backward(o, lse)
    q, do = b.q[0].double().view(Hkv, G, D), b.do[0].double().view(Hkv, G, D)
    v = b.v[at].double().transpose(0, 1)                       # [Hkv, m, D]
    # sums of 64 terms each, and of their n G / 64 results; beside them p: lse's rounding and logf's (2 U each of
    # 4.2), expf's 4 U; the scale on q, the products, the result: 32 U cover all of them
    rel = (64 + n * G / 64 + 32) * U
    want = (n / m * do.sum(1))[:, None].expand(Hkv, m, D)
    within(dv[at].transpose(0, 1), want, rel * want.abs())
    dp = torch.einsum("hgd,hmd->hgm", do, v)
    mean = dp.mean(2, keepdim=True)
    size = torch.einsum("hgd,hmd->hgm", do.abs(), v.abs())
    # dp and delta: D products each; o: 64 terms, a division, its rounding
    lost = (D + 8) * U * size + ((D + 8) + 64 + 32) * U * size.mean(2, keepdim=True)
    ds = (dp - mean) / m
    want = n * b.scale * torch.einsum("hgm,hgd->hmd", ds, q)
    bound = n * b.scale * torch.einsum("hgm,hgd->hmd", lost / m + rel * ds.abs(), q)
    within(dk[at].transpose(0, 1), want, bound)


@pytest.mark.parametrize("D", [16, 128])
@pytest.mark.parametrize("Hq", [1, 64])
def test_long_sums_of_query_gradients_in_fp32(Hq, D):
    """dq over 32768 equal terms."""
    n, m = 64, 32768
    b = _uniform(n, m, Hq, 1, D, 6)
    b.q[:n] = 0
    at = slice(b.k_at[0], b.k_at[0] + m)
    row = torch.rand(2, D, generator=gen(9), device="cuda") + 1.0
    sign = 1.0 - 2.0 * (torch.arange(m, device="cuda") % 2)
    b.k[at], b.v[at] = (sign[:, None] * row[0])[:, None], (sign[:, None] * row[1])[:, None]
    o, lse = b.forward()
    dq, _, _ = b.backward(o, lse)
    x = b.do[0].double() @ row[1].double()                    # [Hq]: do . v of the even keys; o and delta are 0
    want = b.scale * x[:, None] * row[0].double()
    # sums of 64 terms, and of their m / 64 results; p: 2 U each of lse's 10.4 twice, expf 4 U; x: D + 8 roundings;
    # the scale, the products and the result; what o is not quite 0 by falls out, as the keys' signs do
    rel = (64 + m / 64 + 64 + D + 8) * U
    within(dq[:n], want.expand(n, Hq, D), rel * want.abs())


@pytest.mark.parametrize("B,Hq,Hkv,D", [(385, 4, 2, 64), (1000, 8, 4, 32), (3000, 2, 2, 128)])
def test_single_tokens_of_very_many_requests(B, Hq, Hkv, D):
    """More requests than a block has threads: several to a thread, those without keys or queries among them."""
    lens = [(0 if i % 11 == 5 else 1, 0 if i % 7 == 3 else (37 * i) % 190 + (400 if i % 97 == 0 else 0)) for i in range(B)]
    b = Batch(lens, Hq, Hkv, D, BF, place="cache", max_q=1, seed=B)
    o, lse = b.forward()
    b.check_forward(o, lse)
    b.check_status()
    o2, lse2 = b.forward()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("lens,Hq,Hkv", [([(1, 900), (0, 4), (1, 33), (1, 0), (1, 2000)], 64, 1), ([(4, 500), (1, 70)], 32, 2),
                                         ([(1, 700)], 49, 1)])
def test_fp32_groups_beyond_tiles_of_few_rows(lens, Hq, Hkv, causal):
    """More than 48 rows of a key head over a cache."""
    b = Batch(lens, Hq, Hkv, 64, FP, causal=causal, place="cache", seed=Hq)
    o, lse = b.forward()
    b.check_forward(o, lse)
    b.check_status()
    b.check_backward(*b.backward(o, lse))


@pytest.mark.parametrize("dt,D", [(BF, 64), (FP, 32)])
def test_calls_run_on_the_stream_that_is_given(dt, D):
    """Every call's input is made by work on a side stream that is still running when the call is given that
    stream: on any other it would read what was there before."""
    Hq, Hkv, T = 4, 2, 200
    b = Batch([(T, T)], Hq, Hkv, D, dt, seed=6, tail=0)
    o, lse = b.forward()
    grads = b.backward(o, lse)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    rope = moe.MoERopeConfig.make(T=T, Hq=Hq, Hk=Hkv, D=D, act_dtype=moe.BF16 if dt == BF else moe.F32)
    table = torch.empty(D // 2, dtype=torch.int64, device="cuda")
    moe.moe_rope_table(moe.MoERopeFreq.make(rot=D), table)
    turned, back = ([torch.empty_like(x) for x in (b.q, b.k)] for _ in range(2))
    moe.moe_rope(rope, b.q, b.k, None, pos, None, table, *turned[:1], turned[1], None)
    moe.moe_rope_backward(rope, b.q, b.k, pos, table, *back)
    q, do = b.q.clone(), b.do.clone()
    big = torch.randn(4096, 4096, device="cuda").to(BF)
    sink = torch.empty_like(big)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.mm(big, big, out=sink)  # the library's first call on a stream is slow

    def behind(target, value, call):
        """call, with `target` turned into `value` by the side stream after some milliseconds of other work."""
        target.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(150):
                torch.mm(big, big, out=sink)
            target.copy_(value)
        assert not side.query()  # still at it
        call()
        side.synchronize()
        torch.cuda.synchronize()

    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    behind(b.q, q, lambda: moe.moe_attn(b.cfg, b.q, b.k, b.v, b.q_start, None, None, o2, lse2, b.ws, stream=side))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    got = [torch.empty_like(x) for x in grads]
    behind(b.do, do, lambda: moe.moe_attn_backward(b.cfg, b.q, b.k, b.v, b.q_start, None, None, o, lse, b.do, *got, b.bws, stream=side))
    assert all(torch.equal(x, y) for x, y in zip(grads, got))
    got = [torch.empty_like(x) for x in turned]
    behind(b.q, q, lambda: moe.moe_rope(rope, b.q, b.k, None, pos, None, table, *got, None, stream=side))
    assert all(torch.equal(x, y) for x, y in zip(turned, got))
    got = [torch.empty_like(x) for x in back]
    behind(b.q, q, lambda: moe.moe_rope_backward(rope, b.q, b.k, pos, table, *got, stream=side))
    assert all(torch.equal(x, y) for x, y in zip(back, got))
