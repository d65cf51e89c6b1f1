"""The operators around the layer against plain implementations in 64 bits.

Tolerances are bounds, per element, on what the documented arithmetic can lose: U = 2^-24 is
half a step of fp32, HALF[t] half a step of an output type. A sum of n fp32 terms that is added
in any order is off by at most n U times the sum of the terms' magnitudes, and usually the depth
of the additions stands in n's place where it is known.
"""
import math

import pytest
import torch

import token_routing_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
CODE = {torch.float32: moe.F32, torch.bfloat16: moe.BF16}
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _built(lib):
    pass


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=FP, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def workspace(size):
    ws = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")  # what a fresh buffer may hold
    moe.moe_workspace_init(ws)
    return ws


def poisoned(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def within(got, want, bound):
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all()
    over = ((got - want).abs() - bound).max().item()
    assert over <= 0, f"off by {(got - want).abs().max().item():.3g}, {over:.3g} over the bound"


# ---------------------------------------------------------------------------------- norms
EPS, RES = 1e-6, 0.875
NORM_CASES = [
    # T, H, dtype, post, next, gate, token gate
    (1, 7168, BF, 1, 1, 1, 1), (3, 8, BF, 1, 1, 1, 0), (5, 1, FP, 1, 1, 1, 1), (1, 2, BF, 1, 1, 0, 1),
    (700, 2048, BF, 1, 1, 1, 1), (641, 264, BF, 0, 1, 1, 0), (333, 1001, FP, 1, 1, 1, 1), (130, 999, BF, 1, 1, 0, 1),
    (65, 512, FP, 1, 0, 0, 1), (97, 4096, FP, 1, 1, 1, 0), (40, 4100, FP, 1, 1, 1, 1), (20, 8200, BF, 1, 1, 1, 1),
    (9, 16384, BF, 1, 1, 1, 1), (9, 16384, FP, 1, 1, 1, 1), (7, 16383, FP, 0, 1, 0, 0), (6, 5001, BF, 1, 1, 1, 1),
    (2000, 64, BF, 1, 1, 1, 1), (50, 96, BF, 0, 0, 0, 0), (400, 7168, BF, 1, 1, 0, 0), (700, 1002, BF, 1, 1, 1, 1),
    (30, 5002, BF, 1, 1, 1, 1), (500, 7168, FP, 1, 1, 1, 1), (300, 12296, BF, 1, 1, 1, 1), (1100, 1500, FP, 0, 1, 0, 1)]


def norm_inputs(T, H, dt, post, nxt, gate, tgate, seed=0):
    g = gen(seed)
    d = dict(x=normal(g, T, H, dtype=dt, std=2.0), y=normal(g, T, H, dtype=dt, std=0.7),
             w_post=normal(g, H, std=0.2, mean=1.0) if post else None,
             w_next=normal(g, H, std=0.2, mean=1.0) if nxt else None,
             gate=normal(g, H, std=0.3, mean=0.5) if gate else None,
             token_gate=torch.rand(T, generator=g, device="cuda") if tgate else None)
    if T > 2:
        d["x"][1] = 0  # a row of zeros in both: rho = 1 / sqrt(eps)
        d["y"][1] = 0
    return d


def rho(v):
    return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def norm_reference(d):
    """The new residual, its norm, and the branch, in 64 bits and differentiable."""
    q = {k: None if v is None else v.double().requires_grad_(True) for k, v in d.items()}
    u = q["y"] if q["w_post"] is None else q["y"] * rho(q["y"]) * q["w_post"]
    u = u if q["gate"] is None else u * q["gate"]
    u = u if q["token_gate"] is None else u * q["token_gate"][:, None]
    r = RES * q["x"] + u
    n = None if q["w_next"] is None else r * rho(r) * q["w_next"]
    return q, u, r, n


@pytest.mark.parametrize("T,H,dt,post,nxt,gate,tgate", NORM_CASES)
def test_block_norm(T, H, dt, post, nxt, gate, tgate):
    d = norm_inputs(T, H, dt, post, nxt, gate, tgate)
    cfg = moe.MoENormConfig.make(T=T, H=H, act_dtype=CODE[dt], eps=EPS, res_scale=RES)
    r, n = poisoned(T, H, dtype=dt), poisoned(T, H, dtype=dt) if nxt else None
    moe.moe_block_norm(cfg, d["x"], d["y"], d["w_post"], d["w_next"], r, n, gate=d["gate"], token_gate=d["token_gate"])
    with torch.no_grad():
        _, u, rr, nn = norm_reference(d)
        # rho: a sum of depth 16 + 5 + 5, the mean, eps, root and quotient: 32 U / 2 and a few more
        lost = 40 * U * ((RES * d["x"].double()).abs() + u.abs())
        within(r, rr, lost + HALF[dt] * (rr.abs() + lost))
        if nxt:
            ln = lost * rho(rr) * d["w_next"].double().abs() + 40 * U * nn.abs()
            # rho(r) also sees r's own error, at most its row norm's relative part
            ln = ln + nn.abs() * (lost.norm(dim=1, keepdim=True) / (rr.norm(dim=1, keepdim=True) + math.sqrt(H * EPS)))
            within(n, nn, ln + HALF[dt] * (nn.abs() + ln))
    # without the residual or without the norm, and in place: the same bits
    if nxt:
        n2 = d["y"].clone()
        x2 = d["x"].clone()
        moe.moe_block_norm(cfg, x2, n2, d["w_post"], d["w_next"], x2, n2, gate=d["gate"], token_gate=d["token_gate"])
        assert torch.equal(x2, r) and torch.equal(n2, n)
        n3 = poisoned(T, H, dtype=dt)
        moe.moe_block_norm(cfg, d["x"], d["y"], d["w_post"], d["w_next"], None, n3, gate=d["gate"],
                           token_gate=d["token_gate"])
        assert torch.equal(n3, n)


def test_block_norm_before_the_first_block():
    T, H = 37, 264
    x, w = normal(gen(1), T, H, dtype=BF), normal(gen(2), H, mean=1.0)
    cfg = moe.MoENormConfig.make(T=T, H=H, eps=EPS)
    n, r = poisoned(T, H, dtype=BF), poisoned(T, H, dtype=BF)
    moe.moe_block_norm(cfg, x, None, None, w, r, n)
    want = x.double() * rho(x.double()) * w.double()
    assert torch.equal(r, x)
    within(n, want, (HALF[BF] + 40 * U) * 1.01 * want.abs())


@pytest.mark.parametrize("T,H,dt,post,nxt,gate,tgate", NORM_CASES)
def test_block_norm_backward(T, H, dt, post, nxt, gate, tgate):
    d = norm_inputs(T, H, dt, post, nxt, gate, tgate, seed=3)
    g = gen(4)
    dr, dn = normal(g, T, H, dtype=dt, std=0.1), normal(g, T, H, dtype=dt, std=0.1) if nxt else None
    cfg = moe.MoENormConfig.make(T=T, H=H, act_dtype=CODE[dt], eps=EPS, res_scale=RES)
    r = d["x"]  # any residual will do: the backward reads only the new one
    dx, dy = poisoned(T, H, dtype=dt), poisoned(T, H, dtype=dt)
    grads = {"dgate": poisoned(H, dtype=FP), "dtoken_gate": poisoned(T, dtype=FP),
             "dw_post": poisoned(H, dtype=FP) if post else None, "dw_next": poisoned(H, dtype=FP) if nxt else None}
    ws = workspace(moe.moe_block_norm_workspace_size(cfg))
    call = lambda a, b, gr: moe.moe_block_norm_backward(  # noqa: E731
        cfg, r, d["y"], d["w_post"], d["w_next"], dr, dn, a, b, gr, ws, gate=d["gate"], token_gate=d["token_gate"])
    call(dx, dy, grads)

    # the formula, written out with the magnitudes of its terms (for the bounds)
    R, Y, DR = r.double(), d["y"].double(), dr.double()
    one = torch.ones((), dtype=torch.float64, device="cuda")
    wp = d["w_post"].double() if post else one
    G = d["gate"].double() if gate else one
    gt = d["token_gate"].double()[:, None] if tgate else one
    full, mag = DR, DR.abs()
    if nxt:
        p, a = rho(R), dn.double() * d["w_next"].double()
        full = DR + p * a - p ** 3 * R * (a * R).mean(1, keepdim=True)
        mag = DR.abs() + p * a.abs() + p ** 3 * R.abs() * (a * R).abs().mean(1, keepdim=True)
    k = 64 * U  # row sums of depth 26 and the handful of products around them
    lost = k * mag
    within(dx, RES * full, RES * (lost + HALF[dt] * (full.abs() + lost)) + U * full.abs())
    py = rho(Y) if post else one
    b, bl = wp * G * full, (wp * G).abs() * mag
    q, ql = (b * Y).sum(1, keepdim=True), (bl * Y.abs()).sum(1, keepdim=True)
    want = gt * (py * b - (py ** 3 * Y * q / H if post else 0))
    wl = 2 * k * gt * (py * bl + (py ** 3 * Y.abs() * ql / H if post else 0))
    within(dy, want, wl + HALF[dt] * (want.abs() + wl))
    within(grads["dtoken_gate"], (py * q)[:, 0], 2 * k * (py * ql)[:, 0])
    col = (2 * k + T * U)
    S, Sl = gt * full * Y * py, gt * mag * (Y * py).abs()
    within(grads["dgate"], (S * wp).sum(0), col * (Sl * wp.abs()).sum(0))
    if post:
        within(grads["dw_post"], (S * G).sum(0), col * (Sl * G.abs()).sum(0))
    if nxt:
        N = dn.double() * R * rho(R)
        within(grads["dw_next"], N.sum(0), col * N.abs().sum(0))

    # the formula against differentiation of the forward, and the same bits a second time and in place
    x0 = (R - gt * G * wp * Y * py) / RES
    q_ = {k_: None if v is None else v.double().requires_grad_(True) for k_, v in {**d, "x": x0}.items()}
    u = q_["y"] if not post else q_["y"] * rho(q_["y"]) * q_["w_post"]
    u = u if not gate else u * q_["gate"]
    u = u if not tgate else u * q_["token_gate"][:, None]
    rr = RES * q_["x"] + u
    total = (rr * DR).sum() + ((rr * rho(rr) * q_["w_next"] * dn.double()).sum() if nxt else 0)
    total.backward()
    torch.testing.assert_close(q_["x"].grad, RES * full, rtol=1e-7, atol=1e-9)
    torch.testing.assert_close(q_["y"].grad, want, rtol=1e-7, atol=1e-7)
    dx2, dy2 = dr.clone(), dn.clone() if nxt else poisoned(T, H, dtype=dt)
    grads2 = {k_: None if v is None else torch.empty_like(v) for k_, v in grads.items()}
    moe.moe_block_norm_backward(cfg, r, d["y"], d["w_post"], d["w_next"], dx2, dy2 if nxt else None, dx2, dy2, grads2,
                                ws, gate=d["gate"], token_gate=d["token_gate"])
    assert torch.equal(dx, dx2) and torch.equal(dy, dy2)
    for name, v in grads.items():
        assert v is None or torch.equal(v, grads2[name]), name
    # no rows: zero column gradients
    z = torch.full((H,), 3.0, device="cuda")
    empty = torch.empty(0, H, dtype=dt, device="cuda")
    cfg0 = moe.MoENormConfig.make(T=0, H=H, act_dtype=CODE[dt], eps=EPS)
    if nxt:
        moe.moe_block_norm_backward(cfg0, None, None, None, d["w_next"], None, None, empty, None, {"dw_next": z}, None)
        assert (z == 0).all()


@pytest.mark.parametrize("dt", [FP, BF])
def test_block_norm_backward_of_zero_rows_with_a_tiny_eps(dt):
    """rho = 1e15 there: its cube does not fit fp32, and meets sums that are 0."""
    T, H = 6, 64
    g = gen(3)
    zero = torch.zeros(T, H, dtype=dt, device="cuda")
    w_post, w_next = normal(g, H, std=0.2, mean=1.0), normal(g, H, std=0.2, mean=1.0)
    dr, dn = normal(g, T, H, dtype=dt), normal(g, T, H, dtype=dt)
    dx, dy = poisoned(T, H, dtype=dt), poisoned(T, H, dtype=dt)
    cfg = moe.MoENormConfig.make(T=T, H=H, act_dtype=CODE[dt], eps=1e-30, res_scale=RES)
    r = torch.tensor(1e-30, dtype=FP).double().item() ** -0.5
    moe.moe_block_norm_backward(cfg, zero, zero, w_post, w_next, dr, dn, dx, dy, {}, None)
    d = dr.double() + r * dn.double() * w_next.double()
    # rho (2 steps of rsqrt, the mean's), three products and a sum
    for got, want in ((dx, RES * d), (dy, r * w_post.double() * d)):
        within(got, want, (HALF[dt] + 16 * U) * want.abs() + 16 * U * r * (r if got is dy else 1))


def test_block_norm_backward_by_differences():
    """A small central-difference check of the kernels' own forward and backward, in fp32."""
    T, H = 3, 16
    d = norm_inputs(T, H, FP, 1, 1, 1, 1, seed=9)
    d["x"][1] = 1.5
    d["y"][1] = -0.5
    cfg = moe.MoENormConfig.make(T=T, H=H, act_dtype=moe.F32, eps=EPS, res_scale=RES)
    dr, dn = normal(gen(5), T, H), normal(gen(6), T, H)

    def forward(v):
        r, n = poisoned(T, H, dtype=FP), poisoned(T, H, dtype=FP)
        moe.moe_block_norm(cfg, v["x"], v["y"], v["w_post"], v["w_next"], r, n, gate=v["gate"],
                           token_gate=v["token_gate"])
        return r, (r.double() * dr.double()).sum().item() + (n.double() * dn.double()).sum().item()

    r, _ = forward(d)
    dx, dy = poisoned(T, H, dtype=FP), poisoned(T, H, dtype=FP)
    grads = {"dw_post": poisoned(H, dtype=FP), "dw_next": poisoned(H, dtype=FP), "dgate": poisoned(H, dtype=FP),
             "dtoken_gate": poisoned(T, dtype=FP)}
    moe.moe_block_norm_backward(cfg, r, d["y"], d["w_post"], d["w_next"], dr, dn, dx, dy, grads,
                                workspace(moe.moe_block_norm_workspace_size(cfg)), gate=d["gate"],
                                token_gate=d["token_gate"])
    step = 2.0 ** -8
    for name, grad in (("x", dx), ("y", dy), ("w_post", grads["dw_post"]), ("w_next", grads["dw_next"]),
                       ("gate", grads["dgate"]), ("token_gate", grads["dtoken_gate"])):
        for at in range(0, grad.numel(), 5):
            lo, hi = ({k: v.clone() for k, v in d.items()} for _ in range(2))
            lo[name].view(-1)[at] -= step
            hi[name].view(-1)[at] += step
            diff = (forward(hi)[1] - forward(lo)[1]) / (2 * step)
            # the third derivative's step^2 share, and 96 outputs' fp32 rounding over the step
            assert abs(diff - grad.view(-1)[at].item()) < 3e-3 * (1 + abs(diff)), (name, at)


# ---------------------------------------------------------------------------------- head
HEAD_CASES = [
    # T, H, V, dtype, grad dtype, piece, share of tokens left out
    (1, 64, 1, BF, BF, 0, 0.0), (1, 8, 300, BF, FP, 0, 0.0), (33, 512, 1000, BF, BF, 0, 0.2),
    (128, 256, 777, BF, FP, 256, 0.1), (129, 264, 1025, BF, BF, 0, 0.3), (300, 128, 5003, BF, BF, 1024, 0.1),
    (513, 1032, 2500, BF, FP, 1000, 0.0), (256, 64, 257, BF, BF, 256, 1.0), (70, 2048, 40000, BF, BF, 39936, 0.0),
    (2, 128, 33000, BF, BF, 0, 0.0), (1, 1, 1, FP, FP, 0, 0.0), (7, 33, 129, FP, FP, 0, 0.3),
    (200, 128, 1003, FP, FP, 256, 0.1), (130, 77, 300, BF, BF, 0, 0.1), (64, 96, 20000, FP, BF, 0, 0.0),
    (150, 33, 400, FP, FP, 256, 0.1), (140, 35, 300, FP, BF, 0, 0.2), (1100, 72, 300, BF, FP, 256, 0.1),
    (1500, 40, 700, FP, FP, 0, 0.5), (300, 101, 600, BF, FP, 256, 0.0)]


@pytest.mark.parametrize("T,H,V,dt,gdt,piece,skip", HEAD_CASES)
def test_head_loss_and_gradients(T, H, V, dt, gdt, piece, skip):
    g = gen(T + H + V)
    w, t = normal(g, V, H, dtype=dt, std=0.05), torch.randint(0, V, (T,), generator=g, device="cuda")
    x = (normal(g, T, H) + 8.0 / (0.05 ** 2 * H) * w[t].float() * torch.rand(T, 1, generator=g, device="cuda")).to(dt)
    out = torch.rand(T, generator=g, device="cuda") < skip
    target = torch.where(out, -1 - (t % 3), t).to(torch.int32)
    cfg = moe.MoEHeadConfig.make(T=T, H=H, V=V, act_dtype=CODE[dt], grad_dtype=CODE[gdt], piece=piece)
    ws = workspace(moe.moe_head_workspace_size(cfg))
    loss, lse, mean = poisoned(T, dtype=FP), poisoned(T, dtype=FP), poisoned(2, dtype=FP)
    moe.moe_head_loss(cfg, x, w, target, loss, lse, mean, ws)

    X, W = x.double(), w.double()
    z = X @ W.t()
    keep = target >= 0
    wl = torch.logsumexp(z, 1)
    wloss = torch.where(keep, wl - z.gather(1, t[:, None])[:, 0], 0.0)
    # a logit: H exact products added in fp32 (the tensor core may truncate: a whole step each)
    dz = 2 * U * H * (X.abs() @ W.abs().t()).amax(1) + 8 * U * z.abs().amax(1)
    within(lse, wl, dz + 64 * U * (1 + wl.abs()))
    within(loss, wloss, torch.where(keep, 2 * dz + 64 * U * (1 + wl.abs() + wloss), 0.0))
    n = int(keep.sum())
    within(mean[1:], torch.full((1,), 1 / n if n else 0.0, device="cuda"), U * 2)
    within(mean[:1], (wloss.sum() / max(n, 1))[None], (2 * dz + 80 * U * (1 + wl.abs() + wloss)).max() + 8 * U)

    p = torch.exp(z - wl[:, None])
    hot = torch.zeros_like(z).scatter_(1, t[:, None], 1.0)
    for weights in (None, torch.rand(T, generator=g, device="cuda") + 0.1):
        dl = torch.where(keep, 1.0 / max(n, 1), 0.0) if weights is None else torch.where(keep, weights.double(), 0.0)
        D = (p - hot) * dl[:, None]
        tc = dt == BF and H % 8 == 0
        # dz: p off by its exponent's error, then rounded to bf16 for the tensor cores
        Dl = (p * (2 * dz + 32 * U * (1 + wl.abs()))[:, None] + 4 * U * (p + hot)) * dl[:, None]
        Dl = Dl + (HALF[BF] if tc else 0) * (D.abs() + Dl)
        dx, dw = poisoned(T, H, dtype=dt), poisoned(V, H, dtype=gdt)
        moe.moe_head_loss_backward(cfg, x, w, target, lse, dx, dw, ws, dloss=weights,
                                   mean=mean if weights is None else None)
        for got, want, lost in ((dx, D @ W, Dl @ W.abs() + 2 * U * (V + 64) * (D.abs() @ W.abs())),
                                (dw, D.t() @ X, Dl.t() @ X.abs() + 2 * U * (T + 64) * (D.abs().t() @ X.abs()))):
            within(got, want, lost + HALF[got.dtype] * (want.abs() + lost) + 1e-37)
        assert not bool(dx[~keep].any())
    # either gradient alone: the same bits
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    moe.moe_head_loss_backward(cfg, x, w, target, lse, dx2, None, ws, dloss=weights)
    moe.moe_head_loss_backward(cfg, x, w, target, lse, None, dw2, ws, dloss=weights)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    assert moe.moe_read_status(ws) == moe.MOE_OK


def test_head_gradients_by_differences():
    T, H, V = 5, 24, 40
    g = gen(8)
    x, w = normal(g, T, H), normal(g, V, H, std=0.3)
    target = torch.tensor([0, 39, -1, 7, 7], dtype=torch.int32, device="cuda")
    cfg = moe.MoEHeadConfig.make(T=T, H=H, V=V, act_dtype=moe.F32)
    ws = workspace(moe.moe_head_workspace_size(cfg))

    def forward(a, b):
        loss, lse, mean = poisoned(T, dtype=FP), poisoned(T, dtype=FP), poisoned(2, dtype=FP)
        moe.moe_head_loss(cfg, a, b, target, loss, lse, mean, ws)
        return lse, mean, loss.double().sum().item() / 4

    lse, mean, _ = forward(x, w)
    dx, dw = poisoned(T, H, dtype=FP), poisoned(V, H, dtype=FP)
    moe.moe_head_loss_backward(cfg, x, w, target, lse, dx, dw, ws, mean=mean)
    step = 2.0 ** -6
    for v, grad in ((x, dx), (w, dw)):
        for at in range(0, v.numel(), 37):
            lo, hi = v.clone(), v.clone()
            lo.view(-1)[at] -= step
            hi.view(-1)[at] += step
            pair = ((hi, w), (lo, w)) if v is x else ((x, hi), (x, lo))
            diff = (forward(*pair[0])[2] - forward(*pair[1])[2]) / (2 * step)
            # losses of about 4 in fp32, added over 4 tokens, divided by the step; the step's cubic share
            assert abs(diff - grad.view(-1)[at].item()) < 2e-4, (at, diff)


def test_head_bad_target_and_large_logits():
    T, H, V = 40, 64, 500
    g = gen(2)
    x, w = normal(g, T, H, dtype=BF, std=30.0), normal(g, V, H, dtype=BF, std=3.0)
    target = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    target[7] = V
    target[9] = 2 ** 31 - 1
    cfg = moe.MoEHeadConfig.make(T=T, H=H, V=V, grad_dtype=moe.BF16)
    ws = workspace(moe.moe_head_workspace_size(cfg))
    loss, lse, mean = poisoned(T, dtype=FP), poisoned(T, dtype=FP), poisoned(2, dtype=FP)
    moe.moe_head_loss(cfg, x, w, target, loss, lse, mean, ws)
    z = x.double() @ w.double().t()
    bound = 2 * U * H * (x.double().abs() @ w.double().abs().t()).amax(1) + 64 * U * (1 + z.abs().amax(1))
    within(lse, torch.logsumexp(z, 1), bound)
    assert loss[7] == 0 and loss[9] == 0 and mean[1].item() == pytest.approx(1 / 38)
    assert moe.moe_read_status(ws) == moe.MOE_ERR_DEVICE_BAD_INPUT
    dx, dw = poisoned(T, H, dtype=BF), poisoned(V, H, dtype=BF)
    moe.moe_head_loss_backward(cfg, x, w, target, lse, dx, dw, ws, mean=mean)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    assert not bool(dx[7].any()) and not bool(dx[9].any())
    # no tokens: a zero weight gradient and a zero mean
    c0 = moe.MoEHeadConfig.make(T=0, H=H, V=V, grad_dtype=moe.BF16)
    moe.moe_head_loss(c0, None, w, None, None, None, mean, ws)
    moe.moe_head_loss_backward(c0, None, w, None, None, None, dw, ws)
    assert not bool(mean.any()) and not bool(dw.any())


@pytest.mark.parametrize("T,H,V,dt", [(300, 256, 1000, BF), (40, 64, 500, BF), (200, 33, 300, BF), (70, 40, 260, FP)])
def test_head_left_out_tokens_may_hold_anything(T, H, V, dt):
    """Padded rows of x, and their loss gradients, may be NaN or infinite: the other tokens' losses
    and both gradients have the bits that they have with zeros there."""
    g = gen(T)
    x, w = normal(g, T, H, dtype=dt), normal(g, V, H, dtype=dt, std=0.2)
    target = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    target[3::4], target[T - 1] = -1, V
    keep = (target >= 0) & (target < V)
    cfg = moe.MoEHeadConfig.make(T=T, H=H, V=V, act_dtype=CODE[dt])
    ws = workspace(moe.moe_head_workspace_size(cfg))

    def step(fill):
        xf, dl = x.clone(), torch.rand(T, generator=gen(5), device="cuda")
        xf[~keep], dl[~keep] = fill, fill
        loss, lse, mean = poisoned(T, dtype=FP), poisoned(T, dtype=FP), poisoned(2, dtype=FP)
        moe.moe_head_loss(cfg, xf, w, target, loss, lse, mean, ws)
        out = [loss, lse[keep], mean]
        for d in (None, dl):
            dx, dw, dx2 = poisoned(T, H, dtype=dt), poisoned(V, H, dtype=FP), poisoned(T, H, dtype=dt)
            moe.moe_head_loss_backward(cfg, xf, w, target, lse, dx, dw, ws, dloss=d, mean=mean if d is None else None)
            moe.moe_head_loss_backward(cfg, xf, w, target, lse, dx2, None, ws, dloss=d, mean=mean if d is None else None)
            out += [dx, dw, dx2]
        return out

    want = step(0.0)
    assert all(torch.isfinite(v).all() for v in want)
    for fill in (float("nan"), float("inf"), -3e38):
        assert all(torch.equal(a, b) for a, b in zip(step(fill), want))


@pytest.mark.parametrize("T,H,V,dt,share", [(1500, 64, 300, BF, 0.6), (700, 40, 260, FP, 0.9), (130, 136, 5000, BF, 0.99),
                                           (300, 33, 700, BF, 1.0), (100, 64, 4000, BF, 1.0), (90000, 8, 40, BF, 0.5),
                                           (70001, 16, 24, FP, 0.2)])
def test_head_gradients_of_the_tokens_that_count(T, H, V, dt, share):
    """Left-out tokens cost nothing and change nothing: the gradients have the bits of a call with
    only the others (in the same pieces), at their rows of dx, zeros at the rest."""
    g = gen(T)
    x, w = normal(g, T, H, dtype=dt), normal(g, V, H, dtype=dt, std=0.2)
    target = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    target[torch.rand(T, generator=g, device="cuda") < share] = -1
    keep = target >= 0
    n = int(keep.sum())
    dl = torch.rand(T, generator=g, device="cuda")

    def step(x, target, dl):
        T = x.shape[0]
        cfg = moe.MoEHeadConfig.make(T=T, H=H, V=V, act_dtype=CODE[dt], piece=512)
        ws = workspace(moe.moe_head_workspace_size(cfg))
        loss, lse = poisoned(T, dtype=FP), poisoned(T, dtype=FP)
        dx, dw = poisoned(T, H, dtype=dt), poisoned(V, H, dtype=FP)
        moe.moe_head_loss(cfg, x, w, target, loss, lse, None, ws)
        moe.moe_head_loss_backward(cfg, x, w, target, lse, dx, dw, ws, dloss=dl)
        return lse, dx, dw

    lse, dx, dw = step(x, target, dl)
    assert not bool(dx[~keep].any())
    if n == 0:
        assert not bool(dw.any())
        return
    lse2, dx2, dw2 = step(x[keep], target[keep], dl[keep])
    if n > 128 or T <= 128:  # up to 128 tokens the tiles are others
        assert torch.equal(lse[keep], lse2) and torch.equal(dx[keep], dx2) and torch.equal(dw, dw2)
    # and against the formula
    X, W = x[keep].double(), w.double()
    z = X @ W.t()
    D = (torch.exp(z - lse2.double()[:, None]) - torch.zeros_like(z).scatter_(1, target[keep].long()[:, None], 1.0)) * dl[keep].double()[:, None]
    tc = HALF[BF] if dt == BF and H % 8 == 0 else 0.0
    # z within a truncated step per product, the exponent's own rounding, dz in bf16
    lost = (2 * U * H * (X.abs() @ W.abs().t()) + 64 * U * (1 + z.abs())) * dl[keep].double()[:, None] + (tc + 8 * U) * D.abs() * 1.01
    for got, want, l, k in ((dx[keep], D @ W, lost @ W.abs(), V), (dw, D.t() @ X, lost.t() @ X.abs(), n)):
        mag = (D.abs() @ W.abs()) if k == V else (D.abs().t() @ X.abs())
        within(got, want, l + 2 * U * (k + 64) * mag + HALF[got.dtype] * (want.abs() + l) + 1e-37)


# ---------------------------------------------------------------------------------- embedding
def tokens_of(kind, T, V, g):
    if kind == "uniform":
        return torch.randint(0, V, (T,), generator=g, device="cuda")
    if kind == "one":        # every position the same token
        return torch.full((T,), V - 1, device="cuda")
    if kind == "hot":        # half of them one token, the rest spread
        t = torch.randint(0, V, (T,), generator=g, device="cuda")
        return torch.where(torch.rand(T, generator=g, device="cuda") < 0.5, V // 2, t)
    if kind == "none":       # all padding
        return torch.full((T,), -1, device="cuda")
    return torch.arange(T, device="cuda") % V  # "ramp": runs of T / V that straddle the chunks


EMBED_CASES = [
    (1, 64, 1, BF, FP, "uniform"), (1, 3, 7, FP, FP, "uniform"), (31, 8, 5, BF, BF, "ramp"), (64, 2048, 300, BF, FP, "hot"),
    (2048, 40, 97, BF, FP, "ramp"), (2049, 16, 1000, FP, FP, "uniform"), (4100, 264, 7, BF, BF, "hot"),
    (5000, 24, 300, BF, FP, "one"), (3000, 33, 64, BF, FP, "hot"), (2500, 9, 2000, FP, BF, "ramp"),
    (100, 128, 70, BF, FP, "none"), (40000, 16, 50257, BF, FP, "hot"), (300000, 8, 1000, BF, FP, "hot"),
    (70, 4104, 129, BF, FP, "uniform")]


@pytest.mark.parametrize("T,H,V,dt,gdt,kind", EMBED_CASES)
def test_embed_and_gradient(T, H, V, dt, gdt, kind):
    g = gen(T + V)
    table, token = normal(g, V, H, dtype=dt), tokens_of(kind, T, V, g).to(torch.int32)
    if kind == "uniform" and T > 10:
        token[torch.rand(T, generator=g, device="cuda") < 0.1] = -5
    scale = 1.7
    cfg = moe.MoEEmbedConfig.make(T=T, H=H, V=V, act_dtype=CODE[dt], grad_dtype=CODE[gdt], scale=scale)
    ws = workspace(moe.moe_embed_workspace_size(cfg))
    s = torch.tensor(scale, dtype=FP).double().item()  # the scale as the library holds it
    keep = token >= 0
    out = poisoned(T, H, dtype=dt)
    moe.moe_embed(cfg, table, token, out, ws)
    want = torch.where(keep[:, None], table.double()[token.clamp(min=0).long()] * s, 0.0)
    within(out, want, (HALF[dt] + U) * 1.01 * want.abs())

    dout = normal(g, T, H, dtype=dt)
    dt_ = poisoned(V, H, dtype=gdt)
    moe.moe_embed_backward(cfg, token, dout, dt_, ws)
    at = token[keep].long()
    want = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, at, dout[keep].double()) * s
    mag = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, at, dout[keep].double().abs()) * s
    # at most 256 positions of a chunk in sequence, then T / 1024 (or T / 32) / 8 chunks and 8 lanes
    lost = (256 + 8 + max(T / 32 if T <= 32768 else 1024, T / 256) / 8 + 4) * U * mag
    within(dt_, want, lost + HALF[gdt] * (want.abs() + lost))
    again = torch.empty_like(dt_)
    moe.moe_embed_backward(cfg, token, dout, again, ws)
    assert torch.equal(dt_, again)
    # added to what is there; rows of tokens that do not occur are not touched
    base = normal(g, V, H, dtype=gdt)
    acc = base.clone()
    moe.moe_embed_backward(cfg, token, dout, acc, ws, accumulate=True)
    want2 = base.double() + want
    within(acc, want2, lost + HALF[gdt] * (want2.abs() + lost) + U * want2.abs())
    absent = torch.ones(V, dtype=torch.bool, device="cuda")
    absent[at] = False
    assert torch.equal(acc[absent], base[absent])
    assert moe.moe_read_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("T,V,share", [(32768, 700, 0.0), (32769, 700, 0.3), (70001, 100, 0.5), (131072, 50257, 0.02),
                                       (262145, 3, 0.1), (600000, 2000000, 0.01), (2200000, 40, 0.9), (100000, 9, 1.0)])
def test_embed_gradient_of_long_sequences(T, V, share):
    """Sorted in several steps, with `share` of the tokens left out. Small whole numbers: every sum is exact."""
    H, g = 2, gen(T)
    token = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    token[torch.rand(T, generator=g, device="cuda") < share] = -1
    dout = torch.randint(-2, 3, (T, H), generator=g, device="cuda").to(BF)
    cfg = moe.MoEEmbedConfig.make(T=T, H=H, V=V)
    ws = workspace(moe.moe_embed_workspace_size(cfg))
    dtable = poisoned(V, H, dtype=FP)
    moe.moe_embed_backward(cfg, token, dout, dtable, ws)
    keep = token >= 0
    want = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, token[keep].long(), dout[keep].double())
    assert torch.equal(dtable.double(), want)


@pytest.mark.parametrize("T", [50, 5000])
def test_embed_bad_tokens(T):
    H, V = 64, 100
    g = gen(T)
    token = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    token[3], token[T - 1] = V, 2 ** 31 - 1
    cfg = moe.MoEEmbedConfig.make(T=T, H=H, V=V)
    ws = workspace(moe.moe_embed_workspace_size(cfg))
    out, dout, d = poisoned(T, H, dtype=BF), normal(g, T, H, dtype=BF), poisoned(V, H, dtype=FP)
    moe.moe_embed(cfg, normal(g, V, H, dtype=BF), token, out, ws)
    assert moe.moe_read_status(ws) == moe.MOE_ERR_DEVICE_BAD_INPUT
    assert not bool(out[3].any()) and not bool(out[T - 1].any())
    moe.moe_embed_backward(cfg, token, dout, d, ws)
    assert moe.moe_read_status(ws) == moe.MOE_ERR_DEVICE_BAD_INPUT
    dout[3] = 0
    dout[T - 1] = 0
    token[3] = token[T - 1] = 0
    want = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, token.long(), dout.double())
    mag = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, token.long(), dout.double().abs())
    within(d, want, 300 * U * mag + U * want.abs())
    # no tokens: a zero gradient, or nothing to add
    c0 = moe.MoEEmbedConfig.make(T=0, H=H, V=V)
    moe.moe_embed_backward(c0, None, None, d, ws, accumulate=True)
    assert bool(d.any())
    moe.moe_embed_backward(c0, None, None, d, ws)
    assert not bool(d.any())


# ---------------------------------------------------------------------------------- clipping
def clip_views(sizes, dtypes, g, std=0.1, lead=1):
    """Gradients as views of one buffer per type, with `lead` guard elements around each."""
    out = []
    flat = {d: normal(g, sum(n + 2 * lead for n in sizes) + 8, dtype=d, std=std) for d in set(dtypes)}
    at = 0
    for n, d in zip(sizes, dtypes):
        out.append(flat[d][at + lead:at + lead + n])
        at += n + 2 * lead
    return flat, out


CLIP_CASES = [
    ([1], [FP], 0), ([5], [BF], 1), ([0, 7, 0], [FP, BF, FP], 1), ([8192 * 3 + 5, 1, 2, 3], [FP, BF, FP, BF], 3),
    ([100003, 70001], [BF, FP], 1), ([33] * 130, [FP, BF] * 65, 1), ([1000] * 400, [FP] * 400, 0),
    ([3_000_000, 17], [FP, FP], 0), ([5_000_000, 1_000_003, 33], [FP, FP, BF], 1)]


@pytest.mark.parametrize("sizes,dtypes,lead", CLIP_CASES)
def test_grad_norm_and_clip(sizes, dtypes, lead):
    g = gen(len(sizes) + sum(sizes))
    flat, grads = clip_views(sizes, dtypes, g, lead=lead)
    outs_flat, outs = clip_views(sizes, dtypes, g, lead=lead + 2)  # other alignments than the gradients'
    before = {d: v.clone() for d, v in flat.items()}
    guard = {d: v.clone() for d, v in outs_flat.items()}
    norm = poisoned(1, dtype=FP)
    lst = moe.MoEGradList.from_tensors(grads, outs)
    ws = workspace(moe.moe_grad_clip_workspace_size(lst))
    want = math.sqrt(sum(v.double().square().sum().item() for v in grads))
    moe.moe_grad_norm(lst, norm, ws)
    # squares and sums of 64 elements in fp32: half of 65 roundings under the root, then one
    assert abs(norm.item() - want) <= 40 * U * want
    for max_norm in (0.5 * want + 1e-30, 2 * want + 1.0):
        factor = min(1.0, max_norm / want) if want else 1.0
        moe.moe_grad_clip(lst, max_norm, norm, ws)
        for v, o in zip(grads, outs):
            if v.numel():
                w = v.double() * factor
                within(o, w, (HALF[o.dtype] + 44 * U) * 1.01 * w.abs() + 1e-40)
                if factor == 1.0:
                    assert torch.equal(o, v)
    for d, v in flat.items():
        assert torch.equal(v, before[d])       # out of place: the gradients stay
    # in place gives the same bits, and touches nothing around the views
    moe.moe_grad_clip(lst, 0.5 * want + 1e-30, norm, ws)
    inplace = moe.MoEGradList.from_tensors(grads)
    moe.moe_grad_clip(inplace, 0.5 * want + 1e-30, norm, ws)
    for v, o in zip(grads, outs):
        assert torch.equal(v, o)
    for f, saved, pad in ((flat, before, lead), (outs_flat, guard, lead + 2)):
        for d, v in f.items():
            mask = torch.ones_like(v, dtype=torch.bool)
            at = 0
            for n, k in zip(sizes, dtypes):
                if k == d:
                    mask[at + pad:at + pad + n] = False
                at += n + 2 * pad
            assert torch.equal(v[mask], saved[d][mask])
    assert moe.moe_read_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("dt", [FP, BF])
@pytest.mark.parametrize("size", [1e30, 1e-30, 2.0 ** -70])
def test_grad_norm_keeps_large_and_small_values(dt, size):
    v = (normal(gen(1), 5001) * size).to(dt)
    norm = poisoned(1, dtype=FP)
    lst = moe.MoEGradList.from_tensors([v])
    ws = workspace(moe.moe_grad_clip_workspace_size(lst))
    want = v.double().norm().item()
    moe.moe_grad_clip(lst, 1.0, norm, ws)
    assert abs(norm.item() - want) <= 40 * U * want
    assert v.double().norm().item() == pytest.approx(min(want, 1.0), rel=2 ** -8)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_grad_clip_leaves_non_finite_gradients(bad):
    v = normal(gen(1), 5001)
    v[4000] = bad
    before = v.clone()
    norm = poisoned(1, dtype=FP)
    lst = moe.MoEGradList.from_tensors([v])
    ws = workspace(moe.moe_grad_clip_workspace_size(lst))
    norm.zero_()
    moe.moe_grad_clip(lst, 1.0, norm, ws)
    assert not math.isfinite(norm.item())
    assert torch.equal(v.view(torch.int32), before.view(torch.int32))
    assert moe.moe_read_status(ws) == moe.MOE_ERR_DEVICE_BAD_INPUT
    # an empty list has norm 0; the next call on the same workspace is sound
    empty = moe.MoEGradList.from_tensors([])
    moe.moe_grad_clip(empty, 1.0, norm, ws)
    assert norm.item() == 0.0 and moe.moe_read_status(ws) == moe.MOE_OK


def test_grad_clip_of_a_norm_beyond_fp32():
    """Finite elements, a norm that fp32 does not hold: as any norm that is not finite."""
    v = torch.full((1000,), 3e38, device="cuda")
    norm = poisoned(1, dtype=FP)
    lst = moe.MoEGradList.from_tensors([v])
    ws = workspace(moe.moe_grad_clip_workspace_size(lst))
    moe.moe_grad_clip(lst, 1.0, norm, ws)
    assert norm.item() == math.inf and bool((v == 3e38).all())
    assert moe.moe_read_status(ws) == moe.MOE_ERR_DEVICE_BAD_INPUT


# ---------------------------------------------------------------------------------- streams, graphs
def test_captured_in_a_graph_on_another_stream():
    """Every call is stream-ordered and capturable: a graph of all of them, replayed on new
    inputs, gives the bits of the direct calls."""
    T, H, V = 300, 256, 1000
    g = gen(11)
    token = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    target = torch.randint(-1, V, (T,), generator=g, device="cuda").to(torch.int32)
    table, w = normal(g, V, H, dtype=BF), normal(g, H, mean=1.0, std=0.1)
    ecfg = moe.MoEEmbedConfig.make(T=T, H=H, V=V)
    ncfg = moe.MoENormConfig.make(T=T, H=H)
    hcfg = moe.MoEHeadConfig.make(T=T, H=H, V=V)
    x, n, dn, dx = (torch.empty(T, H, dtype=BF, device="cuda") for _ in range(4))
    loss, lse, mean, norm = (torch.empty(k, device="cuda") for k in (T, T, 2, 1))
    dw, dtable, dwn = torch.empty(V, H, device="cuda"), torch.empty(V, H, device="cuda"), torch.empty(H, device="cuda")
    lst = moe.MoEGradList.from_tensors([dw, dtable, dwn])
    we, wn = workspace(moe.moe_embed_workspace_size(ecfg)), workspace(moe.moe_block_norm_workspace_size(ncfg))
    wh, wc = workspace(moe.moe_head_workspace_size(hcfg)), workspace(moe.moe_grad_clip_workspace_size(lst))

    def step():
        moe.moe_embed(ecfg, table, token, x, we)
        moe.moe_block_norm(ncfg, x, None, None, w, None, n)
        moe.moe_head_loss(hcfg, n, table, target, loss, lse, mean, wh)
        moe.moe_head_loss_backward(hcfg, n, table, target, lse, dn, dw, wh, mean=mean)
        moe.moe_block_norm_backward(ncfg, x, None, None, w, None, dn, dx, None, {"dw_next": dwn}, wn)
        moe.moe_embed_backward(ecfg, token, dx, dtable, we)
        moe.moe_grad_clip(lst, 1e-3, norm, wc)

    outs = (x, n, dn, dx, loss, lse, mean, norm, dw, dtable, dwn)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for seed in (21, 22):
        token.copy_(torch.randint(0, V, (T,), generator=gen(seed), device="cuda"))
        table.copy_(normal(gen(seed), V, H, dtype=BF))
        step()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
    for ws in (we, wn, wh, wc):
        assert moe.moe_read_status(ws) == moe.MOE_OK
