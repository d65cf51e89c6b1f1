"""The vocabulary head where its arithmetic can go wrong: tokens that the model is sure of, products of
many tiles, K stages and splits, the planes of fp32 operands.

Bounds are per element, or by norm: a value rounded to bf16 is off by at most HALF of itself and,
over many values, by HALF / sqrt(3) of their norm.
"""
import math

import pytest
import torch

import token_routing_expert_router_gb300 as moe
from test_step_gpu import BF, CODE, FP, HALF, U, gen, normal, poisoned, within, workspace

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


# ------------------------------------------------------- tiles, K stages and splits of full-size products
def plan(T, H, V, dt, piece, rows):
    """(whole tiles, splits of each further one) of the input gradient of `rows` tokens that count, by the
    library's rule; what is kept of the vocabulary at once."""
    laid_out = dt == FP or H % 8 != 0
    planes, up = 3 if laid_out else 1, lambda a, b: -(-a // b) * b  # noqa: E731
    row_bytes = 2 * planes * (up(T, 64) + (up(H, 8) if laid_out else 0))
    piece = up(min(piece or max(4096, (256 << 20) // row_bytes), V), 256)
    tm, tn = (128, 128) if T <= 128 else (256, 128 if laid_out else 256)
    units, kblocks = 152 if T <= 128 else 76, -(-min(piece, V) // 64)
    stage, part = 0.14 * tn / 256 * (6 if laid_out else 1), 0.08 * tm * tn / 65536
    tiles = -(-rows // tm) * -(-H // tn)
    tail, best = tiles % units, (kblocks * stage, 1)
    for s in range(2, 33):
        if tail and s * 4 <= kblocks and tail * s <= 4 * units:
            best = min(best, (-(-tail * s // units) * -(-kblocks // s) * stage + tail * s * part + 4.0, s))
    return (tiles - tail if best[1] > 1 else tiles), best[1], piece


SPLIT_CASES = [
    # T, H, V, dtype, piece, share left out: whole tiles first?
    (300, 256, 12000, BF, 0, 0.0, False), (2500, 2048, 12000, BF, 0, 0.0, True), (600, 1032, 20000, BF, 0, 0.0, False),
    (1500, 512, 9000, BF, 0, 0.8, False),       # the split follows the tokens that count
    (300, 256, 11876, BF, 11776, 0.0, False),   # a last piece of two K stages: splits without any
    (256, 128, 5003, FP, 0, 0.0, False), (200, 131, 6000, FP, 0, 0.0, False), (300, 131, 6000, BF, 0, 0.2, False),
    (200, 132, 4200, FP, 4096, 0.0, False),
    (70, 1032, 40000, BF, 0, 0.0, False), (128, 520, 30000, BF, 0, 0.3, False), (64, 96, 20000, FP, 0, 0.0, False)]  # single CTAs


@pytest.mark.parametrize("T,H,V,dt,piece,skip,whole", SPLIT_CASES)
def test_split_input_gradient_and_many_tiles(T, H, V, dt, piece, skip, whole):
    """Products of several tiles to a CTA pair and several K stages, the input gradient's tail of tiles split
    along K. The rows of x and of w have means, so that what is lost of a sum shows: the bounds
    are a small part of one tile's share of a token's sum, of one split's of dx, of one K stage's of dw."""
    g = gen(T + V)
    half = H // 2
    w, x = normal(g, V, H, std=0.03), normal(g, T, H)
    w[:, :half] += 0.3
    x[:, half:] += 1.0
    w, x = w.to(dt), x.to(dt)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    out = torch.rand(T, generator=g, device="cuda") < skip
    target = torch.where(out, -1, t).to(torch.int32)
    keep = ~out
    dl = torch.rand(T, generator=g, device="cuda") + 0.1
    direct, splits, kept = plan(T, H, V, dt, piece, int(keep.sum()))
    assert splits > 1 and (direct > 0) == whole

    cfg = moe.MoEHeadConfig.make(T=T, H=H, V=V, act_dtype=CODE[dt], piece=piece)
    ws = workspace(moe.moe_head_workspace_size(cfg))
    loss, lse = poisoned(T, dtype=FP), poisoned(T, dtype=FP)
    dx, dw = poisoned(T, H, dtype=dt), poisoned(V, H, dtype=FP)
    moe.moe_head_loss(cfg, x, w, target, loss, lse, None, ws)
    moe.moe_head_loss_backward(cfg, x, w, target, lse, dx, dw, ws, dloss=dl)
    assert moe.moe_read_status(ws) == moe.MOE_OK

    X, W = x[keep].double(), w.double()
    z, at = X @ W.t(), t[keep][:, None]
    wl = torch.logsumexp(z, 1)
    p = torch.exp(z - wl[:, None])
    mag = X.abs() @ W.abs().t()
    planes = dt == FP or H % 8 != 0
    # a logit: 16 products a step, each step truncated by up to two halves of U; the forward's in runs of 32
    # steps, which are added, the backward's in one; planes: runs of one stage of 64, six products each
    ez = ((64 + H / 64 if planes else H / 8) + 8) * U * mag
    el = (p * (ez if planes else (64 + H / 512 + 8) * U * mag)).sum(1) + 64 * U * (1 + wl.abs())
    within(lse[keep], wl, el)
    within(loss[keep], wl - z.gather(1, at)[:, 0], el + (H / 256 + 16) * U * mag.gather(1, at)[:, 0] + 64 * U * wl.abs())
    tile = torch.nn.functional.pad(p, (0, -V % 256)).view(p.shape[0], -1, 256).sum(2)[:, :V // 256]
    assert (el < 0.25 * tile.amin(1)).float().mean() > 0.9  # a lost tile would be seen

    D = p.scatter_add(1, at, torch.full_like(wl[:, None], -1.0)) * dl[keep].double()[:, None]
    eD = p * (ez + el[:, None] + 32 * U * (1 + z.abs()))
    eD.scatter_add_(1, at, (H / 256 + 16) * U * mag.gather(1, at) + el[:, None])
    eD *= dl[keep].double()[:, None]
    if not planes:
        eD += HALF[BF] * (D.abs() + eD)
    elif dt == BF:
        eD += 4 * U * D.abs()
    bound_x = eD @ W.abs() + (min(kept, V) / 8 + 64) * U * (D.abs() @ W.abs())
    bound_w = eD.t() @ X.abs() + (T / 8 + 64) * U * (D.abs().t() @ X.abs())
    within(dx[keep], D @ W, bound_x + HALF[dt] * ((D @ W).abs() + bound_x))
    within(dw, D.t() @ X, bound_w + U * (D.t() @ X).abs())
    assert not bool(dx[out].any())
    part = (D[:, :V // splits] @ W[:V // splits]).abs()[:, :half]
    stage = (D[:64].t() @ X[:64]).abs()[:, half:]
    # most elements would show what is lost
    assert (bound_x[:, :half] < 0.8 * part).float().mean() > 0.5 and (bound_w[:, half:] < 0.8 * stage).float().mean() > 0.5


# ------------------------------------------------------- the planes of fp32 operands
def planes_of(v):
    out, rest = [], v.float()
    for _ in range(3):
        out.append(rest.to(BF).float())
        rest = rest - out[-1]
    return [o.double() for o in out]


@pytest.mark.parametrize("i,j", [(0, 0), (0, 1), (1, 0), (0, 2), (1, 1), (2, 0)])
@pytest.mark.parametrize("T", [40, 200])
def test_each_plane_product_is_taken(T, i, j):
    """Columns whose products cancel but for one: (a - b)(c - d) with a and b alike in every plane but x's
    i-th, c and d in every plane but w's j-th. The logit of row 0 is 1, and 0 without that product."""
    level = [1.0, 1.0 + 2.0 ** -9, 1.0 + 2.0 ** -9 + 2.0 ** -18]
    pair = [(level[0], 0.0), (level[1], level[0]), (level[2], level[1])]
    (a, b), (c, d) = pair[i], pair[j]
    for v, n in ((a, i), (b, i - 1), (c, j), (d, j - 1)):
        assert [bool(q) for q in planes_of(torch.tensor([v]))] == [k <= n for k in range(3)]
    H, V, groups = 64, 100, 16
    # (a - b)(c - d) is 2^-9 for each plane past the first
    scale = 2.0 ** ((9 * (i + j) - 4) / 2 // 1)
    rest = 2.0 ** (9 * (i + j) - 4) / scale
    x = (torch.tensor([a, a, -b, -b], device="cuda") * scale).repeat(groups).expand(T, H).contiguous()
    w = torch.zeros(V, H, device="cuda")
    w[0] = (torch.tensor([c, -d, c, -d], device="cuda") * rest).repeat(groups)
    assert (x[0].double() @ w[0].double()).item() == 1.0
    cfg = moe.MoEHeadConfig.make(T=T, H=H, V=V, act_dtype=moe.F32)
    ws = workspace(moe.moe_head_workspace_size(cfg))
    target = torch.ones(T, dtype=torch.int32, device="cuda")
    loss, lse = poisoned(T, dtype=FP), poisoned(T, dtype=FP)
    dx, dw = poisoned(T, H, dtype=FP), poisoned(V, H, dtype=FP)
    moe.moe_head_loss(cfg, x, w, target, loss, lse, None, ws)
    # steps truncated by up to two halves of U of the large products that cancel: 64 of at most scale * rest
    off = 128 * U * abs(a * c) * scale * rest
    assert off < 0.2
    want = math.log(math.e + V - 1)
    within(lse, torch.full((T,), want, dtype=torch.float64, device="cuda"), 0.03 * off + 8 * U * want)
    # the same logit again in the backward: p of row 0, times x summed over the tokens
    moe.moe_head_loss_backward(cfg, x, w, target, lse, dx, dw, ws, dloss=torch.ones(T, device="cuda"))
    p = math.exp(1 - want)
    within(dw[0], T * p * x[0].double(), 1.5 * off * T * p * x[0].double().abs() + 1e-5 * x[0].double().abs())


@pytest.mark.parametrize("T,H,V", [(64, 64, 64), (64, 40, 128), (192, 64, 64), (250, 72, 128)])
def test_fp32_gradients_need_every_plane_product(T, H, V):
    """By norm the fp32 gradients are nearer to 64 bits than they would be without any one of the
    three small plane products."""
    g = gen(T + H)
    x, w = normal(g, T, H), normal(g, V, H, std=0.2)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    cfg = moe.MoEHeadConfig.make(T=T, H=H, V=V, act_dtype=moe.F32)
    ws = workspace(moe.moe_head_workspace_size(cfg))
    loss, lse = poisoned(T, dtype=FP), poisoned(T, dtype=FP)
    dx, dw = poisoned(T, H, dtype=FP), poisoned(V, H, dtype=FP)
    moe.moe_head_loss(cfg, x, w, t.to(torch.int32), loss, lse, None, ws)
    # lse in 64 bits, rounded: the error of p is then that of the logits alone
    z = x.double() @ w.double().t()
    exact = torch.logsumexp(z, 1)
    assert ((lse.double() - exact).norm() / exact.norm()).item() < 3 * U
    moe.moe_head_loss_backward(cfg, x, w, t.to(torch.int32), lse, dx, dw, ws, dloss=torch.ones(T, device="cuda"))
    D = torch.exp(z - exact[:, None]).scatter_add(1, t[:, None], torch.full((T, 1), -1.0, dtype=torch.float64, device="cuda"))
    Dp, Xp, Wp = planes_of(D), planes_of(x), planes_of(w)
    for got, want, left, right in ((dx, D @ w.double(), Dp, Wp), (dw, D.t() @ x.double(), [q.t() for q in Dp], Xp)):
        least = min((left[a] @ right[b]).norm().item() for a, b in ((0, 2), (1, 1), (2, 0)))
        assert (got.double() - want).norm().item() < 0.7 * least
