"""Cases for the operators around the MoE layer in one training or serving step: the block
norms, the vocabulary head's cross entropy, the token embedding and the clipping of the
gradients by their global norm.

Each case is run in one of two ways. With ``own`` false the operators are computed in plain
form: elementary torch operations in 32 bits (the gradients' long sum of squares in 64),
rounded once at the end. With ``own`` true the same inputs go through the library's entry
points. ``exact`` gives the results in 64 bits, from the definitions (the gradients by
differentiation of the forward definition, not by the formulas of the plain form).
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-6

# Norms. "T" tokens of "H" channels; "post": the block output is normalised before it joins
# the residual; "gate" / "token_gate": it is scaled per channel / per token; "next": the
# next block's norm of the new residual is formed in the same call.
NORM = dict(post=True, gate=True, token_gate=False, next=True)


def listed():
    return [
        # one token of a DeepSeek-V3-shaped layer while serving: latency only
        dict(NORM, name="norm_1x7168", op="norm", T=1, H=7168, dtype=BF16, gate=False),
        # the same layer's prompt or training forward, every part of the norm in use
        dict(NORM, name="norm_8192x7168", op="norm", T=8192, H=7168, dtype=BF16),
        # training backward at the imbalanced 128-expert layer's shape, with both gates
        dict(NORM, name="norm_bwd_16384x2048", op="norm_bwd", T=16384, H=2048, dtype=BF16, token_gate=True),
        # an fp32 layer with an odd width and an odd number of tokens
        dict(NORM, name="norm_bwd_777x1001_f32", op="norm_bwd", T=777, H=1001, dtype=F32),
        # scoring a few answers against a large vocabulary: the head's weights are read once
        dict(name="head_32x4096x131072", op="head", T=32, H=4096, V=131072, dtype=BF16, ignore=0.0),
        # the head of a Mixtral-shaped model in training: loss, input gradient, weight gradient
        dict(name="head_train_4096x4096x32000", op="head_train", T=4096, H=4096, V=32000, dtype=BF16, ignore=0.03),
        # a ragged batch against an odd vocabulary, most of it prompt that is not trained on
        dict(name="head_train_1500x2048x50257", op="head_train", T=1500, H=2048, V=50257, dtype=BF16, ignore=0.6),
        # the tiny fp32 layer's width
        dict(name="head_train_256x128x5003_f32", op="head_train", T=256, H=128, V=5003, dtype=F32, ignore=0.1),
        # the tokens of one serving step
        dict(name="embed_16x7168", op="embed", T=16, H=7168, V=129280, dtype=BF16, grad=F32, zipf=1.0, ignore=0.0),
        # the embedding's gradient for a training batch of natural text: a few tokens are very frequent
        dict(name="embed_bwd_16384x2048", op="embed_bwd", T=16384, H=2048, V=32000, dtype=BF16, grad=F32, zipf=1.0,
             ignore=0.02),
        # every gradient of the imbalanced 128-expert layer, clipped before the optimiser
        dict(name="clip_moe_layer", op="clip", count=6, total=604_045_312, dtype=F32, align=True),
        # many small gradients of both types, taken as views of one flat buffer (odd offsets)
        dict(name="clip_48_views", op="clip", count=48, total=3_000_001, dtype="mixed", align=False),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    return n + 1 if n == 3 * 1024 else n


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "head", "head_train", "embed", "embed_bwd", "clip"])
    dtype = rng.choice([BF16, BF16, F32])
    if op in ("norm", "norm_bwd"):
        H = _log(rng, 64, 8192)
        H = H if rng.random() < 0.3 else -(-H // 8) * 8
        H = H + 8 if H == 3 * 1024 else H
        return dict(op=op, T=_log(rng, 1, min(16384, 8192 * 7168 // H)), H=H, dtype=dtype, post=rng.random() < 0.7,
                    gate=rng.random() < 0.5, token_gate=rng.random() < 0.5, next=rng.random() < 0.7)
    if op in ("head", "head_train"):
        # at most the work of the Mixtral-shaped case; fp32 takes smaller ones
        H = -(-_log(rng, 64, 7168 if dtype == BF16 else 1024) // 8) * 8
        H = H + 8 if H == 3 * 1024 else H
        V = _log(rng, 500, 131072 if dtype == BF16 else 16384)
        most = 4096 * 4096 * 32000 // (1 if dtype == BF16 else 60)
        return dict(op=op, T=_log(rng, 1, max(1, min(8192, most // (H * V)))), H=H, V=V, dtype=dtype,
                    ignore=rng.choice([0.0, 0.05, 0.5]))
    if op in ("embed", "embed_bwd"):
        H, V = _log(rng, 64, 7168), _log(rng, 500, 131072)
        H = H if rng.random() < 0.3 else -(-H // 8) * 8
        H = H + 8 if H == 3 * 1024 else H
        return dict(op=op, T=_log(rng, 1, min(32768, 16384 * 7168 // H)), H=H, V=V, dtype=dtype,
                    grad=rng.choice([F32, dtype]), zipf=rng.choice([0.0, 0.7, 1.0, 1.3]), ignore=rng.choice([0.0, 0.1]))
    return dict(op="clip", count=rng.randint(1, 60), total=_log(rng, 1000, 300_000_000),
                dtype=rng.choice([F32, BF16, "mixed"]), align=rng.random() < 0.5)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).add_(mean).to(dtype)


def _clip_sizes(case):
    """Element counts of the gradients: geometric, so that a few hold most of the elements (a
    layer's expert weights) and the rest are small (its norms, router and biases)."""
    n, total = case["count"], case["total"]
    share = [0.75 ** i for i in range(n)]
    sizes = [max(1, int(total * s / sum(share))) for s in share]
    return [s // 8 * 8 or 8 for s in sizes] if case["align"] else [s | 1 for s in sizes]


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case, "op": op}
    dt = DTYPES.get(case["dtype"])
    if op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        s["x"] = _normal(g, T, H, dtype=dt, std=2.0)            # the residual stream (in _bwd: the new one)
        s["y"] = _normal(g, T, H, dtype=dt, std=0.7)            # the block's output
        s["w_post"] = _normal(g, H, std=0.2, mean=1.0) if case["post"] else None
        s["w_next"] = _normal(g, H, std=0.2, mean=1.0) if case["next"] else None
        s["gate"] = _normal(g, H, std=0.3, mean=0.5) if case["gate"] else None
        s["token_gate"] = torch.rand(T, generator=g, device="cuda") if case["token_gate"] else None
        s["res_scale"] = 0.875
        if op == "norm":
            s["r"] = torch.empty(T, H, device="cuda", dtype=dt)
            s["n"] = torch.empty(T, H, device="cuda", dtype=dt) if case["next"] else None
        else:
            s["dr"] = _normal(g, T, H, dtype=dt, std=0.1)
            s["dn"] = _normal(g, T, H, dtype=dt, std=0.1) if case["next"] else None
            s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
            s["grads"] = {"dw_post": torch.empty_like(s["w_post"]) if case["post"] else None,
                          "dw_next": torch.empty_like(s["w_next"]) if case["next"] else None,
                          "dgate": torch.empty_like(s["gate"]) if case["gate"] else None,
                          "dtoken_gate": torch.empty_like(s["token_gate"]) if case["token_gate"] else None}
    elif op in ("head", "head_train"):
        T, H, V = case["T"], case["H"], case["V"]
        s["w"] = _normal(g, V, H, dtype=dt, std=0.02)
        t = torch.randint(0, V, (T,), generator=g, device="cuda")
        # a trained model's states lean towards their target, by an amount that varies by token
        lean = torch.rand(T, 1, generator=g, device="cuda") * (12.0 / (0.02 * H))
        s["x"] = (_normal(g, T, H) + lean * s["w"][t].float() / 0.02).to(dt)
        skip = torch.rand(T, generator=g, device="cuda") < case["ignore"]
        s["target"] = torch.where(skip, -1, t).to(torch.int32)
        f = dict(device="cuda", dtype=torch.float32)
        s["loss"], s["lse"] = torch.empty(T, **f), torch.empty(T, **f)
        s["mean"] = torch.empty(2, **f)
        if op == "head_train":
            s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
    elif op in ("embed", "embed_bwd"):
        T, H, V = case["T"], case["H"], case["V"]
        # ranks with probability ~ 1 / rank^zipf by the continuous inverse, ids permuted over the vocabulary
        u, z = torch.rand(T, generator=g, device="cuda", dtype=torch.float64), case["zipf"]
        rank = (V + 1.0) ** u if z == 1.0 else (1.0 + u * ((V + 1.0) ** (1 - z) - 1.0)) ** (1.0 / (1 - z))
        rank = (rank.long() - 1).clamp_(0, V - 1)
        t = torch.randperm(V, generator=g, device="cuda")[rank]
        skip = torch.rand(T, generator=g, device="cuda") < case["ignore"]
        s["token"] = torch.where(skip, -1, t).to(torch.int32)
        s["scale"] = math.sqrt(H)
        if op == "embed":
            s["table"] = _normal(g, V, H, dtype=dt, std=0.02)
            s["out"] = torch.empty(T, H, device="cuda", dtype=dt)
        else:
            s["dout"] = _normal(g, T, H, dtype=dt, std=0.01)
            s["dtable"] = torch.empty(V, H, device="cuda", dtype=DTYPES[case["grad"]])
    else:
        sizes = _clip_sizes(case)
        kinds = [torch.float32 if case["dtype"] == F32 or (case["dtype"] == "mixed" and i % 3) else torch.bfloat16
                 for i in range(len(sizes))]
        flat = {k: _normal(g, sum(n for n, d in zip(sizes, kinds) if d == k), dtype=k, std=0.03) for k in set(kinds)}
        out = {k: torch.empty_like(v) for k, v in flat.items()}
        at = {k: 0 for k in flat}
        s["grads"], s["outs"] = [], []
        for n, k in zip(sizes, kinds):
            s["grads"].append(flat[k][at[k]:at[k] + n])
            s["outs"].append(out[k][at[k]:at[k] + n])
            at[k] += n
        s["max_norm"] = 1.0
        s["norm"] = torch.empty(1, device="cuda")
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a user of the library keeps from call to call: the configuration and a workspace."""
    import token_routing_expert_router_gb300 as moe

    case, op = s["case"], s["op"]
    code = {BF16: moe.BF16, F32: moe.F32}
    if op in ("norm", "norm_bwd"):
        s["cfg"] = moe.MoENormConfig.make(T=case["T"], H=case["H"], act_dtype=code[case["dtype"]], eps=EPS,
                                          res_scale=s["res_scale"])
        size = moe.moe_block_norm_workspace_size(s["cfg"])
    elif op in ("head", "head_train"):
        s["cfg"] = moe.MoEHeadConfig.make(T=case["T"], H=case["H"], V=case["V"], act_dtype=code[case["dtype"]],
                                          grad_dtype=code[case["dtype"]])
        size = moe.moe_head_workspace_size(s["cfg"])
    elif op in ("embed", "embed_bwd"):
        s["cfg"] = moe.MoEEmbedConfig.make(T=case["T"], H=case["H"], V=case["V"], act_dtype=code[case["dtype"]],
                                           grad_dtype=code[case["grad"]], scale=s["scale"])
        size = moe.moe_embed_workspace_size(s["cfg"])
    else:
        s["list"] = moe.MoEGradList.from_tensors(s["grads"], s["outs"])
        size = moe.moe_grad_clip_workspace_size(s["list"])
    s["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(s["ws"])


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import token_routing_expert_router_gb300 as moe

    op = s["op"]
    if op == "norm":
        moe.moe_block_norm(s["cfg"], s["x"], s["y"], s["w_post"], s["w_next"], s["r"], s["n"], gate=s["gate"],
                           token_gate=s["token_gate"])
        return {"r": s["r"], "n": s["n"]}
    if op == "norm_bwd":
        moe.moe_block_norm_backward(s["cfg"], s["x"], s["y"], s["w_post"], s["w_next"], s["dr"], s["dn"], s["dx"],
                                    s["dy"], s["grads"], s["ws"], gate=s["gate"], token_gate=s["token_gate"])
        return {"dx": s["dx"], "dy": s["dy"], **s["grads"]}
    if op == "head":
        moe.moe_head_loss(s["cfg"], s["x"], s["w"], s["target"], s["loss"], s["lse"], s["mean"], s["ws"])
        return {"loss": s["loss"], "lse": s["lse"], "mean": s["mean"]}
    if op == "head_train":
        moe.moe_head_loss(s["cfg"], s["x"], s["w"], s["target"], s["loss"], s["lse"], s["mean"], s["ws"])
        moe.moe_head_loss_backward(s["cfg"], s["x"], s["w"], s["target"], s["lse"], s["dx"], s["dw"], s["ws"],
                                   mean=s["mean"])
        return {"loss": s["loss"], "lse": s["lse"], "mean": s["mean"], "dx": s["dx"], "dw": s["dw"]}
    if op == "embed":
        moe.moe_embed(s["cfg"], s["table"], s["token"], s["out"], s["ws"])
        return s["out"]
    if op == "embed_bwd":
        moe.moe_embed_backward(s["cfg"], s["token"], s["dout"], s["dtable"], s["ws"])
        return s["dtable"]
    moe.moe_grad_clip(s["list"], s["max_norm"], s["norm"], s["ws"])
    return {"norm": s["norm"], "grads": s["outs"]}


def _rms(v):
    """1 / sqrt(mean of squares + eps) of every row."""
    return (v.square().mean(1, keepdim=True) + EPS).rsqrt()


def _gates(s):
    """The product of the gates that a case has, or 1."""
    gate = 1.0 if s["gate"] is None else s["gate"]
    return gate if s["token_gate"] is None else gate * s["token_gate"][:, None]


def _run_plain(s):
    op, dt = s["op"], DTYPES.get(s["case"]["dtype"])
    if op == "norm":
        x, y = s["x"].float(), s["y"].float()
        u = y if s["w_post"] is None else y * _rms(y) * s["w_post"]
        r = s["res_scale"] * x + _gates(s) * u
        n = None if s["w_next"] is None else (r * _rms(r) * s["w_next"]).to(dt)
        return {"r": r.to(dt), "n": n}
    if op == "norm_bwd":
        r, y, dr = s["x"].float(), s["y"].float(), s["dr"].float()
        dw_post = dw_next = dgate = dtoken = None
        if s["w_next"] is not None:
            dn, rho = s["dn"].float(), _rms(r)
            nh = r * rho
            a = dn * s["w_next"]
            dr = dr + rho * (a - nh * (a * nh).mean(1, keepdim=True))
            dw_next = (dn * nh).sum(0)
        rho = 1.0 if s["w_post"] is None else _rms(y)
        yh = y * rho
        u = yh if s["w_post"] is None else yh * s["w_post"]
        if s["gate"] is not None:
            dgate = (dr * u if s["token_gate"] is None else dr * u * s["token_gate"][:, None]).sum(0)
        if s["token_gate"] is not None:
            dtoken = (dr * u if s["gate"] is None else dr * u * s["gate"]).sum(1)
        dy = dr * _gates(s)
        if s["w_post"] is not None:
            dw_post = (dy * yh).sum(0)
            a = dy * s["w_post"]
            dy = rho * (a - yh * (a * yh).mean(1, keepdim=True))
        return {"dx": (s["res_scale"] * dr).to(dt), "dy": dy.to(dt), "dw_post": dw_post, "dw_next": dw_next,
                "dgate": dgate, "dtoken_gate": dtoken}
    if op in ("head", "head_train"):
        x, w = s["x"].float(), s["w"].float()
        z = x @ w.t()
        m = z.amax(1, keepdim=True)
        lse = m + (z - m).exp().sum(1, keepdim=True).log()
        keep = s["target"] >= 0
        at = s["target"].clamp(min=0).long()[:, None]
        loss = torch.where(keep, (lse - z.gather(1, at))[:, 0], 0.0)
        inv = torch.where(keep.any(), 1.0 / keep.sum(), 0.0)
        out = {"loss": loss, "lse": lse[:, 0], "mean": torch.stack([loss.sum() * inv, inv])}
        if op == "head_train":
            dz = (z - lse).exp()
            dz.scatter_add_(1, at, torch.full_like(lse, -1.0))
            dz *= (keep * inv)[:, None]
            out.update(dx=(dz @ w).to(dt), dw=(dz.t() @ x).to(dt))
        return out
    if op == "embed":
        keep = s["token"] >= 0
        rows = s["table"][s["token"].clamp(min=0).long()].float()
        return torch.where(keep[:, None], rows * s["scale"], 0.0).to(dt)
    if op == "embed_bwd":
        keep = s["token"] >= 0
        rows = torch.where(keep[:, None], s["dout"].float(), 0.0)
        d = torch.zeros(s["dtable"].shape, device="cuda")
        d.index_add_(0, s["token"].clamp(min=0).long(), rows)
        return (d * s["scale"]).to(s["dtable"].dtype)
    squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]])
    norm = squares.sum().sqrt()
    scale = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0).float()
    return {"norm": norm.float()[None], "grads": [(g.float() * scale).to(g.dtype) for g in s["grads"]]}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = s["op"]
    d = lambda v: None if v is None else v.detach().to(torch.float64).requires_grad_(True)  # noqa: E731
    if op in ("norm", "norm_bwd"):
        def rms_norm(v, w):
            return v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS) * w

        w_post, w_next, gate, token = d(s["w_post"]), d(s["w_next"]), d(s["gate"]), d(s["token_gate"])
        y = d(s["y"])
        branch = y if w_post is None else rms_norm(y, w_post)
        branch = branch if gate is None else branch * gate
        branch = branch if token is None else branch * token.unsqueeze(1)
        if op == "norm":
            r = s["x"].double() * s["res_scale"] + branch
            return {"r": r.detach(), "n": None if w_next is None else rms_norm(r, w_next).detach()}
        # the new residual is given: differentiate around it
        x = ((s["x"].double() - branch.detach()) / s["res_scale"]).requires_grad_(True)
        r = x * s["res_scale"] + branch
        total = (r * s["dr"].double()).sum()
        if w_next is not None:
            total = total + (rms_norm(r, w_next) * s["dn"].double()).sum()
        total.backward()
        grad = lambda v: None if v is None else v.grad  # noqa: E731
        return {"dx": x.grad, "dy": y.grad, "dw_post": grad(w_post), "dw_next": grad(w_next), "dgate": grad(gate),
                "dtoken_gate": grad(token)}
    if op in ("head", "head_train"):
        x, w = d(s["x"]), d(s["w"])
        logp = torch.log_softmax(x @ w.t(), 1)
        keep = (s["target"] >= 0).nonzero()[:, 0]
        picked = -logp[keep, s["target"][keep].long()]
        loss = torch.zeros(case["T"], dtype=torch.float64, device="cuda").index_put((keep,), picked)
        count = keep.numel()
        mean = loss.sum() / count if count else loss.sum() * 0.0
        lse = ((x * w[0]).sum(1) - logp[:, 0]).detach()
        out = {"loss": loss.detach(), "lse": lse,
               "mean": torch.stack([mean.detach(), torch.tensor(1.0 / count if count else 0.0, dtype=torch.float64,
                                                                device="cuda")])}
        if op == "head_train":
            mean.backward()
            out.update(dx=x.grad, dw=w.grad)
        return out
    if op == "embed":
        keep = s["token"] >= 0
        out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        out[keep] = s["table"][s["token"][keep].long()].double() * s["scale"]
        return out
    if op == "embed_bwd":
        keep = (s["token"] >= 0).nonzero()[:, 0]
        out = torch.zeros(case["V"], case["H"], dtype=torch.float64, device="cuda")
        return out.index_add_(0, s["token"][keep].long(), s["dout"][keep].double()).mul_(s["scale"])
    squares = sum(g.double().pow(2).sum() for g in s["grads"])
    norm = squares.sqrt()
    scale = min(1.0, s["max_norm"] / float(norm))
    return {"norm": norm[None], "grads": [g.double() * scale for g in s["grads"]]}


def work(case):
    op, size = case["op"], {BF16: 2, F32: 4}
    if op in ("norm", "norm_bwd"):
        T, H, e = case["T"], case["H"], size[case["dtype"]]
        vectors = 4 * H * (case["post"] + case["next"] + case["gate"]) + 4 * T * case["token_gate"]
        if op == "norm":
            return {"bytes": T * H * e * (3 + case["next"]) + vectors, "flops": 10.0 * T * H}
        return {"bytes": T * H * e * (5 + case["next"]) + 2 * vectors, "flops": 25.0 * T * H}
    if op in ("head", "head_train"):
        T, H, V, e = case["T"], case["H"], case["V"], size[case["dtype"]]
        if op == "head":
            return {"bytes": (T + V) * H * e + 12 * T, "flops": 2.0 * T * H * V}
        # the products of the logits, the input gradient and the weight gradient; the logits
        # are not kept, so a pass forms them twice, but the work counts them once
        return {"bytes": 2 * (T + V) * H * e + 12 * T, "flops": 6.0 * T * H * V}
    if op == "embed":
        return {"bytes": 2 * case["T"] * case["H"] * size[case["dtype"]] + 4 * case["T"], "flops": case["T"] * case["H"]}
    if op == "embed_bwd":
        T, H, V = case["T"], case["H"], case["V"]
        return {"bytes": T * H * size[case["dtype"]] + V * H * size[case["grad"]] + 4 * T, "flops": T * H}
    sizes = _clip_sizes(case)
    if case["dtype"] == "mixed":
        bytes_ = sum(n * (4 if i % 3 else 2) for i, n in enumerate(sizes))
    else:
        bytes_ = sum(sizes) * size[case["dtype"]]
    return {"bytes": 2 * bytes_, "flops": 3.0 * sum(sizes)}
