"""Cases for the attention block beside the MoE layer: rotary positions and their backward,
attention over packed prompts and over a cache, and its gradients.

Each case is run in one of two ways. With ``own`` false the operators are computed in plain
form: elementary torch operations in 32 bits (angles in 64), rounded once at the end. With
``own`` true the same inputs go through the library's entry points. ``exact`` gives the results
in 64 bits, from the definitions (gradients by differentiation of the forward definition).
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}

# Rotary positions. "T" tokens of "Hq" query and "Hk" key heads of "D" channels, of which "rot" are
# rotated from channel "first" on; "cache": K and V are stored into rows of a cache; positions up
# to "far".
ROPE = dict(op="rope", layout="half", first=0, scaling="none", cache=False, far=8192, dtype=BF16)
# Attention. "B" sequences with "T" query rows in all, spread evenly ("spread" 0) up to very
# differently (1), over "past" earlier keys each, spread the same way; "packed": q, k and v are
# views of one projection's rows; "cache": every sequence has a region of its own in a cache.
ATTN = dict(op="attn", causal=True, packed=False, cache=False, past=0, spread=0.0, dtype=BF16)


def listed():
    return [
        # one new token while serving: q and k rotated, k and v put into the cache; latency only
        dict(ROPE, name="rope_1_32x128", T=1, Hq=32, Hk=8, D=128, rot=128, cache=True),
        # a long prompt on its way into the cache
        dict(ROPE, name="rope_8192_32x128", T=8192, Hq=32, Hk=8, D=128, rot=128, cache=True),
        # the backward of a training batch
        dict(ROPE, name="rope_bwd_16384_16x128", op="rope_bwd", T=16384, Hq=16, Hk=2, D=128, rot=128),
        # a part of the head, neighbouring channels, one key head, positions scaled far beyond the trained length
        dict(ROPE, name="rope_bwd_4095_128x192_far", op="rope_bwd", T=4095, Hq=128, Hk=1, D=192, rot=64, first=128,
             layout="interleaved", scaling="yarn", far=163840),
        # one new token of one request: latency only
        dict(ATTN, name="attn_1_over_700", B=1, T=1, past=700, Hq=32, Hkv=8, D=128, cache=True),
        # one step of a busy server: a token for each of 64 requests of different lengths
        dict(ATTN, name="attn_64_over_6000", B=64, T=64, past=6000, spread=0.8, Hq=32, Hkv=8, D=128, cache=True),
        # a long prompt
        dict(ATTN, name="attn_16384", B=1, T=16384, Hq=32, Hkv=8, D=128),
        # a batch of short prompts of odd lengths, a key head for every query head
        dict(ATTN, name="attn_packed_40_prompts", B=40, T=9001, spread=0.9, Hq=12, Hkv=12, D=64, packed=True),
        # the next part of prompts that are taken in pieces
        dict(ATTN, name="attn_chunks_over_5000", B=4, T=2048, past=5000, spread=0.5, Hq=32, Hkv=8, D=128, cache=True),
        # training on packed documents, gradients in the layout of the fused projection
        dict(ATTN, name="attn_train_8192", op="attn_train", B=5, T=8192, spread=0.7, Hq=32, Hkv=8, D=128, packed=True),
        # an encoder's batch: no mask, heads of 80 channels
        dict(ATTN, name="attn_train_2001_all", op="attn_train", B=3, T=2001, spread=0.4, Hq=12, Hkv=4, D=80, causal=False),
        # the tiny fp32 layer's width and tokens
        dict(ATTN, name="attn_train_256_f32", op="attn_train", B=2, T=256, spread=0.3, Hq=4, Hkv=2, D=32, dtype=F32),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "attn", "attn", "decode", "decode", "attn_train", "attn_train"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    if op in ("rope", "rope_bwd"):
        D = rng.choice([32, 64, 72, 80, 96, 128, 192, 256])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 8, 16])
        rot = D if rng.random() < 0.5 else rng.randrange(2, D + 1, 2)
        most = 8192 * 40 * 128 // ((Hq + Hk) * D * (1 if dtype == BF16 else 2))
        return dict(ROPE, op=op, T=_log(rng, 1, min(32768, most)), Hq=Hq, Hk=Hk, D=D, rot=rot,
                    first=rng.randrange(0, D - rot + 1), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "yarn"]), cache=op == "rope" and rng.random() < 0.5,
                    far=_log(rng, 1000, 1_000_000), dtype=dtype)
    D = rng.choice([32, 64, 64, 80, 96, 128, 128, 128]) if dtype == BF16 else rng.choice([16, 32, 50, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    spread = rng.random()
    if op == "decode":
        Hq = Hkv * rng.choice([1, 2, 4, 8, 16])
        B = _log(rng, 1, 128)
        new = rng.choice([1, 1, 1, 2, 4])
        cost = Hkv * D * (1 if dtype == BF16 else 8 * Hq // Hkv)  # fp32 scores are not formed by tensor cores
        return dict(ATTN, B=B, T=B * new, past=_log(rng, 16, min(65536, 64 * 6000 * 8 * 128 // (B * cost))),
                    spread=0.0 if new > 1 else spread, Hq=Hq, Hkv=Hkv, D=D, cache=True, dtype=dtype)
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    # at most the work of the listed long prompt or training batch
    most = (16384 ** 2 * 32 * 128 if op == "attn" else 8192 ** 2 * 32 * 128 // 4) // (1 if dtype == BF16 else 64)
    longest = int(math.sqrt(most / (Hq * D)))
    B = _log(rng, 1, 64)
    T = max(B, _log(rng, 32, min(16384, max(64, longest))))
    past = _log(rng, 100, max(100, min(8192, longest))) if op == "attn" and rng.random() < 0.3 else 0
    if past:
        T = max(B, min(T, most // (Hq * D * (past + T))))
    return dict(ATTN, op=op, B=B, T=T, past=past, spread=spread, Hq=Hq, Hkv=Hkv, D=D, causal=rng.random() < 0.8,
                packed=not past and rng.random() < 0.5, cache=past > 0, dtype=dtype)


def _lengths(case):
    """Query rows and keys of every sequence: fixed by the case's numbers, the same for every seed."""
    rng = random.Random(f"{case['B']} {case['T']} {case['past']} {case['spread']:.6f} {case['D']}")
    B, T = case["B"], case["T"]
    share = [math.exp(2.5 * case["spread"] * rng.uniform(-1, 1)) for _ in range(B)]
    new = [1 + int((T - B) * s / sum(share)) for s in share]
    for i in range(T - sum(new)):
        new[i % B] += 1
    past = [max(0, int(case["past"] * (1 + case["spread"] * rng.uniform(-1, 1)))) for _ in range(B)]
    return new, [p + n for p, n in zip(past, new)]


def _pairs(case):
    """Visible (query, key) pairs of one head, over every sequence."""
    total = 0
    for n, m in zip(*_lengths(case)):
        total += n * m - (n * (n - 1) // 2 if case["causal"] else 0)
    return total


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _frequencies(case):
    """Radians per position of every pair of channels, in 64 bits on the host."""
    rot = case["rot"]
    f = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        f = [v / 4.0 for v in f]
    elif case["scaling"] == "yarn":
        # whole turns within the trained length: from 32 on kept, up to 1 divided by the factor
        keep = [min(1.0, max(0.0, (4096 * v / (2 * math.pi) - 1.0) / (32.0 - 1.0))) for v in f]
        f = [v * k + v / 40.0 * (1.0 - k) for v, k in zip(f, keep)]
    return f


def _magnitude(case):
    return 0.1 * math.log(40.0) + 1.0 if case["scaling"] == "yarn" else 1.0


def prepare(case, seed):
    g, op, dt = _gen(seed), case["op"], DTYPES[case["dtype"]]
    s = {"case": case, "op": op}
    if op in ("rope", "rope_bwd"):
        T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
        # one projection's rows: the query heads, the key heads, the value heads
        row = _normal(g, T, Hq + 2 * Hk, D, dtype=dt)
        s["q"], s["k"], s["v"] = row[:, :Hq], row[:, Hq:Hq + Hk], row[:, Hq + Hk:]
        # the far end of a long text, or anywhere in it
        start = torch.randint(0, max(1, case["far"] - T), (1,), generator=g, device="cuda")
        s["pos"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
        s["qo"] = torch.empty(T, Hq, D, device="cuda", dtype=dt)
        s["slot"] = None
        rows = T
        if case["cache"]:
            rows = T + 64
            s["slot"] = torch.randperm(rows, generator=g, device="cuda")[:T].to(torch.int32)
        s["ko"] = torch.zeros(rows, Hk, D, device="cuda", dtype=dt)
        s["vo"] = torch.zeros(rows, Hk, D, device="cuda", dtype=dt) if case["cache"] else None
        if op == "rope_bwd":
            # the gradients of the rotated heads come dense and go into the projection's rows
            s["gq"], s["gk"] = _normal(g, T, Hq, D, dtype=dt, std=0.1), _normal(g, T, Hk, D, dtype=dt, std=0.1)
            row = torch.empty_like(row)
            s["dq"], s["dk"] = row[:, :Hq], row[:, Hq:Hq + Hk]
    else:
        B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
        new, keys = _lengths(case)
        T = sum(new)
        at = [0]
        for n in new:
            at.append(at[-1] + n)
        s["new"], s["keys"], s["at"] = new, keys, at
        s["q_start"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        if case["cache"]:
            region = max(keys) + 13
            s["first"] = [b * region for b in range(B)]
            s["k_start"] = torch.tensor(s["first"], dtype=torch.int32, device="cuda")
            s["k_len"] = torch.tensor(keys, dtype=torch.int32, device="cuda")
            rows = B * region
        else:
            s["first"], s["k_start"], s["k_len"], rows = at[:-1], None, None, T
        # heads differ in how sharply they attend
        sharp = torch.rand(Hq, 1, generator=g, device="cuda") * 2.0 + 0.3
        q = torch.randn(T, Hq, D, generator=g, device="cuda") * sharp
        if case["packed"]:
            row = torch.empty(T, Hq + 2 * Hkv, D, device="cuda", dtype=dt)
            row[:, :Hq] = q
            row[:, Hq:] = torch.randn(T, 2 * Hkv, D, generator=g, device="cuda")
            s["q"], s["k"], s["v"] = row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = q.to(dt), _normal(g, rows, Hkv, D, dtype=dt), _normal(g, rows, Hkv, D, dtype=dt)
        s["scale"] = 1.0 / math.sqrt(D)
        s["o"] = torch.empty(T, Hq, D, device="cuda", dtype=dt)
        s["lse"] = torch.empty(Hq, T, device="cuda")
        if op == "attn_train":
            s["do"] = _normal(g, T, Hq, D, dtype=dt)
            if case["packed"]:
                row = torch.empty(T, Hq + 2 * Hkv, D, device="cuda", dtype=dt)
                s["dq"], s["dk"], s["dv"] = row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:]
            else:
                s["dq"], s["dk"], s["dv"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    if own:
        _prepare_own(s)
    elif op in ("rope", "rope_bwd"):
        s["freq"] = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
    return s


def _prepare_own(s):
    """What a user of the library keeps from call to call: the configuration, a workspace, and
    for rotary positions the table of frequencies."""
    import token_routing_expert_router_gb300 as moe

    case, op = s["case"], s["op"]
    code = {BF16: moe.BF16, F32: moe.F32}[case["dtype"]]
    if op in ("rope", "rope_bwd"):
        scaling = {"none": dict(), "linear": dict(scaling=moe.ROPE_LINEAR, factor=4.0),
                   "yarn": dict(scaling=moe.ROPE_YARN, factor=40.0, trained_len=4096)}[case["scaling"]]
        freq = moe.MoERopeFreq.make(rot=case["rot"], base=10000.0, **scaling)
        s["table"] = torch.empty(max(1, case["rot"] // 2), dtype=torch.int64, device="cuda")
        moe.moe_rope_table(freq, s["table"])
        row = (case["Hq"] + 2 * case["Hk"]) * case["D"]
        s["cfg"] = moe.MoERopeConfig.make(
            T=case["T"], Hq=case["Hq"], Hk=case["Hk"], D=case["D"], rot=case["rot"], first=case["first"],
            layout={"half": moe.ROPE_HALF, "interleaved": moe.ROPE_INTERLEAVED}[case["layout"]], act_dtype=code,
            slots=s["ko"].shape[0], magnitude=_magnitude(case), ld_q=row, ld_k=row, ld_v=row)
        size = moe.WORKSPACE_HEAD
    else:
        row = (case["Hq"] + 2 * case["Hkv"]) * case["D"] if case["packed"] else 0
        s["cfg"] = moe.MoEAttnConfig.make(
            Tq=s["q"].shape[0], Tk=s["k"].shape[0], B=case["B"], Hq=case["Hq"], Hkv=case["Hkv"], D=case["D"],
            causal=int(case["causal"]), max_q=max(s["new"]), act_dtype=code, scale=s["scale"], ld_q=row, ld_k=row, ld_v=row)
        size = moe.moe_attn_workspace_size(s["cfg"])
        if op == "attn_train":
            size = max(size, moe.moe_attn_backward_workspace_size(s["cfg"]))
    s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(s["ws"])


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import token_routing_expert_router_gb300 as moe

    op = s["op"]
    if op == "rope":
        moe.moe_rope(s["cfg"], s["q"], s["k"], s["v"] if s["vo"] is not None else None, s["pos"], s["slot"], s["table"],
                     s["qo"], s["ko"], s["vo"], s["ws"])
        return {"q": s["qo"], "k": s["ko"], "v": s["vo"]}
    if op == "rope_bwd":
        moe.moe_rope_backward(s["cfg"], s["gq"], s["gk"], s["pos"], s["table"], s["dq"], s["dk"])
        return {"dq": s["dq"], "dk": s["dk"]}
    moe.moe_attn(s["cfg"], s["q"], s["k"], s["v"], s["q_start"], s["k_start"], s["k_len"], s["o"], s["lse"], s["ws"])
    out = {"o": s["o"], "lse": s["lse"]}
    if op == "attn_train":
        moe.moe_attn_backward(s["cfg"], s["q"], s["k"], s["v"], s["q_start"], s["k_start"], s["k_len"], s["o"], s["lse"],
                              s["do"], s["dq"], s["dk"], s["dv"], s["ws"])
        out.update(dq=s["dq"], dk=s["dk"], dv=s["dv"])
    return out


def _angles(s):
    """cos and sin of every position and pair, [T, 1, rot / 2]; the angles in 64 bits."""
    a = (s["pos"].double()[:, None] * s["freq"])[:, None, :]
    return a.cos().float(), a.sin().float()


def _turn(s, x, sign):
    case, (c, d) = s["case"], _angles(s)
    first, rot, m = case["first"], case["rot"], _magnitude(case)
    y = x.float().clone()
    part = y[..., first:first + rot]
    half = case["layout"] == "half"
    a, b = (part[..., :rot // 2], part[..., rot // 2:]) if half else (part[..., 0::2], part[..., 1::2])
    u, v = m * (a * c - sign * b * d), m * (b * c + sign * a * d)
    y[..., first:first + rot] = torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)
    return y.to(x.dtype)


def _masked(s, n, m):
    """Which keys a query row may not see: the last query sees every key."""
    if not s["case"]["causal"]:
        return None
    i, j = torch.arange(n, device="cuda"), torch.arange(m, device="cuda")
    return j[None, :] > i[:, None] + (m - n)


def _attend(s, b, kv, out):
    """Sequence b and the kv heads `kv` (a slice), in 32 bits, into `out`."""
    case = s["case"]
    G, D = case["Hq"] // case["Hkv"], case["D"]
    rows, first = slice(s["at"][b], s["at"][b + 1]), s["first"][b]
    n, m = s["new"][b], s["keys"][b]
    heads = slice(kv.start * G, kv.stop * G)
    k = s["k"][first:first + m, kv].float().transpose(0, 1)
    v = s["v"][first:first + m, kv].float().transpose(0, 1)

    def grouped(x):  # [n, heads, D] -> [kv heads, G * n, D]
        return x[rows, heads].float().permute(1, 0, 2).reshape(-1, G * n, D)

    def back(x):
        return x.reshape(-1, n, D).permute(1, 0, 2)

    q = grouped(s["q"])
    z = (q @ k.transpose(1, 2)) * s["scale"]
    mask = _masked(s, n, m)
    if mask is not None:
        z.view(-1, G, n, m).masked_fill_(mask, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = (z - top).exp_()
    total = p.sum(-1, keepdim=True)
    p /= total
    o = p @ v
    out["o"][rows, heads] = back(o).to(out["o"].dtype)
    out["lse"][heads, rows] = (top + total.log()).reshape(-1, n)
    if s["op"] == "attn_train":
        do = grouped(s["do"])
        out["dv"][first:first + m, kv] = (p.transpose(1, 2) @ do).transpose(0, 1).to(out["dv"].dtype)
        ds = p * (do @ v.transpose(1, 2) - (do * o).sum(-1, keepdim=True)) * s["scale"]
        out["dq"][rows, heads] = back(ds @ k).to(out["dq"].dtype)
        out["dk"][first:first + m, kv] = (ds.transpose(1, 2) @ q).transpose(0, 1).to(out["dk"].dtype)


def _run_plain(s):
    case, op = s["case"], s["op"]
    if op == "rope":
        q, k = _turn(s, s["q"], 1.0), _turn(s, s["k"], 1.0)
        if s["slot"] is None:
            return {"q": q, "k": k, "v": None}
        s["ko"][s["slot"].long()] = k
        s["vo"][s["slot"].long()] = s["v"]
        return {"q": q, "k": s["ko"], "v": s["vo"]}
    if op == "rope_bwd":
        return {"dq": _turn(s, s["gq"], -1.0), "dk": _turn(s, s["gk"], -1.0)}
    out = {"o": torch.empty_like(s["o"]), "lse": torch.empty_like(s["lse"])}
    if op == "attn_train":
        out.update({n: torch.empty_like(s[n]) for n in ("dq", "dk", "dv")})
    Hkv, G = case["Hkv"], case["Hq"] // case["Hkv"]
    for b in range(case["B"]):
        # as many heads at once as 2 GB of scores hold
        step = max(1, min(Hkv, (1 << 29) // (G * s["new"][b] * s["keys"][b])))
        for h in range(0, Hkv, step):
            _attend(s, b, slice(h, min(Hkv, h + step)), out)
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] in ("rope", "rope_bwd"):
        return _exact_rope(case, s)
    new, keys = s["new"], s["keys"]
    flops = 4.0 * sum(n * m for n, m in zip(new, keys)) * case["Hq"] * case["D"]
    if flops * (3.5 if case["op"] == "attn_train" else 1.0) > 1.2e13:
        return None
    train = case["op"] == "attn_train"
    names = ("q", "k", "v")
    x = {n: s[n].double() for n in names}
    out = {"o": torch.zeros_like(x["q"]), "lse": torch.zeros(case["Hq"], x["q"].shape[0], dtype=torch.float64, device="cuda")}
    if train:
        out.update({"d" + n: torch.zeros_like(x[n]) for n in names})
    for b in range(case["B"]):
        lo, hi, k0, m = s["at"][b], s["at"][b + 1], s["first"][b], keys[b]
        for h in range(case["Hq"]):
            kv = h * case["Hkv"] // case["Hq"]
            q, k, v = (t.clone().requires_grad_(train) for t in
                       (x["q"][lo:hi, h], x["k"][k0:k0 + m, kv], x["v"][k0:k0 + m, kv]))
            score = torch.einsum("id,jd->ij", q, k) / math.sqrt(case["D"])
            if case["causal"]:
                hidden = torch.ones(hi - lo, m, dtype=torch.bool, device="cuda").triu(m - (hi - lo) + 1)
                score = score.masked_fill(hidden, -math.inf)
            o = torch.softmax(score, 1) @ v
            out["o"][lo:hi, h] = o.detach()
            out["lse"][h, lo:hi] = torch.logsumexp(score.detach(), 1)
            if train:
                (o * s["do"][lo:hi, h].double()).sum().backward()
                out["dq"][lo:hi, h] = q.grad
                out["dk"][k0:k0 + m, kv] += k.grad
                out["dv"][k0:k0 + m, kv] += v.grad
    return out


def _exact_rope(case, s):
    """Channel pairs as complex numbers, multiplied by m exp(i angle) (the backward: by its conjugate)."""
    i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / max(1, case["rot"])
    f = torch.exp(-math.log(10000.0) * i)
    m = 1.0
    if case["scaling"] == "linear":
        f = f / 4.0
    elif case["scaling"] == "yarn":
        ramp = ((4096.0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f / 40.0 * (1.0 - ramp) + f * ramp
        m = 1.0 + 0.1 * math.log(40.0)
    angle = (s["pos"].double().unsqueeze(1) * f).unsqueeze(1)
    turn = torch.polar(torch.full_like(angle, m), angle)
    first, rot = case["first"], case["rot"]

    def apply(x, by):
        y = x.double()
        part = y[..., first:first + rot]
        if case["layout"] == "half":
            z = torch.complex(part[..., :rot // 2].contiguous(), part[..., rot // 2:].contiguous()) * by
            part = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(part.reshape(*part.shape[:-1], rot // 2, 2).contiguous()) * by
            part = torch.view_as_real(z).reshape(part.shape)
        return torch.cat([y[..., :first], part, y[..., first + rot:]], -1)

    if case["op"] == "rope_bwd":
        return {"dq": apply(s["gq"], turn.conj()), "dk": apply(s["gk"], turn.conj())}
    q, k, v = apply(s["q"], turn), apply(s["k"], turn), None
    if case["cache"]:
        rows = s["slot"].long()
        k = torch.zeros(s["ko"].shape, dtype=torch.float64, device="cuda").index_copy_(0, rows, k)
        v = torch.zeros(s["vo"].shape, dtype=torch.float64, device="cuda").index_copy_(0, rows, s["v"].double())
    return {"q": q, "k": k, "v": v}


def work(case):
    e = {BF16: 2, F32: 4}[case["dtype"]]
    if case["op"] in ("rope", "rope_bwd"):
        T, D = case["T"], case["D"]
        heads = case["Hq"] + case["Hk"] * (2 if case["cache"] else 1)
        return {"bytes": 2 * T * heads * D * e + 4 * T * (2 if case["cache"] else 1),
                "flops": 3.0 * T * (case["Hq"] + case["Hk"]) * case["rot"]}
    new, keys = _lengths(case)
    T, K, Hq, Hkv, D = sum(new), sum(keys), case["Hq"], case["Hkv"], case["D"]
    pairs = _pairs(case)
    once = (2 * T * Hq + 2 * K * Hkv) * D * e + 4 * T * Hq
    if case["op"] == "attn":
        return {"bytes": once, "flops": 4.0 * pairs * Hq * D}
    # forward and backward: the output's gradient read, three gradients written; seven products
    return {"bytes": once + (2 * T * Hq + 2 * K * Hkv) * D * e, "flops": 14.0 * pairs * Hq * D}
