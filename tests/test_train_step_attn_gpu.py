"""The example's training step with its attention block: gradients against the same model in 64 bits,
and a step captured in a graph against direct ones."""
import torch
import pytest

from test_train_step_gpu import example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_gradients_with_attention_against_64_bits(example):  # noqa: F811
    m = example.Model(T=128, seed=3, heads=4)
    tokens, targets = example.text(128, m.head.V, seed=5)
    m.d_experts["aux_loss_coeff"] = 0.0
    table0, proj0 = m.table.clone(), {n: v.clone() for n, v in m.proj.items()}
    experts0 = {n: v.clone() for n, v in m.experts.items()}
    m.step(tokens, targets, lr=0.0, max_norm=1e9)
    m.check()

    def rms(v, w):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w

    d = lambda v: v.double().requires_grad_(True)  # noqa: E731
    table, ex, proj = d(table0), {n: d(v) for n, v in experts0.items()}, {n: d(v) for n, v in proj0.items()}
    vec = {n: d(torch.ones(m.norm.H, device="cuda")) for n in m.vectors}
    x = table[tokens.long()]
    D, heads, kv = m.D, m.heads, m.kv
    qkv = (rms(x, vec["w_attn"]) @ proj["w_qkv"].t()).view(128, heads + 2 * kv, D)
    angle = m.pos.double()[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda").double() / D)

    def rope(u):
        a, b, c, s = u[..., :D // 2], u[..., D // 2:], angle.cos()[:, None], angle.sin()[:, None]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q, k, v = rope(qkv[:, :heads]), rope(qkv[:, heads:heads + kv]), qkv[:, heads + kv:]
    outs = []
    for lo, hi in zip(m.starts, m.starts[1:]):
        kk, vv = (t[lo:hi].repeat_interleave(heads // kv, 1) for t in (k, v))
        s = torch.einsum("ihd,jhd->hij", q[lo:hi], kk) / D ** 0.5
        s = s.masked_fill(torch.ones(hi - lo, hi - lo, device="cuda", dtype=torch.bool).triu(1), float("-inf"))
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), vv))
    x1 = x + torch.cat(outs).reshape(128, -1) @ proj["w_o"].t()
    n0 = rms(x1, vec["w_in"])
    top = (n0 @ ex["w_router"].t()).topk(m.layer.k, dim=1)
    weight = torch.softmax(top.values, 1)
    y = torch.zeros_like(x)
    for e in range(m.layer.E):
        h = torch.nn.functional.silu(n0 @ ex["w_gate"][e].t()) * (n0 @ ex["w_up"][e].t())
        y = y + (weight * (top.indices == e)).sum(1, keepdim=True) * (h @ ex["w_down"][e].t())
    n1 = rms(x1 + vec["gate"] * rms(y, vec["w_post"]), vec["w_out"])
    keep = targets >= 0
    loss = torch.nn.functional.cross_entropy((n1 @ table.t())[keep], targets[keep].long())
    loss.backward()
    # bf16 steps between the operators, some ten more than without the block: two dozen roundings of
    # 2^-9 each on average along the chain, compared by norm
    assert float(m.mean[0]) == pytest.approx(loss.item(), rel=4e-3)
    pairs = {"table": (m.d_table, table), **{n: (m.d_vectors[n], vec[n]) for n in vec},
             **{n: (m.d_proj[n], proj[n]) for n in proj},
             **{n: (m.d_experts["d" + n], ex[n]) for n in ("w_gate", "w_up", "w_down", "w_router")}}
    for name, (got, want) in pairs.items():
        err = ((got.double() - want.grad).norm() / want.grad.norm()).item()
        assert err < 24 * 2.0 ** -8, (name, err)


def test_step_with_attention_in_a_graph(example):  # noqa: F811
    a, b = example.Model(seed=1, heads=4), example.Model(seed=1, heads=4)
    tokens, targets = example.text(a.layer.T, a.head.V, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        b.step(tokens, targets)  # first use: function attributes are set outside the capture
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            b.step(tokens, targets)
    torch.cuda.synchronize()
    for _ in range(3):
        a.step(tokens, targets)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.table, b.table) and torch.equal(a.mean, b.mean)
    for n in a.proj:
        assert torch.equal(a.proj[n], b.proj[n]), n
    a.check()
    b.check()
