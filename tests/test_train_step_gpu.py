"""The example's training step: its loss falls, its gradients are those of the same model written
in 64 bits, and a step captured in a graph gives the bits of a direct one."""
import importlib.util
import os

import pytest
import torch

import token_routing_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(lib):
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_loss_falls(example):
    losses = example.main(steps=61)
    # from log(2000) = 7.6: the frequent tokens' successors are learnt within some dozens of steps
    assert losses[0] == pytest.approx(7.6, abs=0.3)
    assert losses[-1] < losses[0] - 1.0


def test_gradients_against_64_bits(example):
    m = example.Model(T=128, seed=3)
    tokens, targets = example.text(128, m.head.V, seed=5)
    m.d_experts["aux_loss_coeff"] = 0.0
    table0 = m.table.clone()
    experts0 = {n: v.clone() for n, v in m.experts.items()}
    m.step(tokens, targets, lr=0.0, max_norm=1e9)
    m.check()

    def rms(v, w):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w

    d = lambda v: v.double().requires_grad_(True)  # noqa: E731
    table, ex = d(table0), {n: d(v) for n, v in experts0.items()}
    vec = {n: d(torch.ones(m.norm.H, device="cuda")) for n in m.vectors}
    x = table[tokens.long()]
    n0 = rms(x, vec["w_in"])
    logits = n0 @ ex["w_router"].t()
    top = logits.topk(m.layer.k, dim=1)
    weight = torch.softmax(top.values, 1)
    y = torch.zeros_like(x)
    for e in range(m.layer.E):
        h = torch.nn.functional.silu(n0 @ ex["w_gate"][e].t()) * (n0 @ ex["w_up"][e].t())
        share = (weight * (top.indices == e)).sum(1, keepdim=True)
        y = y + share * (h @ ex["w_down"][e].t())
    r = x + vec["gate"] * rms(y, vec["w_post"])
    n1 = rms(r, vec["w_out"])
    keep = targets >= 0
    loss = torch.nn.functional.cross_entropy((n1 @ table.t())[keep], targets[keep].long())
    loss.backward()
    # bf16 steps between the operators: a dozen roundings of 2^-9 each on average along the chain,
    # compared by norm
    assert float(m.mean[0]) == pytest.approx(loss.item(), rel=2e-3)
    pairs = {"table": (m.d_table, table), **{n: (m.d_vectors[n], vec[n]) for n in vec},
             "gate": (m.d_vectors["gate"], vec["gate"]),
             **{n: (m.d_experts["d" + n], ex[n]) for n in ("w_gate", "w_up", "w_down", "w_router")}}
    for name, (got, want) in pairs.items():
        err = ((got.double() - want.grad).norm() / want.grad.norm()).item()
        assert err < 12 * 2.0 ** -8, (name, err)
    total = torch.sqrt(sum(w.grad.square().sum() for _, w in pairs.values()))
    assert float(m.grad_norm) == pytest.approx(total.item(), rel=12 * 2.0 ** -8)


def test_step_in_a_graph(example):
    a, b = example.Model(seed=1), example.Model(seed=1)
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
    for n in a.experts:
        assert torch.equal(a.experts[n], b.experts[n]), n
    a.check()
    b.check()
