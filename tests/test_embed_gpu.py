"""The embedding's gradient where one token takes a large share of the positions."""
import pytest
import torch

import token_routing_expert_router_gb300 as moe
from test_step_gpu import BF, FP, gen, poisoned, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(lib):
    pass


def gradient(token, dout, V):
    T, H = dout.shape
    cfg = moe.MoEEmbedConfig.make(T=T, H=H, V=V)
    ws, dtable = workspace(moe.moe_embed_workspace_size(cfg)), poisoned(V, H, dtype=FP)
    return dtable, lambda: moe.moe_embed_backward(cfg, token, dout, dtable, ws)


def microseconds(call):
    times = []
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        times.append(1000 * a.elapsed_time(b))
    return min(times[3:])


def test_time_does_not_follow_the_most_frequent_token():
    """The rows of zeros are found without a walk over every position of a token: half of a million
    positions of one token take at most half as long again as a million spread ones."""
    T, H, V, g = 1 << 20, 8, 50000, gen(1)
    dout = torch.randint(-2, 3, (T, H), generator=g, device="cuda").to(BF)
    spread = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    hot = torch.where(torch.rand(T, generator=g, device="cuda") < 0.5, V // 3, spread).to(torch.int32)
    base = microseconds(gradient(spread, dout, V)[1])
    taken = microseconds(gradient(hot, dout, V)[1])
    print(f"spread {base:.0f} us, one token in half of the positions {taken:.0f} us")
    assert taken < 1.5 * base


@pytest.mark.parametrize("T,V,hot", [(1, 300, [0]), (256, 300, [0]), (257, 300, [299]), (5000, 300, [7]), (5000, 300, [0, 1, 2]),
                                     (5000, 700, [255, 256]), (40000, 5000, [31, 32, 33, 4999]), (20000, 70, list(range(0, 70, 2))),
                                     (70000, 400, [399])])
@pytest.mark.parametrize("rest", [0.0, 0.01])
def test_rows_of_zeros_around_frequent_tokens(T, V, hot, rest):
    """Small whole numbers: every sum is exact, and a row that was taken for absent or present would show."""
    H, g = 8, gen(T + V)
    pick = torch.tensor(hot, device="cuda")[torch.randint(0, len(hot), (T,), generator=g, device="cuda")]
    other = torch.randint(0, V, (T,), generator=g, device="cuda")
    token = torch.where(torch.rand(T, generator=g, device="cuda") < rest, other, pick).to(torch.int32)
    dout = torch.randint(1, 3, (T, H), generator=g, device="cuda").to(BF)
    dtable, call = gradient(token, dout, V)
    call()
    want = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, token.long(), dout.double())
    assert torch.equal(dtable.double(), want)
