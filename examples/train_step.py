"""One-layer MoE language model, trained for a few steps on made-up text, with every part of a
step in the library's kernels: token embedding, block norms around the MoE layer, the vocabulary
head's cross entropy, the backward of each, and clipping by the global gradient norm. PyTorch
supplies memory and the plain SGD update.

    x  = embed(tokens)                       n0 = norm(x)
    y  = moe(n0)                             r  = x + gate * norm(y),  n1 = norm(r)   (one pass)
    loss = cross entropy(n1, table)          (the table is shared with the embedding)

With query heads the layer stands behind an attention block: rotary positions, causal attention over
packed documents and their backward are the library's, the two projections PyTorch's matrix products:

    q, k, v = norm(x) w_qkv,  q, k = rope(q, k)
    x <- x + attention(q, k, v) w_o          (in the pass that forms n0)

    python examples/train_step.py [steps [heads]]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import token_routing_expert_router_gb300 as moe  # noqa: E402


class Model:
    """bf16 parameters, fp32 gradients, one workspace per operator; T tokens a step. heads: query
    heads of an attention block in front of the layer, two to a key head (0: none)."""

    def __init__(self, T=512, H=256, E=8, k=2, F=512, V=2000, seed=0, heads=0, D=64):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        bf, f32 = dict(device="cuda", dtype=torch.bfloat16), dict(device="cuda", dtype=torch.float32)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.layer = moe.MoEConfig.make(T=T, H=H, E=E, k=k, F=F, score_fn=moe.SOFTMAX, renorm=1)
        self.norm = moe.MoENormConfig.make(T=T, H=H)
        self.embed = moe.MoEEmbedConfig.make(T=T, H=H, V=V)
        self.head = moe.MoEHeadConfig.make(T=T, H=H, V=V)
        self.table = normal(V, H, std=0.05)
        self.experts = {"w_router": normal(E, H, std=0.02), "w_gate": normal(E, F, H, std=0.05),
                        "w_up": normal(E, F, H, std=0.05), "w_down": normal(E, H, F, std=0.05)}
        self.vectors = {"w_in": torch.ones(H, **f32), "w_post": torch.ones(H, **f32), "w_out": torch.ones(H, **f32),
                        "gate": torch.ones(H, **f32)}

        self.heads, self.D = heads, D
        if heads:
            self.kv, self.width = max(1, heads // 2), (heads + 2 * max(1, heads // 2)) * D
            self.proj = {"w_qkv": normal(self.width, H, std=0.05), "w_o": normal(H, heads * D, std=0.05)}
            self.vectors["w_attn"] = torch.ones(H, **f32)
            # documents of different lengths, one behind the other; positions count in each
            self.starts = sorted({0, T // 2 + 1, T // 2 + T // 3, T - 1, T})
            self.q_start = torch.tensor(self.starts, device="cuda", dtype=torch.int32)
            self.pos = torch.cat([torch.arange(b - a, device="cuda", dtype=torch.int32)
                                  for a, b in zip(self.starts, self.starts[1:])])
            row = dict(ld_q=self.width, ld_k=self.width, ld_v=self.width)
            self.attn = moe.MoEAttnConfig.make(Tq=T, Tk=T, B=len(self.starts) - 1, Hq=heads, Hkv=self.kv, D=D, **row)
            self.rope = moe.MoERopeConfig.make(T=T, Hq=heads, Hk=self.kv, D=D, ld_q=self.width, ld_k=self.width,
                                               ld_q_out=self.width, ld_k_out=self.width)
            self.turns = torch.empty(D // 2, device="cuda", dtype=torch.int64)
            moe.moe_rope_table(moe.MoERopeFreq.make(rot=D), self.turns)

        self.d_table = torch.empty(V, H, **f32)
        self.d_experts = {"dw_gate": torch.empty(E, F, H, **f32), "dw_up": torch.empty(E, F, H, **f32),
                          "dw_down": torch.empty(E, H, F, **f32), "dw_router": torch.empty(E, H, **f32),
                          "aux_loss_coeff": 0.01}
        self.d_vectors = {n: torch.empty(H, **f32) for n in self.vectors}
        grads = [self.d_table, *(v for v in self.d_experts.values() if torch.is_tensor(v)), *self.d_vectors.values()]
        params = [self.table, self.experts["w_gate"], self.experts["w_up"], self.experts["w_down"],
                  self.experts["w_router"], *self.vectors.values()]
        if heads:
            self.d_proj = {n: torch.empty(w.shape, **f32) for n, w in self.proj.items()}
            grads += self.d_proj.values()
            params += self.proj.values()
        self.updates = list(zip(params, grads))
        self.grads = moe.MoEGradList.from_tensors(grads)  # clipped in place

        rows = lambda: torch.empty(T, H, **bf)  # noqa: E731
        self.x, self.n0, self.y, self.r, self.n1 = rows(), rows(), rows(), rows(), rows()
        self.dn1, self.dr, self.dy, self.dn0, self.dx = rows(), rows(), rows(), rows(), rows()
        self.gu, self.dtopk = torch.empty(T * k, 2 * F, **bf), torch.empty(T, k, **f32)
        self.loss, self.lse, self.mean = torch.empty(T, **f32), torch.empty(T, **f32), torch.empty(2, **f32)
        self.aux, self.grad_norm = torch.empty(1, **f32), torch.empty(1, **f32)

        if heads:
            self.na, self.y0, self.x1, self.dx1, self.dy0, self.dna = (rows() for _ in range(6))
            self.qkv, self.dqkv = torch.empty(T, heads + 2 * self.kv, D, **bf), torch.empty(T, heads + 2 * self.kv, D, **bf)
            self.o, self.do = torch.empty(T, heads, D, **bf), torch.empty(T, heads, D, **bf)
            self.attn_lse = torch.empty(heads, T, **f32)

        def workspace(size):
            ws = torch.empty(size, device="cuda", dtype=torch.uint8)
            moe.moe_workspace_init(ws)
            return ws

        self.ws_layer = workspace(moe.moe_forward_workspace_size(self.layer))
        self.ws_back = workspace(moe.moe_backward_workspace_size(self.layer))
        self.ws_norm = workspace(moe.moe_block_norm_workspace_size(self.norm))
        self.ws_embed = workspace(moe.moe_embed_workspace_size(self.embed))
        self.ws_head = workspace(moe.moe_head_workspace_size(self.head))
        self.ws_clip = workspace(moe.moe_grad_clip_workspace_size(self.grads))
        self.spaces = [self.ws_layer, self.ws_back, self.ws_norm, self.ws_embed, self.ws_head, self.ws_clip]
        if heads:
            self.ws_attn = workspace(max(moe.moe_attn_workspace_size(self.attn), moe.moe_attn_backward_workspace_size(self.attn)))
            self.spaces.append(self.ws_attn)

    def split(self, qkv):
        return qkv[:, :self.heads], qkv[:, self.heads:self.heads + self.kv], qkv[:, self.heads + self.kv:]

    def attention(self):
        """x -> x1 = x + attention, and n0 = norm(x1)."""
        v = self.vectors
        q, k, val = self.split(self.qkv)
        moe.moe_block_norm(self.norm, self.x, None, None, v["w_attn"], None, self.na)
        torch.mm(self.na, self.proj["w_qkv"].t(), out=self.qkv.view(len(self.na), -1))
        moe.moe_rope(self.rope, q, k, None, self.pos, None, self.turns, q, k, None)
        moe.moe_attn(self.attn, q, k, val, self.q_start, None, None, self.o, self.attn_lse, self.ws_attn)
        torch.mm(self.o.view(len(self.o), -1), self.proj["w_o"].t(), out=self.y0)
        moe.moe_block_norm(self.norm, self.x, self.y0, None, v["w_in"], self.x1, self.n0)

    def attention_backward(self):
        """dr (of x1) and dn0 -> dx (of x), and the block's own gradients."""
        v, dv = self.vectors, self.d_vectors
        T = len(self.x)
        moe.moe_block_norm_backward(self.norm, self.x1, self.y0, None, v["w_in"], self.dr, self.dn0, self.dx1, self.dy0,
                                    {"dw_next": dv["w_in"]}, self.ws_norm)
        torch.mm(self.dy0, self.proj["w_o"], out=self.do.view(T, -1))
        torch.mm(self.dy0.t().float(), self.o.view(T, -1).float(), out=self.d_proj["w_o"])
        (q, k, val), (dq, dk, dval) = self.split(self.qkv), self.split(self.dqkv)
        moe.moe_attn_backward(self.attn, q, k, val, self.q_start, None, None, self.o, self.attn_lse, self.do, dq, dk, dval,
                              self.ws_attn)
        moe.moe_rope_backward(self.rope, dq, dk, self.pos, self.turns, dq, dk)
        dqkv = self.dqkv.view(T, -1)
        torch.mm(dqkv.t().float(), self.na.float(), out=self.d_proj["w_qkv"])
        torch.mm(dqkv, self.proj["w_qkv"], out=self.dna)
        moe.moe_block_norm_backward(self.norm, self.x, None, None, v["w_attn"], self.dx1, self.dna, self.dx, None,
                                    {"dw_next": dv["w_attn"]}, self.ws_norm)

    def step(self, tokens, targets, lr=0.3, max_norm=1.0):
        """One training step, stream-ordered; self.mean[0] is the loss, self.grad_norm the norm."""
        v, dv = self.vectors, self.d_vectors
        # forward
        moe.moe_embed(self.embed, self.table, tokens, self.x, self.ws_embed)
        if self.heads:
            self.attention()
        else:
            moe.moe_block_norm(self.norm, self.x, None, None, v["w_in"], None, self.n0)
        x = self.x1 if self.heads else self.x
        moe.moe_forward_train(self.layer, self.n0, self.experts, self.y, self.ws_layer, self.gu, aux_alpha=0.01,
                              aux_loss=self.aux)
        moe.moe_block_norm(self.norm, x, self.y, v["w_post"], v["w_out"], self.r, self.n1, gate=v["gate"])
        moe.moe_head_loss(self.head, self.n1, self.table, targets, self.loss, self.lse, self.mean, self.ws_head)
        # backward
        moe.moe_head_loss_backward(self.head, self.n1, self.table, targets, self.lse, self.dn1, self.d_table,
                                   self.ws_head, mean=self.mean)
        moe.moe_block_norm_backward(self.norm, self.r, self.y, v["w_post"], v["w_out"], None, self.dn1, self.dr, self.dy,
                                    {"dw_post": dv["w_post"], "dw_next": dv["w_out"], "dgate": dv["gate"]},
                                    self.ws_norm, gate=v["gate"])
        moe.moe_backward_kept(self.layer, self.n0, self.experts, self.dy, self.ws_layer, self.gu, self.dn0, self.dtopk,
                              self.d_experts, self.ws_back)
        if self.heads:
            self.attention_backward()
        else:
            moe.moe_block_norm_backward(self.norm, self.x, None, None, v["w_in"], self.dr, self.dn0, self.dx, None,
                                        {"dw_next": dv["w_in"]}, self.ws_norm)
        # the table's second share joins the head's
        moe.moe_embed_backward(self.embed, tokens, self.dx, self.d_table, self.ws_embed, accumulate=True)
        moe.moe_grad_clip(self.grads, max_norm, self.grad_norm, self.ws_clip)
        for param, grad in self.updates:
            param.add_(grad, alpha=-lr)

    def check(self):
        for ws in self.spaces:
            status = moe.moe_read_status(ws)
            if status != moe.MOE_OK:
                raise moe.MoEError(status, "train_step")


def text(T, V, seed):
    """Made-up text that can be learnt: every token's successor is fixed but for one in ten."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    follows = torch.randperm(V, generator=g, device="cuda")
    g.manual_seed(seed)
    tokens = (V ** torch.rand(T, generator=g, device="cuda")).long().clamp_(max=V - 1)
    noise = torch.randint(0, V, (T,), generator=g, device="cuda")
    targets = torch.where(torch.rand(T, generator=g, device="cuda") < 0.1, noise, follows[tokens])
    targets[: T // 16] = -1  # a prompt that is not trained on
    return tokens.to(torch.int32), targets.to(torch.int32)


def main(steps=200, heads=0):
    model = Model(heads=heads)
    losses = []
    for i in range(steps):
        tokens, targets = text(model.layer.T, model.head.V, seed=100 + i)
        model.step(tokens, targets)
        if i % 20 == 0 or i == steps - 1:
            losses.append(float(model.mean[0]))
            print(f"step {i:4d}  loss {losses[-1]:.4f}  aux {float(model.aux):.4f}  grad norm {float(model.grad_norm):.3f}")
    model.check()
    return losses


if __name__ == "__main__":
    moe.build()
    main(*(int(v) for v in sys.argv[1:3]))
