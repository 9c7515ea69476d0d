"""A small recurrent language model, trained and then served token by token with the library's
operators: the gated delta rule and the channel scan as mixers, the gated feed-forward block after
each, and linear cross entropy as the loss.

    python examples/recurrent_lm.py            # trains for a few hundred steps, then generates

The remaining projections, norms and the optimizer are plain torch. The data is synthetic: each
sequence follows next = (a * token + c) mod V with its own a and c drawn from a handful, so that the
model has to look back to tell which.
"""
from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gated_delta_rule_70_amd import binding  # noqa: E402

DT = torch.bfloat16


class ChannelScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, a, b, A_log, dt_bias):
        out, _, states = binding.channel_scan_fwd(x, a, b, A_log, dt_bias, want_state=False, want_states=True)
        ctx.save_for_backward(x, a, b, A_log, dt_bias, states)
        return out

    @staticmethod
    def backward(ctx, dout):
        return binding.channel_scan_bwd(*ctx.saved_tensors, dout.contiguous(), want_dh0=False)[:5]


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_alpha, beta):
        out, _ = binding.chunk_fwd(q, k, v, log_alpha, beta, want_state=False)
        ctx.save_for_backward(q, k, v, log_alpha, beta)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, log_alpha, beta = ctx.saved_tensors
        dq, dk, dv, dla, dbeta, _ = binding.chunk_bwd(q, k, v, log_alpha, beta, dout.contiguous())
        return dq.to(q.dtype), dk.to(k.dtype), dv.to(v.dtype), dla, dbeta


class GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up):
        h, gate, up = binding.gated_ffn_fwd(x, w_gate, w_up, want_saved=True)
        ctx.save_for_backward(x, w_gate, w_up, gate, up)
        return h

    @staticmethod
    def backward(ctx, dh):
        return binding.gated_ffn_bwd(*ctx.saved_tensors, dh.contiguous())


class LinearCe(torch.autograd.Function):
    """The mean loss over the tokens whose target is in the vocabulary."""

    @staticmethod
    def forward(ctx, x, weight, targets):
        loss, lse = binding.linear_ce_fwd(x, weight, targets)
        scale = 1.0 / ((targets >= 0) & (targets < weight.shape[0])).sum().clamp(min=1)
        ctx.save_for_backward(x, weight, targets, lse, scale)
        return loss.sum() * scale

    @staticmethod
    def backward(ctx, g):
        x, weight, targets, lse, scale = ctx.saved_tensors
        dx, dw = binding.linear_ce_bwd(x, weight, targets, lse, (g * scale).float().expand_as(lse).contiguous())
        return dx, dw, None


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Model:
    def __init__(self, vocab=509, width=256, heads=4, hidden=704, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def w(*shape, std=None):
            t = torch.randn(*shape, generator=g) * (shape[-1] ** -0.5 if std is None else std)
            return t.to(device).requires_grad_()

        self.heads, self.head = heads, width // heads
        self.master = dict(embed=w(vocab, width, std=1.0), head=w(vocab, width))
        for i, kind in enumerate(("delta", "scan")):
            wide = 3 * width + 2 * heads if kind == "delta" else 3 * width
            self.master.update({"%s.in" % kind: w(wide, width), "%s.out" % kind: w(width, width),
                                "%s.gate" % kind: w(hidden, width), "%s.up" % kind: w(hidden, width),
                                "%s.down" % kind: w(width, hidden)})
        self.master["scan.A_log"] = torch.log(1.0 + 15.0 * torch.rand(width, generator=g)).to(device).requires_grad_()
        self.master["scan.dt_bias"] = torch.full((width,), -5.0, device=device).requires_grad_()
        self.p = {}

    def cast(self):
        """Weights in the compute type for one step (matrices in bf16, scan parameters in fp32)."""
        self.p = {k: v if v.dim() == 1 else v.to(DT) for k, v in self.master.items()}

    # ------------------------------------------------------------------ mixers over whole sequences

    def delta_inputs(self, x):
        """q, k (unit rows), v, log alpha, beta in the library's head-major layouts; x [B, T, width]."""
        B, T, D = x.shape
        y = F.linear(x, self.p["delta.in"])
        q, k, v, a, b = y.split([D, D, D, self.heads, self.heads], -1)
        heads = lambda t: t.reshape(B, T, self.heads, -1).transpose(1, 2).contiguous()
        q, k, v = heads(q), heads(k), heads(v)
        q, k = (F.normalize(t.float(), dim=-1).to(DT) for t in (q, k))
        la = -F.softplus(a.float() - 4.0).transpose(1, 2).contiguous()
        return q, k, v, la, torch.sigmoid(b.float()).transpose(1, 2).contiguous()

    def scan_inputs(self, x):
        return [t.contiguous() for t in F.linear(x, self.p["scan.in"]).chunk(3, -1)]

    def ffn(self, x, kind):
        return x + F.linear(GatedFfn.apply(norm(x), self.p[kind + ".gate"], self.p[kind + ".up"]), self.p[kind + ".down"])

    def hidden(self, tokens):
        x = F.embedding(tokens, self.p["embed"])
        B, T, D = x.shape
        o = DeltaRule.apply(*self.delta_inputs(norm(x)))
        x = self.ffn(x + F.linear(o.transpose(1, 2).reshape(B, T, D), self.p["delta.out"]), "delta")
        o = ChannelScan.apply(*self.scan_inputs(norm(x)), self.p["scan.A_log"], self.p["scan.dt_bias"])
        x = self.ffn(x + F.linear(o, self.p["scan.out"]), "scan")
        return norm(x)

    def loss(self, tokens):
        h = self.hidden(tokens[:, :-1].contiguous())
        return LinearCe.apply(h.reshape(-1, h.shape[-1]), self.p["head"], tokens[:, 1:].reshape(-1))

    # ------------------------------------------------------------------ one token at a time

    def start(self, N, device="cuda"):
        width = self.heads * self.head
        return dict(delta=torch.zeros(N, self.heads, self.head, self.head, device=device),
                    scan=torch.zeros(N, width, device=device))

    @torch.no_grad()
    def step(self, tokens, state):
        """The final hidden row of each of N sequences after one more token; the states in place."""
        x = F.embedding(tokens, self.p["embed"])
        q, k, v, la, beta = (t.squeeze(2).contiguous() for t in self.delta_inputs(norm(x)[:, None]))
        o, _ = binding.decode_step(q, k, v, la, beta, state["delta"], state["delta"])
        x = self.ffn(x + F.linear(o.reshape(x.shape), self.p["delta.out"]), "delta")
        o, _ = binding.channel_scan_step(*self.scan_inputs(norm(x)), self.p["scan.A_log"], self.p["scan.dt_bias"],
                                         state["scan"], state["scan"])
        return norm(self.ffn(x + F.linear(o, self.p["scan.out"]), "scan"))


def batch(B, T, vocab, g, device="cuda"):
    rules = torch.tensor([[3, 7], [5, 11], [2, 1], [7, 3]])
    r = rules[torch.randint(0, len(rules), (B,), generator=g)]
    t = torch.zeros(B, T, dtype=torch.int64)
    t[:, 0] = torch.randint(0, vocab, (B,), generator=g)
    for i in range(1, T):
        t[:, i] = (r[:, 0] * t[:, i - 1] + r[:, 1]) % vocab
    return t.to(device)


def train(model, steps, B=16, T=129, lr=2e-3, seed=1, say=None):
    g = torch.Generator().manual_seed(seed)
    vocab = model.master["head"].shape[0]
    opt = torch.optim.AdamW(model.master.values(), lr=lr, weight_decay=0.0)
    losses = []
    for i in range(steps):
        model.cast()
        loss = model.loss(batch(B, T, vocab, g))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if say and (i + 1) % 50 == 0:
            say("step %4d loss %.3f" % (i + 1, loss.item()))
    model.cast()
    return [x.item() for x in losses]


@torch.no_grad()
def score_both_ways(model, tokens):
    """Each token's loss after its prefix: from whole sequences, and one token at a time."""
    h = model.hidden(tokens[:, :-1].contiguous())
    B, T, D = h.shape
    whole = binding.linear_ce_fwd(h.reshape(-1, D), model.p["head"], tokens[:, 1:].reshape(-1))[0].view(B, T)
    state, cols = model.start(B), []
    for i in range(T):
        row = model.step(tokens[:, i].contiguous(), state)
        cols.append(binding.linear_ce_fwd(row, model.p["head"], tokens[:, i + 1].contiguous())[0])
    return whole, torch.stack(cols, 1)


@torch.no_grad()
def generate(model, prompt, n):
    state, out = model.start(prompt.shape[0]), [prompt]
    for i in range(prompt.shape[1]):
        row = model.step(prompt[:, i].contiguous(), state)
    for _ in range(n):
        nxt = F.linear(row, model.p["head"]).float().argmax(-1)
        out.append(nxt[:, None])
        row = model.step(nxt, state)
    return torch.cat(out, 1)


def main(steps=300):
    model = Model()
    losses = train(model, steps, say=lambda m: print(m, flush=True))
    print("loss %.3f -> %.3f" % (losses[0], losses[-1]))
    test = batch(4, 65, model.master["head"].shape[0], torch.Generator().manual_seed(99))
    whole, stepped = score_both_ways(model, test)
    print("mean loss of unseen sequences: %.3f in one pass, %.3f token by token" % (whole.mean().item(), stepped.mean().item()))
    made = generate(model, test[:, :16], 16)
    print("generated tokens that follow their sequence's rule: %d of %d" % ((made[:, 16:] == test[:, 16:32]).sum().item(), 4 * 16))


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 300)
