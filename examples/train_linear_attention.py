"""A one-layer language model on linear attention with a decay for each head: trained for a
few steps on synthetic sequences, then run as it would be served, a prompt and then token by
token.

    python examples/train_linear_attention.py [--steps 60] [--io bf16]

The mixer (linattn_fwd / linattn_bwd / linattn_step), the gated norm of its heads
(group_norm_fwd / group_norm_bwd) and the gradients' clipping (clip_grad_norm) are the
library's; projections, loss and optimizer are torch's.  Decays are learned: log_decay =
-softplus(raw).  The task: every sequence repeats one of eight patterns of 16 tokens, from a
random place in it.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_66_amd as ssm  # noqa: E402


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay):
        ctx.save_for_backward(q, k, v, log_decay)
        return ssm.linattn_fwd(q, k, v, log_decay, return_last_state=False)[0]

    @staticmethod
    def backward(ctx, do):
        g = ssm.linattn_bwd(*ctx.saved_tensors, do.contiguous())
        return g["dq"], g["dk"], g["dv"], g["dlog_decay"]


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, weight, groups):
        y, mean, rstd = ssm.group_norm_fwd(x, groups, weight=weight, z=z)
        ctx.save_for_backward(x, z, weight, mean, rstd)
        ctx.groups = groups
        return y

    @staticmethod
    def backward(ctx, dy):
        x, z, weight, mean, rstd = ctx.saved_tensors
        g = ssm.group_norm_bwd(x, ctx.groups, dy.contiguous(), mean, rstd, weight=weight, z=z)
        return g["dx"], g["dz"], g["dweight"], None


class Model(torch.nn.Module):
    def __init__(self, vocab=32, dim=128, heads=4, dk=64, dv=64, io=torch.bfloat16):
        super().__init__()
        self.heads, self.dk, self.dv, self.io = heads, dk, dv, io
        # the current token and the one before it, as a short convolution would give them
        self.embed = torch.nn.Parameter(0.5 * torch.randn(2, vocab, dim))
        self.proj = torch.nn.Parameter(torch.randn(dim, heads * (2 * dk + 2 * dv)) * dim ** -0.5)
        self.out = torch.nn.Parameter(torch.randn(heads * dv, dim) * (heads * dv) ** -0.5)
        self.head = torch.nn.Parameter(torch.randn(dim, vocab) * dim ** -0.5)
        self.norm = torch.nn.Parameter(torch.ones(heads * dv))
        self.raw_decay = torch.nn.Parameter(torch.linspace(-4.0, -2.0, heads))

    def log_decay(self):
        return -F.softplus(self.raw_decay)

    def split(self, tokens, before):
        """q, k (.., heads, dk), v (.., heads, dv) and the gate z (.., heads * dv)."""
        x = self.embed[0][tokens] + self.embed[1][before]
        h, dk, dv = self.heads, self.dk, self.dv
        q, k, v, z = (x @ self.proj).to(self.io).split([h * dk, h * dk, h * dv, h * dv], -1)
        lead = tokens.shape
        return (x, q.reshape(*lead, h, dk).contiguous(), k.reshape(*lead, h, dk).contiguous(),
                v.reshape(*lead, h, dv).contiguous(), z.contiguous())

    def logits(self, x, o, z, normed=None):
        """o and z: (rows, 1, heads * dv), every token an entry of the norm."""
        y = GatedNorm.apply(o, z, self.norm, self.heads) if normed is None else normed
        return (x.reshape(-1, x.shape[-1]) + y.reshape(-1, y.shape[-1]).float() @ self.out) @ self.head

    def forward(self, tokens):
        before = F.pad(tokens, (1, 0))[:, :-1]
        x, q, k, v, z = self.split(tokens, before)
        o = LinearAttention.apply(q, k, v, self.log_decay())
        flat = (-1, 1, self.heads * self.dv)
        return self.logits(x, o.reshape(flat), z.reshape(flat)).reshape(*tokens.shape, -1)

    @torch.no_grad()
    def prompt(self, tokens):
        """Logits of the last token, and the state that single tokens continue from."""
        before = F.pad(tokens, (1, 0))[:, :-1]
        x, q, k, v, z = self.split(tokens, before)
        o, state = ssm.linattn_fwd(q, k, v, self.log_decay())
        return self.serve(x[:, -1], o[:, -1], z[:, -1]), state

    @torch.no_grad()
    def step(self, tokens, before, state):
        x, q, k, v, z = self.split(tokens, before)
        o = ssm.linattn_step(state, q, k, v, self.log_decay())
        return self.serve(x, o, z)

    def serve(self, x, o, z):
        rows = (x.shape[0], 1, self.heads * self.dv)
        y = ssm.group_norm_fwd(o.reshape(rows).contiguous(), self.heads, weight=self.norm.detach(),
                               z=z.reshape(rows).contiguous(), return_stats=False)[0]
        return self.logits(x, None, None, normed=y)


def batch(generator, size, length, vocab, device):
    patterns = torch.randint(0, vocab, (8, 16), generator=torch.Generator().manual_seed(3)).to(device)
    which = torch.randint(0, 8, (size, 1), generator=generator, device=device)
    start = torch.randint(0, 16, (size, 1), generator=generator, device=device)
    return patterns[which, (start + torch.arange(length, device=device)) % 16]


def train(steps=60, io=torch.bfloat16, device="cuda:0", seed=0):
    """Trains and returns (model, losses, gradient norms)."""
    torch.manual_seed(seed)
    generator = torch.Generator(device=device)
    generator.manual_seed(seed)
    model = Model(io=io).to(device)
    params = list(model.parameters())
    opt = torch.optim.Adam(params, lr=5e-3)
    losses, norms = [], []
    for _ in range(steps):
        tokens = batch(generator, 16, 129, 32, device)
        logits = model(tokens[:, :-1])
        loss = F.cross_entropy(logits[:, 16:].reshape(-1, 32), tokens[:, 17:].reshape(-1))
        opt.zero_grad()
        loss.backward()
        norms.append(ssm.clip_grad_norm([p.grad for p in params], 1.0))
        opt.step()
        losses.append(loss.detach())
    return model, [float(x) for x in losses], [float(x) for x in norms]


@torch.no_grad()
def generate(model, prompt, count):
    """Greedy continuation: (tokens, the logits each was chosen from)."""
    logits, state = model.prompt(prompt)
    before, tokens, seen = prompt[:, -1], [], []
    for _ in range(count):
        seen.append(logits)
        token = logits.argmax(-1)
        tokens.append(token)
        logits = model.step(token, before, state)
        before = token
    return torch.stack(tokens, 1), torch.stack(seen, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--io", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args()
    io = torch.bfloat16 if a.io == "bf16" else torch.float32
    model, losses, norms = train(a.steps, io)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}, last gradient norm {norms[-1]:.3f}")
    generator = torch.Generator(device="cuda:0")
    generator.manual_seed(1)
    text = batch(generator, 4, 96, 32, "cuda:0")
    prompt, want = text[:, :64], text[:, 64:]
    tokens, _ = generate(model, prompt, 32)
    print(f"continued {tokens.shape[1]} tokens, {float((tokens == want).float().mean()):.2f} of them the pattern's")


if __name__ == "__main__":
    main()
