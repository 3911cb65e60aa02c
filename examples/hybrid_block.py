"""A small hybrid language model over the framework's operators, trained and then served.

Every layer is  stream -> norm -> mixer -> residual scale -> stream; mixers alternate between the
gated delta rule and the selective scan.  A mixer passes its inputs through the short causal
convolution and its output through a gated norm.  The residual add of a layer and the norm in front
of the next one are one call (block_norm), on an fp32 stream.

    python examples/hybrid_block.py [--steps 100] [--dtype bfloat16]

trains on a synthetic task (every token's successor under a fixed permutation), then answers prompts token by
token from the states that the prompt left in the pools, and compares the logits with those of the
whole sequence run at once.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_04_gb300 as gdr  # noqa: E402


def param(*shape, std=None, value=None):
    t = torch.empty(*shape)
    return nn.Parameter(t.fill_(value) if value is not None else t.normal_(0, std))


class DeltaMixer(nn.Module):
    """q, k, v through the convolution, the gated delta rule with its input prologue, a norm per head
    gated by z."""

    def __init__(self, dim, heads, width, taps=4):
        super().__init__()
        self.H, self.D, self.taps = heads, width, taps
        inner = heads * width
        self.sizes = [3 * inner, inner, heads, heads]  # q k v, z, decay logit, beta logit
        self.proj = nn.Linear(dim, sum(self.sizes), bias=False)
        self.out = nn.Linear(inner, dim, bias=False)
        self.conv = param(3 * inner, taps, std=1 / math.sqrt(taps))
        self.norm = param(width, value=1.0)
        self.decay = param(heads, value=3.0)

    def state(self, slots, dtype):
        return [torch.zeros(slots, self.taps - 1, 3 * self.H * self.D, device="cuda", dtype=dtype),
                torch.zeros(slots, self.H, self.D, self.D, device="cuda")]

    def split(self, x):
        qkv, z, a, b = self.proj(x).split(self.sizes, -1)
        return qkv, z.unflatten(-1, (self.H, self.D)), a.float() + self.decay, b.contiguous()

    def forward(self, x, pool=None, slots=None):
        B, T = x.shape[:2]
        qkv, z, a, b = self.split(x)
        outs, lasts = [], []
        for i in range(3):  # slices of the projection, used where they lie; what comes out is contiguous
            c = slice(i * self.H * self.D, (i + 1) * self.H * self.D)
            y, last = gdr.causal_conv(qkv[..., c], self.conv[c])
            outs.append(y.view(B, T, self.H, self.D))
            lasts.append(last)
        o, S = gdr.chunk_gated_delta_rule(*outs, a, b, prologue=gdr.GDR_PROLOGUE_ALL)
        if pool is not None:
            pool[0][slots.long()] = torch.cat(lasts, -1)
            pool[1][slots.long()] = S
        y, _ = gdr.block_norm(o, self.norm, z)
        return self.out(y.flatten(-2))

    def step(self, x, pool, slots):
        qkv, z, a, b = self.split(x)
        y = gdr.conv_step(qkv, pool[0], self.conv, slots=slots)
        q, k, v = (t.unflatten(-1, (self.H, self.D)).contiguous() for t in y.chunk(3, -1))
        o = gdr.step(q, k, v, a, b, pool[1], slots=slots, prologue=gdr.GDR_PROLOGUE_ALL)
        y, _ = gdr.norm_forward(o, self.norm, z.contiguous())
        return self.out(y.flatten(-2))


class ScanMixer(nn.Module):
    """x through the convolution, the selective scan, a norm over all channels gated by z."""

    def __init__(self, dim, inner, states=16, taps=4):
        super().__init__()
        self.inner, self.N, self.taps = inner, states, taps
        self.sizes = [inner, inner, inner, states, states]  # x, z, dt, B, C
        self.proj = nn.Linear(dim, sum(self.sizes), bias=False)
        self.out = nn.Linear(inner, dim, bias=False)
        self.conv, self.conv_bias = param(inner, taps, std=1 / math.sqrt(taps)), param(inner, value=0.0)
        self.norm, self.skip = param(inner, value=1.0), param(inner, value=1.0)
        self.A_log = nn.Parameter(torch.log(torch.arange(1, states + 1).float()).expand(inner, states).clone())
        self.dt_bias = param(inner, value=math.log(math.expm1(0.03)))

    def state(self, slots, dtype):
        return [torch.zeros(slots, self.taps - 1, self.inner, device="cuda", dtype=dtype),
                torch.zeros(slots, self.inner, self.N, device="cuda")]

    def forward(self, x, pool=None, slots=None):
        u, z, dt, Bm, Cm = self.proj(x).split(self.sizes, -1)
        u, last = gdr.causal_conv(u, self.conv, self.conv_bias)
        y, S = gdr.selective_scan(u, dt, -torch.exp(self.A_log), Bm.unsqueeze(2), Cm.unsqueeze(2), self.skip, self.dt_bias)
        if pool is not None:
            pool[0][slots.long()] = last
            pool[1][slots.long()] = S
        y, _ = gdr.block_norm(y, self.norm, z)
        return self.out(y)

    def step(self, x, pool, slots):
        u, z, dt, Bm, Cm = self.proj(x).split(self.sizes, -1)
        u = gdr.conv_step(u, pool[0], self.conv, self.conv_bias, slots)
        y = gdr.ssm_step(u, dt, -torch.exp(self.A_log), Bm.unsqueeze(1), Cm.unsqueeze(1), pool[1], self.skip, self.dt_bias,
                         slots)
        y, _ = gdr.norm_forward(y, self.norm, z.contiguous())
        return self.out(y)


class HybridModel(nn.Module):
    def __init__(self, vocab=64, dim=128, layers=4, heads=2, width=64, dtype=torch.bfloat16):
        super().__init__()
        self.dtype = dtype
        self.embed = nn.Embedding(vocab, dim)
        self.mixers = nn.ModuleList(DeltaMixer(dim, heads, width) if i % 2 == 0 else ScanMixer(dim, heads * width)
                                    for i in range(layers))
        self.norms = nn.ParameterList(param(dim, value=1.0) for _ in range(layers + 1))
        self.scales = nn.ParameterList(param(dim, value=0.5) for _ in range(layers))
        self.head = nn.Linear(dim, vocab, bias=False)
        # matrix products and activations in dtype; convolutions, norms, rates and scales stay in fp32
        for m in self.modules():
            if isinstance(m, (nn.Linear, nn.Embedding)):
                m.to(dtype)

    def state(self, slots):
        return [m.state(slots, self.dtype) for m in self.mixers]

    def run(self, tokens, mix):
        x = self.embed(tokens)
        r = x.float()  # the stream
        _, y = gdr.block_norm(x, pre_weight=self.norms[0])
        for m, scale, norm in zip(self.mixers, self.scales, self.norms[1:]):
            # residual scale, residual add and the next layer's norm in one pass
            r, y = gdr.block_norm(mix(m, y), scale=scale, residual=r, pre_weight=norm)
        return self.head(y).float()

    def forward(self, tokens, pools=None, slots=None):
        """Logits of whole sequences; with pools their states go to the given slots."""
        pools = dict(zip(self.mixers, pools)) if pools is not None else {}
        return self.run(tokens, lambda m, y: m(y, pools.get(m), slots))

    @torch.no_grad()
    def step(self, tokens, pools, slots):
        """Logits of one token per row, states updated in their slots."""
        pools = dict(zip(self.mixers, pools))
        return self.run(tokens, lambda m, y: m.step(y, pools[m], slots))


def permutation(vocab):
    return torch.randperm(vocab, generator=torch.Generator().manual_seed(7))


def walks(n, length, vocab, gen):
    """Sequences that follow a fixed permutation of the tokens from a random start."""
    successor = permutation(vocab)
    seq = [torch.randint(0, vocab, (n,), generator=gen)]
    while len(seq) < length:
        seq.append(successor[seq[-1]])
    return torch.stack(seq, 1).cuda()


def train(model, steps, vocab, batch=16, length=96, lr=3e-3, seed=0):
    gen = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        seq = walks(batch, length + 1, vocab, gen)
        logits = model(seq[:, :-1])
        loss = nn.functional.cross_entropy(logits.flatten(0, 1), seq[:, 1:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


@torch.no_grad()
def serve(model, vocab, batch=5, prompt=41, new=20, seed=1):
    """Answers prompts token by token; returns the tokens and the largest difference of the step logits
    from those of the whole sequences, relative to the largest logit."""
    gen = torch.Generator().manual_seed(seed)
    seq = walks(batch, prompt, vocab, gen)
    pools = model.state(slots=batch + 3)
    slots = torch.randperm(batch + 3, generator=gen)[:batch].to(torch.int32).cuda()
    logits = model(seq, pools, slots)[:, -1]
    steps = []
    for _ in range(new):
        seq = torch.cat([seq, logits.argmax(-1, keepdim=True)], 1)
        logits = model.step(seq[:, -1], pools, slots)
        steps.append(logits)
    whole = model(seq)[:, prompt:]
    diff = (torch.stack(steps, 1) - whole).abs().max() / whole.abs().max()
    return seq, diff.item()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--dtype", choices=["bfloat16", "float32"], default="bfloat16")
    a = ap.parse_args()
    torch.manual_seed(0)
    vocab = 64
    model = HybridModel(vocab, dtype=getattr(torch, a.dtype)).cuda()
    losses = train(model, a.steps, vocab)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
    seq, diff = serve(model, vocab)
    successor = permutation(vocab).cuda()
    right = (seq[:, 41:] == successor[seq[:, 40:-1]]).float().mean().item()
    print(f"step logits within {diff:.2e} of the whole sequences'; {100 * right:.0f}% of the answered tokens are right")


if __name__ == "__main__":
    main()
