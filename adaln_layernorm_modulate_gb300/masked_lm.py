"""A small masked-token model on packed sequences, from the packed AdaLN node to the vocabulary
loss: the operators of this package together, as a training step uses them.

    python -m adaln_layernorm_modulate_gb300.masked_lm [--steps N] [--heads H]

Every sequence draws a noise level t in (0.1, 1] and hides each of its tokens with probability t.
The model sees the rest; its rows pass one AdaLN-modulated block (a sequence's shift and scale
come from its t) with a mixing step along the packed rows (each with the row before and the one
after it, which at a sequence's ends are its neighbours' in the pack), a final affine layer norm and the
vocabulary head, whose loss counts the hidden tokens only, weighted by 1 / t. With ``heads`` the block
also has self-attention within each sequence: queries and keys normed a head and rotated by their places. Tokens follow a
fixed successor table, so a hidden token can be told from its neighbours and the loss falls.
"""
from __future__ import annotations

import argparse

import torch

from .autograd import LayerNorm, QKNormRope, adaln_modulate, attention, linear_cross_entropy

IGNORE = -100


class MaskedLM(torch.nn.Module):
    def __init__(self, vocab: int, dim: int, device="cuda", heads: int = 0):
        super().__init__()
        if heads and (dim % heads or dim // heads % 8 or dim // heads > 128):
            raise ValueError("heads of a multiple of 8 elements, at most 128: dim %d, heads %d" % (dim, heads))
        kw = dict(device=device, dtype=torch.bfloat16)
        self.embed = torch.nn.Embedding(vocab + 1, dim, **kw)  # the last word hides a token
        self.modulation = torch.nn.Linear(2, 2 * dim, **kw)
        self.up = torch.nn.Linear(3 * dim, 2 * dim, **kw)
        self.down = torch.nn.Linear(2 * dim, dim, **kw)
        self.norm = LayerNorm(dim, device=device, dtype=torch.bfloat16)
        self.head = torch.nn.Parameter(torch.randn(vocab, dim, **kw) / dim ** 0.5)
        self.heads = heads
        if heads:
            self.qkv = torch.nn.Linear(dim, 3 * dim, **kw)
            self.rope = QKNormRope(dim // heads, (dim // heads,), **kw)
            self.out = torch.nn.Linear(dim, dim, **kw)

    def forward(self, tokens, t, cu_seqlens, mod_idx):
        h = self.embed(tokens)
        cond = torch.stack([t, t * t], 1).to(h.dtype)
        shift, scale = self.modulation(cond).chunk(2, dim=1)
        y = adaln_modulate(h, shift.contiguous(), scale.contiguous(), cu_seqlens, mod_idx)
        if self.heads:
            places = torch.arange(len(y), device=y.device, dtype=torch.int32)
            starts = torch.repeat_interleave(cu_seqlens[:-1], cu_seqlens[1:] - cu_seqlens[:-1], output_size=len(y))
            q, k, v = (x.unflatten(1, (self.heads, -1)) for x in self.qkv(y).chunk(3, dim=1))
            q, k = self.rope(q, k, (places - starts)[:, None])
            h = h + self.out(attention(q, k, v, cu_seqlens).flatten(1))
        near = torch.cat([y, torch.roll(y, 1, 0), torch.roll(y, -1, 0)], dim=1)
        return self.norm(h + self.down(torch.nn.functional.silu(self.up(near))))


def batch(gen, lengths, vocab, device="cuda"):
    """Packed tokens, what the model sees, targets (IGNORE where a token is seen), the noise
    level of every sequence and the segment tables."""
    tokens, seen, targets = [], [], []
    t = 0.1 + 0.9 * torch.rand(len(lengths), generator=gen)
    for i, n in enumerate(lengths):
        first = int(torch.randint(vocab, (1,), generator=gen))
        seq = (first * 3 + 7 * torch.arange(n)) % vocab
        hide = torch.rand(n, generator=gen) < t[i]
        tokens.append(seq)
        seen.append(torch.where(hide, torch.full_like(seq, vocab), seq))
        targets.append(torch.where(hide, seq, torch.full_like(seq, IGNORE)))
    cu = torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32)
    mod = torch.arange(len(lengths), dtype=torch.int32)
    return tuple(v.to(device) for v in (torch.cat(seen), torch.cat(targets), t, cu, mod))


def train(steps: int = 60, vocab: int = 997, dim: int = 256, seed: int = 0, lr: float = 3e-3, heads: int = 0):
    """Runs `steps` steps; returns the losses (weighted, a hidden token)."""
    torch.manual_seed(seed)
    gen = torch.Generator().manual_seed(seed)
    model = MaskedLM(vocab, dim, heads=heads)
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0)
    losses = []
    for _ in range(steps):
        lengths = [int(v) for v in torch.randint(16, 400, (8,), generator=gen)]
        seen, target, t, cu, mod = batch(gen, lengths, vocab)
        h = model(seen, t, cu, mod)
        rows = linear_cross_entropy(h, model.head, target, IGNORE, reduction="none")
        weight = torch.repeat_interleave(1 / t, (cu[1:] - cu[:-1]).long())
        hidden = (target != IGNORE).sum().clamp(min=1)
        loss = (rows * weight).sum() / hidden
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in torch.stack(losses)]


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--heads", type=int, default=0, help="heads of self-attention (0: none)")
    args = p.parse_args()
    losses = train(args.steps, heads=args.heads)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print("step %4d  loss %.4f" % (i, losses[i]))
    print("step %4d  loss %.4f" % (len(losses) - 1, losses[-1]))


if __name__ == "__main__":
    main()
