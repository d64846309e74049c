"""Training steps of a small language model whose mixer is KDA, on synthetic tokens.

    python examples/train_lm.py [--steps 40]

Token embedding -> per layer: residual norm, projections, gates, KDA prefill, gated
norm, output projection -> residual norm -> cross entropy over the vocabulary.  The
embedding, the norms, the mixer and the loss, forward and backward, are libkda
kernels; the projections are plain matrix products.  The sequence to learn: every
token follows from the one before it by a fixed random permutation, in packed
sequences of unequal length.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from kimi_delta_attention_18_gb300.autograd import (kda_embedding, kda_gated_norm,  # noqa: E402
                                                    kda_linear_cross_entropy, kda_prefill,
                                                    kda_residual_norm)

HEAD = 128  # d_k = d_v


class Layer(torch.nn.Module):
    def __init__(self, width, heads):
        super().__init__()
        self.heads = heads
        inner = heads * HEAD
        bf16 = dict(device="cuda", dtype=torch.bfloat16)

        def weight(rows, cols):
            return torch.nn.Parameter(torch.randn(rows, cols, **bf16) / cols ** 0.5)

        self.qkvz = weight(4 * inner, width)  # queries, keys, values, output gate
        self.decay = weight(inner, width)
        self.beta = weight(heads, width)
        self.out = weight(width, inner)
        self.norm = torch.nn.Parameter(torch.ones(width, device="cuda"))
        self.out_norm = torch.nn.Parameter(torch.ones(HEAD, device="cuda"))

    def forward(self, x, cu_seqlens, status):
        T, H = x.shape[0], self.heads
        p = (x @ self.qkvz.T).view(T, 4, H, HEAD)
        q, k = (torch.nn.functional.normalize(p[:, i].float(), dim=-1).to(x.dtype) for i in (0, 1))
        g = -5.0 * torch.sigmoid((x @ self.decay.T).float() - 4.0).view(T, H, HEAD)
        beta = torch.sigmoid((x @ self.beta.T).float())
        o, _ = kda_prefill(q.contiguous(), k.contiguous(), p[:, 2].contiguous(), g, beta, None,
                           cu_seqlens, dev_status=status)
        u = kda_gated_norm(o, p[:, 3], self.out_norm, dev_status=status)  # the gate: a slice of the projection
        return u.view(T, H * HEAD) @ self.out.T


class Model(torch.nn.Module):
    def __init__(self, vocab, width, heads, layers):
        super().__init__()
        bf16 = dict(device="cuda", dtype=torch.bfloat16)
        self.table = torch.nn.Parameter(torch.randn(vocab, width, **bf16) * 0.02)
        self.layers = torch.nn.ModuleList(Layer(width, heads) for _ in range(layers))
        self.norm = torch.nn.Parameter(torch.ones(width, device="cuda"))
        self.head = torch.nn.Parameter(torch.randn(vocab, width, **bf16) / width ** 0.5)
        self.embed_scale = width ** 0.5
        self.residual_scale = layers ** -0.5

    def forward(self, ids, targets, cu_seqlens, status):
        """``status`` gets the first error of any kernel of the step (see train)."""
        h = kda_embedding(self.table, ids, scale=self.embed_scale, dev_status=status)
        y, norm = None, dict(scale=self.residual_scale, dev_status=status)
        for layer in self.layers:
            h, x = kda_residual_norm(h, y, layer.norm, **norm)
            y = layer(x, cu_seqlens, status)
        _, x = kda_residual_norm(h, y, self.norm, **norm)
        return kda_linear_cross_entropy(x, self.head, targets, dev_status=status)


def batch(vocab, lengths, gen):
    """Packed sequences, the last position of each without a target."""
    step = torch.randperm(vocab, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    ids, targets = [], []
    for n in lengths:
        t = [torch.randint(0, vocab, (1,), generator=gen, device="cuda")]
        for _ in range(n - 1):
            t.append(step[t[-1]])
        t = torch.cat(t)
        ids.append(t)
        targets.append(torch.cat([t[1:], torch.full((1,), -100, device="cuda")]))
    cu = torch.tensor([0] + list(lengths), device="cuda").cumsum(0).to(torch.int32)
    return torch.cat(ids), torch.cat(targets), cu


def train(steps=40, vocab=199, width=256, heads=2, layers=2, lengths=(96, 64, 31), seed=0, log=print):
    """Runs ``steps`` steps; returns their losses."""
    torch.manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = Model(vocab, width, heads, layers)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    losses = []
    for i in range(steps):
        loss = model(*batch(vocab, lengths, gen), status)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if int(status):  # the host waits for the loss anyway
            raise RuntimeError("step %d: a kernel reported status %d" % (i, int(status)))
        if i % 10 == 0 or i == steps - 1:
            log("step %d: loss %.3f" % (i, losses[-1]))
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=40)
    train(ap.parse_args().steps)
