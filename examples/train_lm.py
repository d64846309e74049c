"""Training steps of a small language model whose mixer is KDA, on synthetic tokens.

    python examples/train_lm.py [--steps 40] [--full] [--dropout 0.05]

Token embedding -> per layer: residual norm, projections, gates, KDA prefill, gated
norm, output projection -> residual norm -> cross entropy over the vocabulary.  --full:
every second layer's mixer is a gated linear recurrence instead (projections, recurrence,
gated norm, output projection), and every mixer is followed by a residual norm and a gated
feed-forward block.  --dropout: each block's output is dropped out before it is added to
the residual stream.  The embedding, the norms with their dropout, the mixers, the
feed-forward block and the loss, forward and backward, are libkda kernels; the other
projections are plain matrix products.  The sequence to learn: every
token follows from the one before it by a fixed random permutation, in packed
sequences of unequal length.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from kimi_delta_attention_18_gb300.autograd import (kda_embedding, kda_gated_ffn,  # noqa: E402
                                                    kda_gated_norm, kda_linear_cross_entropy,
                                                    kda_linear_recurrence, kda_prefill,
                                                    kda_residual_norm)

HEAD = 128  # d_k = d_v


def weight(*shape):
    return torch.nn.Parameter(torch.randn(*shape, device="cuda", dtype=torch.bfloat16) / shape[-1] ** 0.5)


class KDAMixer(torch.nn.Module):
    def __init__(self, width, heads):
        super().__init__()
        self.heads = heads
        inner = heads * HEAD
        self.qkvz = weight(4 * inner, width)  # queries, keys, values, output gate
        self.decay = weight(inner, width)
        self.beta = weight(heads, width)
        self.out = weight(width, inner)
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


class RecurrenceMixer(torch.nn.Module):
    """A state per channel: the mean of the past tokens with a learnt decay."""

    def __init__(self, width, heads):
        super().__init__()
        self.heads = heads
        inner = heads * HEAD
        self.xgz = weight(3 * inner, width)  # inputs, decays, output gate
        self.out = weight(width, inner)
        self.out_norm = torch.nn.Parameter(torch.ones(HEAD, device="cuda"))

    def forward(self, x, cu_seqlens, status):
        T, H = x.shape[0], self.heads
        p = (x @ self.xgz.T).view(T, 3, H * HEAD)
        g = -torch.nn.functional.softplus(p[:, 1].float())
        o, _ = kda_linear_recurrence(p[:, 0], g, None, cu_seqlens, write="mix", dev_status=status)
        u = kda_gated_norm(o.view(T, H, HEAD), p[:, 2].view(T, H, HEAD), self.out_norm,
                           act="silu", dev_status=status)
        return u.view(T, H * HEAD) @ self.out.T


class Layer(torch.nn.Module):
    def __init__(self, width, mixer, ffn):
        super().__init__()
        self.mixer = mixer
        self.norm = torch.nn.Parameter(torch.ones(width, device="cuda"))
        self.ffn = ffn
        if ffn:
            self.ffn_norm = torch.nn.Parameter(torch.ones(width, device="cuda"))
            self.gate_up, self.down = weight(2, 2 * width, width), weight(width, 2 * width)

    def forward(self, h, y, cu_seqlens, status, norm):
        """The residual stream h and the output y of the block before; the same after this layer."""
        h, x = norm(h, y, self.norm)
        y = self.mixer(x, cu_seqlens, status)
        if self.ffn:
            h, x = norm(h, y, self.ffn_norm)
            y = kda_gated_ffn(x, self.gate_up, dev_status=status) @ self.down.T
        return h, y


class Model(torch.nn.Module):
    def __init__(self, vocab, width, heads, layers, full=False, dropout=0.0):
        super().__init__()
        bf16 = dict(device="cuda", dtype=torch.bfloat16)
        self.table = torch.nn.Parameter(torch.randn(vocab, width, **bf16) * 0.02)
        self.layers = torch.nn.ModuleList(
            Layer(width, (RecurrenceMixer if full and i % 2 else KDAMixer)(width, heads), full)
            for i in range(layers))
        self.norm = torch.nn.Parameter(torch.ones(width, device="cuda"))
        self.head = torch.nn.Parameter(torch.randn(vocab, width, **bf16) / width ** 0.5)
        self.embed_scale = width ** 0.5
        self.residual_scale = (2 * layers if full else layers) ** -0.5
        self.dropout = dropout

    def forward(self, ids, targets, cu_seqlens, status, rng=None):
        """``status`` gets the first error of any kernel of the step (see train); ``rng`` is the
        step's (seed, offset) for dropout, whose sites are numbered."""
        h = kda_embedding(self.table, ids, scale=self.embed_scale, dev_status=status)
        y, sites = None, iter(range(1 << 16))

        def norm(h, y, w):
            drop = {} if y is None or not self.dropout else dict(dropout=self.dropout, rng=rng,
                                                                 site=next(sites))
            return kda_residual_norm(h, y, w, scale=self.residual_scale, dev_status=status, **drop)

        for layer in self.layers:
            h, y = layer(h, y, cu_seqlens, status, norm)
        _, x = norm(h, y, self.norm)
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


def train(steps=40, vocab=199, width=256, heads=2, layers=2, lengths=(96, 64, 31), seed=0, log=print,
          full=False, dropout=0.0):
    """Runs ``steps`` steps; returns their losses."""
    torch.manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = Model(vocab, width, heads, layers, full, dropout)
    rng = torch.tensor([seed, 0], device="cuda")
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    losses = []
    for i in range(steps):
        loss = model(*batch(vocab, lengths, gen), status, rng)
        rng[1] += 1  # the next step drops other elements
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
    ap.add_argument("--full", action="store_true")
    ap.add_argument("--dropout", type=float, default=0.0)
    args = ap.parse_args()
    train(args.steps, full=args.full, dropout=args.dropout)
