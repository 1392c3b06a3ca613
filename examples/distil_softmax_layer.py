"""A softmax layer trained against a teacher, then served, with reduced formats throughout.

The teacher is a layer that is only read: its weight is packed to 4 bits once
(s2_pack4), and per step its logits of the workers' words come from a 4-bit
product (s2_matmul4); the largest of each token are what the student learns from.
The student is the 8-bit layer of softmax_layer_8bit.py. Per step and worker
s2_distill gives its loss against the teacher's top logits and the words that
followed, and the gradient of its logits in bfloat16, which goes the layer's
way: weight gradient into the worker's row of grad[W][n] (s2_wgrad8), compressed
exchange, update. Tokens of padding have row weight 0.
The trained layer is then packed to 4 bits and serves: one product and one
s2_sample call draw the next words of several requests, each with its own
temperature, top-k, top-p and min-p.

    python examples/distil_softmax_layer.py [--vocab V] [--hidden H] [--tokens T] [--workers W] [--steps N]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import sketch_compressed_sparse_gb300 as s2
from examples.softmax_layer_8bit import SoftmaxLayer


class ReadLayer:
    """A V x H layer in 4 bits, for up to T tokens at a time."""

    def __init__(self, weight, tokens):
        self.V, self.H = weight.shape
        self.w, self.ws = s2.alloc_pack4(self.V, self.H, weight.device)
        self.x, self.xs = s2.alloc_pack4(tokens, self.H, weight.device)
        self.logits = torch.empty((tokens, self.V), device=weight.device)
        s2.s2_pack4(weight, self.w, self.ws)

    def forward(self, hidden):
        """Logits [T, V] of hidden states [T, H] (as many as the layer was made for)."""
        s2.s2_pack4(hidden, self.x, self.xs)
        s2.s2_matmul4(self.x, self.xs, self.w, self.ws, self.logits)
        return self.logits


class DistilledLayer(SoftmaxLayer):
    """The 8-bit layer with a teacher's top logits and the words that followed as its targets."""

    def __init__(self, vocab, hidden, tokens, workers, temperature=2.0, hard=0.25, **kw):
        super().__init__(vocab, hidden, tokens, workers, **kw)
        dev = self.logits.device
        self.temperature, self.hard = temperature, hard
        self.loss = torch.empty((workers, tokens), device=dev)
        self.dlogits = torch.empty((tokens, vocab), dtype=torch.bfloat16, device=dev)

    def distil(self, k, hidden, idx, top, targets, weight):
        """Worker k's losses [T] and the gradient of their mean over all workers' tokens by its logits."""
        s2.s2_distill(self.forward(k, hidden), idx, top, self.loss[k], self.dlogits, targets=targets, row_weight=weight,
                      temperature=self.temperature, soft=self.temperature ** 2, hard=self.hard, scale=1 / (self.T * self.W))
        return self.dlogits

    def distil_step(self, hidden, tops, targets, weight, dhidden, lr):
        """One training step on hidden [W, T, H] and the workers' (indices, logits); returns the mean loss (a tensor)."""
        for k in range(self.W):
            idx, top = tops[k]
            self.backward(k, self.distil(k, hidden[k], idx, top, targets[k], weight[k]), dhidden[k])
        self.weight -= lr * self.exchange()
        self.pack_weight()
        return self.loss.mean()


def batches(teacher, workers, tokens, entries, steps, seed=1):
    """Hidden states around the teacher's words, its top logits there, the words, and weights with some padding."""
    dev = teacher.w.device
    g = torch.Generator(device=dev).manual_seed(seed)
    words = torch.empty((teacher.V, teacher.H), device=dev)
    s2.s2_unpack4(teacher.w, teacher.ws, words)
    for _ in range(steps):
        t = torch.randint(teacher.V, (workers, tokens), generator=g, device=dev)
        h = (words[t] + 0.3 * torch.randn((workers, tokens, teacher.H), generator=g, device=dev)).to(torch.bfloat16)
        tops = []
        for k in range(workers):
            top, idx = torch.topk(teacher.forward(h[k]), entries, dim=1)
            tops.append((idx.to(torch.int32), top))
        weight = (torch.rand((workers, tokens), generator=g, device=dev) > 0.1).float()
        yield h, tops, t.to(torch.int32), weight


def serve(layer, hidden, seed=2):
    """The next words of hidden [B, H], every request with its own settings."""
    B, dev = hidden.shape[0], hidden.device
    g = torch.Generator(device=dev).manual_seed(seed)
    head = ReadLayer(layer.weight, B)
    tokens = torch.empty(B, dtype=torch.int32, device=dev)
    of = lambda *v: torch.tensor(v, device=dev).repeat(-(-B // len(v)))[:B].contiguous()  # noqa: E731
    s2.s2_sample(head.forward(hidden), torch.rand(B, generator=g, device=dev), tokens, temperature=of(0.0, 0.7, 1.0, 1.3),
                 top_k=of(0, 50, 0).to(torch.int32), top_p=of(1.0, 0.9, 0.95, 1.0, 0.8), min_p=of(0.0, 0.0, 0.02))
    return tokens


def train(vocab=1003, hidden=256, tokens=512, workers=4, steps=20, lr=20.0, entries=32, requests=24):
    """Losses of the steps, and words served afterwards."""
    g = torch.Generator(device="cuda").manual_seed(0)
    teacher = ReadLayer(torch.randn((vocab, hidden), generator=g, device="cuda"), tokens)
    layer = DistilledLayer(vocab, hidden, tokens, workers)
    dhidden = torch.empty((workers, tokens, hidden), device="cuda")
    before = s2.s2_wait_faults()
    losses, last = [], None
    for h, tops, t, weight in batches(teacher, workers, tokens, entries, steps):
        losses.append(layer.distil_step(h, tops, t, weight, dhidden, lr))
        last = h
    served = serve(layer, last[0][:requests]) if steps else None
    losses = [float(v) for v in losses]
    if s2.s2_wait_faults() != before:  # a kernel gave up a wait: what it wrote is not valid
        raise RuntimeError("a wait in the layer's kernels ran out")
    return losses, served


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--vocab", type=int, default=1003)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--workers", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=20.0)
    a = ap.parse_args()
    losses, served = train(a.vocab, a.hidden, a.tokens, a.workers, a.steps, a.lr)
    for i, v in enumerate(losses):
        print(f"step {i}: loss {v:.4f}")
    print("served:", served.tolist())
