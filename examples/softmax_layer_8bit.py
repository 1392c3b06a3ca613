"""Data-parallel training of a softmax layer with 8-bit activations and weights.

W workers (all on this GPU) share one layer of V outputs and H features. Per
step each worker packs its hidden states to 8 bits (s2_pack8), multiplies them
with the packed weight (s2_matmul8), and from the gradient of its logits takes
  - the weight gradient, from the 8-bit hidden states, straight into its row
    of grad[W][n] (s2_wgrad8, n = V * H),
  - the gradient of its hidden states, from the packed transposed weight
    (s2_matmul8), which a model would pass on to the layers below.
The workers' gradients are then exchanged in compressed form: block Top-K with
error feedback (s2_block_topk), bitmap and count-sketch (s2_encode_batched),
their sum (s2_reduce) and its median decode (s2_decode_dense_ws). The update is
applied to the float32 weight, which is packed again, in both orders.

    python examples/softmax_layer_8bit.py [--vocab V] [--hidden H] [--tokens T] [--workers W] [--steps N]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import sketch_compressed_sparse_gb300 as s2


class SoftmaxLayer:
    """A V x H layer: float32 weight, its 8-bit copies, and the buffers of W workers' steps of T tokens."""

    def __init__(self, vocab, hidden, tokens, workers, device="cuda", seed=0, block=256, keep=0.25, rows=5):
        g = torch.Generator(device=device).manual_seed(seed)
        self.V, self.H, self.T, self.W = vocab, hidden, tokens, workers
        n = vocab * hidden
        self.n, self.block, self.K = n, block, max(1, int(keep * -(-n // block)))
        self.d, self.w, self.seed = rows, max(1024, n // 2), 1234
        self.weight = torch.randn((vocab, hidden), generator=g, device=device) * hidden ** -0.5
        self.codes, self.scales = s2.alloc_pack8(vocab, hidden, "tiles", device)
        self.codes_t, self.scales_t = s2.alloc_pack8(hidden, vocab, "tiles", device)
        self.x, self.xs = zip(*[s2.alloc_pack8(tokens, hidden, "rows", device) for _ in range(workers)])
        self.dy8, self.dys = s2.alloc_pack8(tokens, vocab, "rows", device)
        self.logits = torch.empty((tokens, vocab), device=device)
        self.grad = torch.empty((workers, n), device=device)
        self.residual = torch.zeros((workers, n), device=device)
        self.sparse = torch.empty((workers, n), device=device)
        self.bitmaps, self.sketches = s2.alloc_encode_outputs(workers, n, self.d, self.w, device)
        self.bitmap = torch.empty(s2.nwords(n), dtype=torch.int32, device=device)
        self.sketch = torch.empty((self.d, self.w), device=device)
        self.update = torch.empty(n, device=device)
        self.topk_ws = torch.empty(s2.s2_block_topk_workspace_size(workers, n, block), dtype=torch.uint8, device=device)
        self.decode_ws = torch.empty(s2.s2_decode_dense_workspace_size(n, self.d, self.w), dtype=torch.uint8, device=device)
        self.pack_weight()

    def pack_weight(self):
        s2.s2_pack8(self.weight, self.codes, self.scales, "tiles", self.codes_t, self.scales_t)

    def forward(self, k, hidden):
        """Worker k's logits; its hidden states [T, H] are kept in 8 bits."""
        s2.s2_pack8(hidden, self.x[k], self.xs[k])
        s2.s2_matmul8(self.x[k], self.xs[k], self.codes, self.scales, self.logits)
        return self.logits

    def backward(self, k, dlogits, dhidden):
        """Worker k's weight gradient into grad[k]; the gradient of its hidden states into dhidden [T, H]."""
        s2.s2_wgrad8(dlogits, self.x[k], self.xs[k], self.grad[k].view(self.V, self.H))
        s2.s2_pack8(dlogits, self.dy8, self.dys)
        s2.s2_matmul8(self.dy8, self.dys, self.codes_t, self.scales_t, dhidden)

    def exchange(self):
        """The decoded sum of the workers' kept gradients, [V, H]."""
        s2.s2_block_topk(self.grad, self.residual, self.block, self.K, self.sparse, self.topk_ws)
        s2.s2_encode_batched(self.sparse, self.d, self.w, self.seed, self.bitmaps, self.sketches)
        s2.s2_reduce(self.bitmaps, self.sketches, self.n, self.d, self.w, self.bitmap, self.sketch)
        s2.s2_decode_dense_ws(self.bitmap, self.sketch, self.n, self.d, self.w, self.seed, self.update, self.decode_ws)
        return self.update.view(self.V, self.H)

    def step(self, hidden, targets, dhidden, lr):
        """One training step on hidden [W, T, H] (bfloat16) and targets [W, T]; returns the mean loss (a tensor)."""
        loss = 0.0
        at = torch.arange(self.T, device=targets.device)
        for k in range(self.W):
            logp = torch.log_softmax(self.forward(k, hidden[k]), dim=1)
            loss = loss - logp[at, targets[k]].mean() / self.W
            d = logp.exp()
            d[at, targets[k]] -= 1
            self.backward(k, (d / (self.T * self.W)).to(torch.bfloat16), dhidden[k])
        self.weight -= lr * self.exchange()
        self.pack_weight()
        return loss


def batches(vocab, hidden, tokens, workers, steps, device="cuda", seed=1):
    """Hidden states around one direction per target word."""
    g = torch.Generator(device=device).manual_seed(seed)
    words = torch.randn((vocab, hidden), generator=g, device=device)
    for _ in range(steps):
        t = torch.randint(vocab, (workers, tokens), generator=g, device=device)
        noise = torch.randn((workers, tokens, hidden), generator=g, device=device)
        yield (words[t] + 0.5 * noise).to(torch.bfloat16), t


def train(vocab=1003, hidden=256, tokens=512, workers=4, steps=20, lr=20.0):
    layer = SoftmaxLayer(vocab, hidden, tokens, workers)
    dhidden = torch.empty((workers, tokens, hidden), device="cuda")
    before = s2.s2_wait_faults()
    losses = [layer.step(h, t, dhidden, lr) for h, t in batches(vocab, hidden, tokens, workers, steps)]
    losses = [float(v) for v in losses]
    if s2.s2_wait_faults() != before:  # a kernel gave up a wait: what it wrote is not valid
        raise RuntimeError("a wait in the layer's kernels ran out")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--vocab", type=int, default=1003)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--workers", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=20.0)
    a = ap.parse_args()
    for i, v in enumerate(train(a.vocab, a.hidden, a.tokens, a.workers, a.steps, a.lr)):
        print(f"step {i}: loss {v:.4f}")
