"""Trains a head on pooled features: a gated feed-forward block with a residual, a
classifier, gradient clipping and an SGD step, with the library's calls for every
product, activation and gradient.

    python3 examples/train_head.py [--steps 40] [--dtype bf16]

The data are synthetic: features of a random linear teacher.  Weights, activations
and gradients live in buffers that are allocated once; a step only enqueues work.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import convolution_forward_amd as cf  # noqa: E402

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Head:
    """logits = (x + (silu(x wg^T) * (x wu^T)) wd^T) wc^T + bc, trained by SGD."""

    def __init__(self, rows, width, hidden, classes, dtype, seed=0, max_norm=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        t = TYPES[dtype]

        def normal(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") * shape[-1] ** -0.5).to(t)

        def empty(*shape):
            return torch.empty(shape, dtype=t, device="cuda")

        self.dtype, self.rows, self.classes = dtype, rows, classes
        self.wg, self.wu = normal(hidden, width), normal(hidden, width)
        self.wd, self.wc = normal(width, hidden), normal(classes, width)
        self.bc = torch.zeros(classes, dtype=t, device="cuda")
        self.weights = [self.wg, self.wu, self.wd, self.wc, self.bc]
        self.grads = [torch.empty_like(w) for w in self.weights]
        self.pg, self.pu, self.h = empty(rows, hidden), empty(rows, hidden), empty(rows, hidden)
        self.y, self.logits = empty(rows, width), empty(rows, classes)
        self.dy, self.dh = empty(rows, width), empty(rows, hidden)
        self.up = cf.make_gated_problem(rows, hidden, width, act="silu", save=True)
        self.down = cf.make_linear_problem(rows, width, hidden, residual="after")
        self.classify = cf.make_linear_problem(rows, classes, width, bias=True)
        self.clip = cf.make_grad_clip_problem(self.grads, self.grads, dtype, max_norm=max_norm)
        self.norm = torch.zeros(1, device="cuda")
        # one scratch for all: the calls of a stream use it one after the other
        self.bytes = max(cf.gated_scratch_size(self.up, dtype),
                         cf.gated_backward_scratch_size(self.up, dtype),
                         cf.linear_scratch_size(self.down, dtype),
                         cf.linear_backward_scratch_size(self.down, dtype),
                         cf.linear_scratch_size(self.classify, dtype),
                         cf.linear_backward_scratch_size(self.classify, dtype),
                         cf.grad_clip_scratch_size(self.clip))
        self.scratch = torch.empty(self.bytes, dtype=torch.uint8, device="cuda")

    def forward(self, x):
        d, s = self.dtype, torch.cuda.current_stream().cuda_stream
        room = (self.scratch, self.bytes, s)
        cf.gated_forward(self.up, d, x, self.wg, self.wu, None, None, self.h, self.pg, self.pu, *room)
        cf.linear_forward(self.down, d, self.h, self.wd, None, x, self.y, None, *room)
        cf.linear_forward(self.classify, d, self.y, self.wc, self.bc, None, self.logits, None, *room)
        return self.logits

    def backward(self, x, dlogits):
        """Weight gradients into self.grads, clipped together; their norm into self.norm."""
        d, s = self.dtype, torch.cuda.current_stream().cuda_stream
        room = (self.scratch, self.bytes, s)
        dwg, dwu, dwd, dwc, dbc = self.grads
        cf.linear_backward(self.classify, d, self.y, self.wc, None, dlogits, self.dy, dwc, dbc, None,
                           *room)
        cf.linear_backward(self.down, d, self.h, self.wd, None, self.dy, self.dh, dwd, None, None,
                           *room)
        # x is the first layer's input here: its own gradient is not wanted
        cf.gated_backward(self.up, d, x, self.wg, self.wu, self.pg, self.pu, self.dh, None, dwg, dwu,
                          None, None, *room)
        cf.grad_clip(self.clip, self.norm, *room)

    def step(self, x, labels, rate):
        logits = self.forward(x).float()
        p = torch.softmax(logits, 1)
        at = torch.arange(self.rows, device="cuda")
        loss = -torch.log(p[at, labels]).mean()
        p[at, labels] -= 1.0
        self.backward(x, (p / self.rows).to(TYPES[self.dtype]))
        for w, g in zip(self.weights, self.grads):
            w.add_(g, alpha=-rate)
        return loss


def train(steps=40, dtype="bf16", rows=512, width=256, hidden=688, classes=100, rate=0.5, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    teacher = torch.randn(classes, width, generator=gen, device="cuda")
    head = Head(rows, width, hidden, classes, dtype, seed)
    losses = []
    for i in range(steps):
        x = torch.randn(rows, width, generator=gen, device="cuda")
        labels = (x @ teacher.t()).argmax(1)
        losses.append(head.step(x.to(TYPES[dtype]), labels, rate))
        if i % 10 == 0 or i == steps - 1:
            print(f"step {i}: loss {float(losses[-1]):.3f}, gradient norm {float(head.norm):.3f}",
                  flush=True)
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--dtype", choices=sorted(TYPES), default="bf16")
    args = ap.parse_args()
    train(args.steps, args.dtype)
