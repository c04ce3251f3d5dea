"""Trains a feed-forward block between two layer norms, with dropout, and serves it in 8
bits: every norm, mask, product, activation and gradient is a call of the library.

    python3 examples/train_block.py [--steps 40] [--dtype bf16]

    n = norm(x),  h = drop(silu(n wg^T) * (n wu^T)),  s = x + drop(h wd^T),
    logits = norm(s) wc^T + bc

The masks come from a step number on the device, so the same program can be captured
into a graph: every replay draws new ones, and the backward pass draws them again.  After
training the projection and the classifier run on 8-bit weights, with their inputs
quantized row by row.  The data are synthetic: features of a random linear teacher.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import convolution_forward_amd as cf  # noqa: E402

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def stream():
    return torch.cuda.current_stream().cuda_stream


class Block:
    def __init__(self, rows, width, hidden, classes, dtype, drop=0.1, seed=0, max_norm=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        t = TYPES[dtype]

        def normal(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") * shape[-1] ** -0.5).to(t)

        def empty(*shape, t=t):
            return torch.empty(shape, dtype=t, device="cuda")

        self.dtype, self.rows = dtype, rows
        self.w1, self.w2 = (torch.ones(width, dtype=t, device="cuda") for _ in range(2))
        self.b1, self.b2 = (torch.zeros(width, dtype=t, device="cuda") for _ in range(2))
        self.wg, self.wu = normal(hidden, width), normal(hidden, width)
        self.wd, self.wc = normal(width, hidden), normal(classes, width)
        self.bc = torch.zeros(classes, dtype=t, device="cuda")
        self.weights = [self.w1, self.b1, self.wg, self.wu, self.wd, self.w2, self.b2, self.wc, self.bc]
        self.grads = [torch.empty_like(w) for w in self.weights]
        self.n1, self.s, self.n2 = (empty(rows, width) for _ in range(3))
        self.o, self.do, self.dn, self.ds, self.dx = (empty(rows, width) for _ in range(5))
        self.pg, self.pu, self.h, self.dh = (empty(rows, hidden) for _ in range(4))
        self.logits = empty(rows, classes)
        self.stats = [empty(rows, t=torch.float32) for _ in range(4)]
        # the number of the step: a mask's offset, moved on by every step
        self.step_number = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.norm1 = cf.make_layer_norm_problem(rows, width)
        self.up = cf.make_gated_problem(rows, hidden, width, act="silu", save=True)
        # masks of one step differ by their seeds
        self.mask = cf.make_dropout_problem(rows, hidden, drop, seed=2 * seed)
        self.down = cf.make_linear_problem(rows, width, hidden)
        self.norm2 = cf.make_layer_norm_problem(rows, width, residual=True, drop=drop, seed=2 * seed + 1)
        self.classify = cf.make_linear_problem(rows, classes, width, bias=True)
        self.clip = cf.make_grad_clip_problem(self.grads, self.grads, dtype, max_norm=max_norm)
        self.norm = torch.zeros(1, device="cuda")
        # one scratch for all: the calls of a stream use it one after the other
        self.bytes = max(cf.layer_norm_scratch_size(self.norm2, dtype),
                         cf.layer_norm_backward_scratch_size(self.norm2, dtype),
                         cf.gated_scratch_size(self.up, dtype),
                         cf.gated_backward_scratch_size(self.up, dtype),
                         cf.linear_scratch_size(self.down, dtype),
                         cf.linear_backward_scratch_size(self.down, dtype),
                         cf.linear_scratch_size(self.classify, dtype),
                         cf.linear_backward_scratch_size(self.classify, dtype),
                         cf.grad_clip_scratch_size(self.clip))
        self.scratch = torch.empty(self.bytes, dtype=torch.uint8, device="cuda")

    def forward(self, x):
        d, s, n = self.dtype, stream(), self.step_number
        room = (self.scratch, self.bytes, s)
        cf.layer_norm_forward(self.norm1, d, x, None, self.w1, self.b1, self.n1, None,
                              *self.stats[:2], None, *room)
        cf.gated_forward(self.up, d, self.n1, self.wg, self.wu, None, None, self.h, self.pg, self.pu, *room)
        cf.dropout_forward(self.mask, d, self.h, None, self.h, n, s)
        cf.linear_forward(self.down, d, self.h, self.wd, None, None, self.o, None, *room)
        cf.layer_norm_forward(self.norm2, d, self.o, x, self.w2, self.b2, self.n2, self.s,
                              *self.stats[2:], n, *room)
        cf.linear_forward(self.classify, d, self.n2, self.wc, self.bc, None, self.logits, None, *room)
        return self.logits

    def backward(self, x, dlogits):
        """Weight gradients into self.grads, clipped together; x's gradient into self.dx."""
        d, s, n = self.dtype, stream(), self.step_number
        room = (self.scratch, self.bytes, s)
        dw1, db1, dwg, dwu, dwd, dw2, db2, dwc, dbc = self.grads
        cf.linear_backward(self.classify, d, self.n2, self.wc, None, dlogits, self.dn, dwc, dbc, None, *room)
        cf.layer_norm_backward(self.norm2, d, self.s, self.w2, *self.stats[2:], self.dn, None, self.do,
                               self.ds, dw2, db2, n, *room)
        cf.linear_backward(self.down, d, self.h, self.wd, None, self.do, self.dh, dwd, None, None, *room)
        cf.dropout_backward(self.mask, d, self.dh, self.dh, n, s)
        cf.gated_backward(self.up, d, self.n1, self.wg, self.wu, self.pg, self.pu, self.dh, self.dn, dwg,
                          dwu, None, None, *room)
        # the stream's own gradient joins in the first norm's
        cf.layer_norm_backward(self.norm1, d, x, self.w1, *self.stats[:2], self.dn, self.ds, self.dx,
                               None, dw1, db1, None, *room)
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
        self.step_number.add_(1)
        return loss


class Served:
    """The block without dropout, its projection and classifier in 8 bits."""

    def __init__(self, block, rows):
        self.block, self.rows, d = block, rows, block.dtype
        t = TYPES[d]
        (hidden, width), classes = block.wg.shape, block.wc.shape[0]
        self.weights = []  # laid out once
        for w in (block.wd, block.wc):
            q = torch.empty(w.shape, dtype=torch.int8, device="cuda")
            scale = torch.empty(w.shape[0], device="cuda")
            cf.quantize_rows(cf.make_quantize_problem(*w.shape), d, w, q, scale, stream())
            self.weights += [q, scale]
        self.norm = cf.make_layer_norm_problem(rows, width)
        self.up = cf.make_gated_problem(rows, hidden, width, act="silu")
        self.quant_h, self.quant_n = (cf.make_quantize_problem(rows, k) for k in (hidden, width))
        self.down = cf.make_linear_int8_problem(rows, width, hidden, residual="after")
        self.classify = cf.make_linear_int8_problem(rows, classes, width, bias=True)
        self.n, self.s = (torch.empty(rows, width, dtype=t, device="cuda") for _ in range(2))
        self.h = torch.empty(rows, hidden, dtype=t, device="cuda")
        self.q = torch.empty(rows, max(hidden, width), dtype=torch.int8, device="cuda")
        self.scale = torch.empty(rows, device="cuda")
        self.logits = torch.empty(rows, classes, dtype=t, device="cuda")
        self.bytes = max(cf.layer_norm_scratch_size(self.norm, d), cf.gated_scratch_size(self.up, d),
                         cf.linear_int8_scratch_size(self.down, d),
                         cf.linear_int8_scratch_size(self.classify, d))
        self.scratch = torch.empty(self.bytes, dtype=torch.uint8, device="cuda")

    def forward(self, x):
        b, d, s = self.block, self.block.dtype, stream()
        room = (self.scratch, self.bytes, s)
        wd, wd_scale, wc, wc_scale = self.weights
        cf.layer_norm_forward(self.norm, d, x, None, b.w1, b.b1, self.n, None, None, None, None, *room)
        cf.gated_forward(self.up, d, self.n, b.wg, b.wu, None, None, self.h, None, None, *room)
        cf.quantize_rows(self.quant_h, d, self.h, self.q, self.scale, s)
        cf.linear_int8_forward(self.down, d, self.q, self.scale, wd, wd_scale, None, x, self.s, *room)
        cf.layer_norm_forward(self.norm, d, self.s, None, b.w2, b.b2, self.n, None, None, None, None, *room)
        cf.quantize_rows(self.quant_n, d, self.n, self.q, self.scale, s)
        cf.linear_int8_forward(self.classify, d, self.q, self.scale, wc, wc_scale, b.bc, None,
                               self.logits, *room)
        return self.logits


def train(steps=40, dtype="bf16", rows=512, width=256, hidden=688, classes=100, rate=0.5, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    teacher = torch.randn(classes, width, generator=gen, device="cuda")
    block = Block(rows, width, hidden, classes, dtype, seed=seed)
    losses = []
    for i in range(steps):
        x = torch.randn(rows, width, generator=gen, device="cuda")
        labels = (x @ teacher.t()).argmax(1)
        losses.append(block.step(x.to(TYPES[dtype]), labels, rate))
        if i % 10 == 0 or i == steps - 1:
            print(f"step {i}: loss {float(losses[-1]):.3f}, gradient norm {float(block.norm):.3f}",
                  flush=True)
    x = torch.randn(rows, width, generator=gen, device="cuda")
    right = Served(block, rows).forward(x.to(TYPES[dtype])).argmax(1) == (x @ teacher.t()).argmax(1)
    print(f"served in 8 bits: {float(right.float().mean()):.0%} of {rows} right", flush=True)
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--dtype", choices=sorted(TYPES), default="bf16")
    args = ap.parse_args()
    train(args.steps, args.dtype)
