"""The block example: a step's outputs and gradients against 64-bit arithmetic with the
same masks, a captured step, and the served block against its 8-bit weights."""
import os
import sys

import pytest

import mask_reference as mask

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def reference(block, x, drop, step):
    """Logits of the block in 64 bits, from weights that take gradients."""
    rows, hidden = block.rows, block.wg.shape[0]
    w1, b1, wg, wu, wd, w2, b2, wc, bc = w = [t.double().requires_grad_(True) for t in block.weights]
    xd = x.double().requires_grad_(True)

    def keep(n, seed):
        k = torch.from_numpy(mask.keeps(rows, n, drop, seed, step)).cuda().double()
        return k * mask.scale(drop)

    def norm(v, w, b):
        d = v - v.mean(1, keepdim=True)
        return d * ((d * d).mean(1, keepdim=True) + 1e-5) ** -0.5 * w + b

    n1 = norm(xd, w1, b1)
    g, u = n1 @ wg.t(), n1 @ wu.t()
    h = g * torch.sigmoid(g) * u * keep(hidden, block.mask.seed)
    s = xd + keep(x.shape[1], block.norm2.seed) * (h @ wd.t())
    return norm(s, w2, b2) @ wc.t() + bc, xd, w


def test_a_step_in_float32():
    """float32: sums of at most 200 terms in each of seven layers, relative to their
    largest values 200 * 2^-24 each, a factor of 10 for the layers' slopes and sizes."""
    import train_block
    rows, width, hidden, classes = 96, 64, 120, 33
    block = train_block.Block(rows, width, hidden, classes, "f32", drop=0.25, seed=3, max_norm=1e9)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for w in (block.w1, block.b1, block.w2, block.b2):
        w.add_(torch.randn(width, generator=gen, device="cuda") * 0.2)
    x = torch.randn(rows, width, generator=gen, device="cuda")
    dlogits = torch.randn(rows, classes, generator=gen, device="cuda") / rows
    block.step_number.fill_(17)
    logits, xd, weights = reference(block, x, 0.25, 17)
    want = torch.autograd.grad(logits, [xd, *weights], dlogits.double())
    tol = 10 * 7 * 200 * 2.0 ** -24
    got = block.forward(x)
    assert float((got.double() - logits.detach()).abs().max()) <= tol * float(logits.detach().abs().max())
    block.backward(x, dlogits)
    for a, b in zip([block.dx, *block.grads], want):
        assert float((a.double() - b).abs().max()) <= tol * float(b.abs().max())
    norm = sum(float((b ** 2).sum()) for b in want[1:]) ** 0.5
    assert abs(float(block.norm) - norm) <= tol * norm


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_captured_steps(dtype):
    """A captured forward and backward, replayed: each draws the masks of its step and
    gives the eager calls' bits."""
    import train_block
    rows, width, hidden, classes = 128, 96, 200, 50
    block = train_block.Block(rows, width, hidden, classes, dtype, drop=0.3, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(2)
    new = lambda n: torch.randn(rows, n, generator=gen, device="cuda").to(train_block.TYPES[dtype])  # noqa: E731
    x, dlogits = new(width), new(classes)

    def call():
        block.forward(x)
        block.backward(x, dlogits)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        block.step_number.add_(1)
    block.step_number.zero_()
    seen = []
    for i in range(4):
        x.copy_(new(width) if i != 2 else x)  # twice the same input: other masks
        call()
        want = [t.clone() for t in (block.logits, block.dx, block.norm, *block.grads)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(block.step_number) == i + 1
        assert all(torch.equal(a, b) for a, b in
                   zip(want, (block.logits, block.dx, block.norm, *block.grads)))
        seen.append(want[0])
    assert not torch.equal(seen[1], seen[2])


@pytest.mark.parametrize("rows", [1, 40])
def test_served(rows):
    """Float32 around the 8-bit products: the reference takes the library's own steps of
    h and n (their borders are another test's), so what is left are float32 sums of at
    most 200 terms in five layers: 10 * 5 * 200 * 2^-24 of the largest value."""
    import train_block
    import convolution_forward_amd as cf
    block = train_block.Block(rows, 64, 120, 33, "f32", seed=7)
    served = train_block.Served(block, rows)
    x = torch.randn(rows, 64, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    got = served.forward(x).double()

    def steps(v, k):
        q = torch.empty(rows, k, dtype=torch.int8, device="cuda")
        scale = torch.empty(rows, device="cuda")
        cf.quantize_rows(cf.make_quantize_problem(rows, k), "f32", v, q, scale, train_block.stream())
        return q.double() * scale.double()[:, None]

    def norm(v, w, b):
        d = v - v.mean(1, keepdim=True)
        return d * ((d * d).mean(1, keepdim=True) + 1e-5) ** -0.5 * w.double() + b.double()

    wd, wd_scale, wc, wc_scale = served.weights
    n1 = norm(x.double(), block.w1, block.b1)
    g, u = n1 @ block.wg.double().t(), n1 @ block.wu.double().t()
    tol = 10 * 5 * 200 * 2.0 ** -24
    h = g * torch.sigmoid(g) * u
    assert float((served.h.double() - h).abs().max()) <= tol * float(h.abs().max())
    s = x.double() + steps(served.h, 120) @ (wd.double() * wd_scale.double()[:, None]).t()
    assert float((served.s.double() - s).abs().max()) <= tol * float(s.abs().max())
    n2 = norm(s, block.w2, block.b2)
    assert float((served.n.double() - n2).abs().max()) <= tol * float(n2.abs().max())
    want = steps(served.n, 64) @ (wc.double() * wc_scale.double()[:, None]).t() + block.bc.double()
    assert float((got - want).abs().max()) <= tol * float(want.abs().max())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_example_runs(dtype):
    import train_block
    losses = train_block.train(steps=3, dtype=dtype, rows=64, width=64, hidden=120, classes=20)
    assert len(losses) == 3 and all(v == v for v in losses)
