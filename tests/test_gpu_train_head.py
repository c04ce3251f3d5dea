"""The training example: its first step's gradients against the formulas in 64 bits,
and its loss over some steps."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_gradients_of_a_step():
    """float32: sums of at most 200 terms in each of five layers, relative to their
    largest values 200 * 2^-24 each, a factor of 10 for the layers' slopes and sizes."""
    import train_head
    rows, width, hidden, classes = 96, 64, 120, 33
    head = train_head.Head(rows, width, hidden, classes, "f32", seed=3, max_norm=1e9)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=gen, device="cuda")
    dlogits = torch.randn(rows, classes, generator=gen, device="cuda") / rows
    w = [t.double() for t in head.weights]
    xd, dl = x.double(), dlogits.double()
    g, u = xd @ w[0].t(), xd @ w[1].t()
    q = torch.sigmoid(g)
    h = g * q * u
    y = xd + h @ w[2].t()
    logits = y @ w[3].t() + w[4]
    dy = dl @ w[3]
    dh = dy @ w[2]
    want = [(dh * u * q * (1 + g * (1 - q))).t() @ xd, (dh * g * q).t() @ xd, dy.t() @ h, dl.t() @ y,
            dl.sum(0)]
    tol = 10 * 5 * 200 * 2.0 ** -24
    got = head.forward(x)
    assert float((got.double() - logits).abs().max()) <= tol * float(logits.abs().max())
    head.backward(x, dlogits)
    for a, b in zip(head.grads, want):
        assert float((a.double() - b).abs().max()) <= tol * float(b.abs().max())
    norm = sum(float((b ** 2).sum()) for b in want) ** 0.5
    assert abs(float(head.norm) - norm) <= tol * norm


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_loss_falls(dtype):
    import train_head
    losses = train_head.train(steps=40, dtype=dtype)
    assert all(v == v for v in losses)
    assert sum(losses[-5:]) < 0.9 * sum(losses[:5])
