"""The order of the sums of gradient clipping (include/grad_clip.h) does not depend on
where the tensors lie.  Bounds as in test_gpu_grad_clip.py."""
import math

import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_grad_clip import T, check, clip, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


def test_order_of_the_sum_is_the_same_at_every_address():
    """Elements of a tensor join the sum in an order that its address does not change.
    1 + 2^-24 lies between two float32 numbers; four elements of 0.9 * 2^-53 vanish
    when they are added to it one by one, and move the result when they are added up
    before, so the norm tells the orders apart."""
    n = (1 << 21) + 2048  # chunks of 2048
    g = torch.zeros(n + 8, device="cuda")
    norms = []
    for off in range(5):
        v = g[off:off + n]
        g.zero_()
        v[0], v[1] = 1.0, 2.0 ** -24
        v[2] = v[3] = v[1026] = v[1027] = 0.9 * 2.0 ** -53
        norms.append(float(clip([v], None, "f32", norm=1)))
    assert norms == norms[:1] * 5


@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_views_of_one_flat_buffer(dtype, p):
    """Tensors of odd lengths behind one another, so that most start off 16 bytes."""
    lengths = [1, 3, 7, 1023, 4097, 65_537, 8, 30_001, 5]
    flat, out = (torch.full((sum(lengths),), 7.0, dtype=T[dtype], device="cuda") for _ in range(2))
    grads, outs = list(flat.split(lengths)), list(out.split(lengths))
    for g, v in zip(grads, make(lengths, dtype)):
        g.copy_(v)
    check(grads, outs, clip(grads, outs, dtype, norm=p, max_norm=0.05), p, 0.05)
    kept = [g.clone() for g in grads]
    check(kept, grads, clip(grads, grads, dtype, norm=p, max_norm=0.05), p, 0.05)
