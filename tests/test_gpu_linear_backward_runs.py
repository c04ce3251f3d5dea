"""GPU: gradients asked for one by one where both would share a launch of large tiles,
and reruns of the gradients, bit for bit."""
import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_linear import T, backward, gated_back, gen, rnd, whole

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


@pytest.mark.parametrize("act", ["identity", "relu"])
@pytest.mark.parametrize("m,n,k", [(960, 896, 4352), (1728, 1728, 2112)])
def test_alone_and_together(m, n, k, act):
    dtype = "f16"
    g = gen(m)
    x, w, z, dy = (whole(g, dtype, *s) for s in ((m, k), (n, k), (m, n), (m, n)))
    d = dy.float() * ((z > 0).float() if act == "relu" else 1.0)
    for want in ("xw", "x", "w"):
        dx, dw, _, _ = backward(dtype, x, w, z, dy, act=act, want=want)
        assert dx is None or torch.equal(dx, (d @ w.float()).to(T[dtype]))
        assert dw is None or torch.equal(dw, (d.t() @ x.float()).to(T[dtype]))


@pytest.mark.parametrize("m,n,k", [(4096, 4096, 1024), (4096, 2816, 2048), (1000, 1001, 240), (300, 264, 4104)])
def test_reruns(m, n, k):
    """Sums in a fixed order: the same bits again, with other work on the card between."""
    for dtype in ("bf16", "f32"):
        g = gen(k)
        x, w, u = rnd(g, dtype, m, k), rnd(g, dtype, n, k, scale=k ** -0.5), rnd(g, dtype, n, k, scale=k ** -0.5)
        z, v, dy = rnd(g, dtype, m, n), rnd(g, dtype, m, n), rnd(g, dtype, m, n)
        first = backward(dtype, x, w, z, dy, act="gelu_tanh")[:3] + gated_back(dtype, x, w, u, z, v, dy)
        for i in range(3):
            backward(dtype, rnd(g, dtype, m, k), w, v, dy, act="silu")
            again = backward(dtype, x, w, z, dy, act="gelu_tanh")[:3] + gated_back(dtype, x, w, u, z, v, dy)
            assert all(torch.equal(a, b) for a, b in zip(first, again)), (dtype, i)
