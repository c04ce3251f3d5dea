"""Layer norm of rows at float32's range: squared distances that pass it leave rstd 0 and y
= b, a sum that passes it NaN; below it nothing is lost."""
import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_layer_norm import inputs, run_forward  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [2, 10, 600, 3000, 20_000, 40_000])
def test_range(dtype, n):
    x, _, w, b = inputs(dtype, 4, n, seed=n)
    side = (torch.arange(n, device="cuda") % 2 * 2 - 1).to(x.dtype)  # -1, 1, ..: n is even
    x[0] = side * 2.0 ** 70
    x[1] = 2.0 ** 127
    x[2] = side * 2.0 ** 50
    y, s, mean, rstd = run_forward(dtype, x, None, w, b)
    assert torch.equal(y[0], b) and float(rstd[0]) == 0.0 and float(mean[0]) == 0.0
    assert torch.isnan(y[1]).all()
    # mean 0, deviation 2^50: all steps but the last rounding and w's sum with b are exact
    assert float(mean[2]) == 0.0 and float(rstd[2]) == 2.0 ** -50
    want = (side.float() * w.float() + b.float()).to(x.dtype)
    assert torch.equal(y[2], want)
    assert torch.isfinite(y[3]).all()
