"""Layer norm backward of rows far from zero whose width does not fill the threads that
hold them: what lies past a row's end takes no part in its sums.

The row's values are all 2^110, with eps = 2^-40: mean and rstd = 2^20 are exact, the
row's own u = (s - mean) rstd are 0, and mean * rstd = 2^130 passes float32's range.  Bounds
as in test_gpu_layer_norm.py; u has no error here."""
import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_layer_norm import (TINY, backward64, close, h, inputs, run_backward,  # noqa: E402
                                 run_forward)

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -40


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


def check(dtype, m, n, once):
    plan = cf.layer_norm_backward_describe_variant(cf.make_layer_norm_problem(m, n), dtype)
    assert plan.endswith(".once") == once, plan
    x, dy, w, b = inputs(dtype, m, n, seed=m + n)
    ds = inputs(dtype, m, n, seed=1)[0]
    x[m // 2] = 2.0 ** 110
    y, s, mean, rstd = run_forward(dtype, x, None, w, b, eps=EPS)
    assert torch.equal(y[m // 2], b) and float(mean[m // 2]) == 2.0 ** 110
    assert float(rstd[m // 2]) == 2.0 ** 20
    got = run_backward(dtype, x, w, mean, rstd, dy, ds, drop=0.3)
    want, err = backward64(x, w, mean, rstd, dy, ds, 0.3)
    for name, a, v, e in zip(("dx", "dr", "dw", "db"), got, want, err):
        assert torch.isfinite(a).all(), name
        close(name, a, v, e, h(dtype), TINY[dtype])


# every number of threads a row, one run of 8 too few, a part of one, and none missing
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 7, 9, 56, 64, 100, 200, 300, 520, 1001, 1024, 2040, 2047, 2100,
                               4095, 5000, 8191, 8193, 20_001])
def test_few_rows(dtype, n):
    check(dtype, 5, n, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n", [(1100, 1), (1100, 9), (1100, 64), (1100, 100), (1100, 200), (1100, 300),
                                 (1100, 520), (1100, 1001), (1100, 2047), (1500, 4095),
                                 (1030, 5000), (600, 8193), (300, 20_001)])
def test_many_rows(dtype, m, n):
    check(dtype, m, n, False)
