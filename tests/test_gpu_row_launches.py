"""Rows that take more than one launch (2^32 work-items are the most of one): a row on
either side of the border is worked on once."""
import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_linear import gen, stream  # noqa: E402
from test_gpu_linear_int8 import quantized  # noqa: E402

pytestmark = pytest.mark.gpu

BORDER = 0xFF000000 // 8  # rows of one launch at 8 threads a row
M = BORDER + 1000


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


def test_layer_norm_in_place():
    """s = x + r over x: a row that was taken twice would be x + 2 r.  A row of one element
    is its own mean, so y is b."""
    x = torch.ones(M, 1, dtype=torch.bfloat16, device="cuda")
    r = torch.full_like(x, 2.0)
    some = slice(BORDER - 500, BORDER + 500)
    x[some], r[some] = (torch.randn(1000, 1, generator=gen(i), device="cuda").bfloat16() for i in range(2))
    want = (x[some].float() + r[some].float()).bfloat16()
    w, b = (torch.full((1,), v, dtype=torch.bfloat16, device="cuda") for v in (1.5, -0.25))
    y = torch.zeros_like(x)
    p = cf.make_layer_norm_problem(M, 1, residual=True)
    assert cf.layer_norm_scratch_size(p, "bf16") == 0
    cf.layer_norm_forward(p, "bf16", x, r, w, b, y, x, stream=stream())
    assert torch.equal(x[some], want)
    assert bool((x[:BORDER - 500] == 3).all()) and bool((x[BORDER + 500:] == 3).all())
    assert bool((y == -0.25).all())


def test_quantize():
    x = torch.ones(M, 1, dtype=torch.bfloat16, device="cuda")
    some = slice(BORDER - 500, BORDER + 500)
    x[some] = torch.randn(1000, 1, generator=gen(3), device="cuda").bfloat16()
    q = torch.zeros(M, 1, dtype=torch.int8, device="cuda")
    scale = torch.zeros(M, device="cuda")
    cf.quantize_rows(cf.make_quantize_problem(M, 1), "bf16", x, q, scale, stream())
    want, want_scale = quantized(x[some])
    assert torch.equal(q[some].cpu(), want) and torch.equal(scale[some].cpu(), want_scale)
    one = torch.ones((), device="cuda") / torch.full((), 127.0, device="cuda")
    for part in (slice(0, BORDER - 500), slice(BORDER + 500, M)):
        assert bool((q[part] == 127).all()) and bool((scale[part] == one).all())
