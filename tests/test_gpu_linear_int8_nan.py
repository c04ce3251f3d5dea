"""What becomes of a scale that is NaN (a token that held an infinity or a NaN) under
every activation, on every kind of kernel: its outputs are NaN, but for relu, whose
comparison fails and gives 0; no other output changes."""
import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_linear import ACTS  # noqa: E402
from test_gpu_linear_int8 import forward, operands, quantize  # noqa: E402

pytestmark = pytest.mark.gpu

# streamed, gathered small tiles, split, small tiles, large tiles, the last of them cut
SIZES = [(5, 100, 256, "stream"), (129, 130, 131, "tile64x64"), (64, 256, 4096, "split"),
         (300, 520, 384, "tile"), (2229, 3712, 1728, "tile256x256"), (2033, 9750, 1552, "cut")]


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k,plan", SIZES)
def test_a_token_that_was_not_finite(m, n, k, plan, dtype, act):
    x, xs, w, ws, b, r = operands(dtype, m, n, k)
    bad = [0, m // 2, m - 1]
    token = torch.zeros(2, k, device="cuda")
    token[0, k // 2], token[1, 0] = float("inf"), float("nan")
    q, s = quantize("f32", token)
    assert torch.isnan(s).all() and not q.any()
    good = torch.ones(m, dtype=torch.bool, device="cuda")
    good[bad] = False
    x[bad], other = 0, xs.clone()
    other[bad] = s[[0, 1, 0]]
    for res in ("none", "before", "after"):
        args = (b, None if res == "none" else r)
        use = []
        want = forward(dtype, x, xs, w, ws, *args, act=act, res=res, use=use)
        name = cf.linear_int8_describe_variant(use[0][0], dtype)
        assert plan in name, name
        got = forward(dtype, x, other, w, ws, *args, act=act, res=res)
        assert torch.equal(got[good], want[good])
        if act != "relu":
            assert torch.isnan(got[bad]).all(), res
        else:
            assert torch.equal(got[bad], r[bad] if res == "after" else torch.zeros_like(r[bad])), res


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k,plan", SIZES)
def test_a_channel_whose_scale_is_not_a_number(m, n, k, plan, act):
    x, xs, w, ws, b, _ = operands("bf16", m, n, k)
    bad = [0, n // 2, n - 1]
    good = torch.ones(n, dtype=torch.bool, device="cuda")
    good[bad] = False
    other = ws.clone()
    other[bad] = float("nan")
    want = forward("bf16", x, xs, w, ws, b, act=act)
    got = forward("bf16", x, xs, w, other, b, act=act)
    assert torch.equal(got[:, good], want[:, good])
    assert bool((got[:, bad] == 0).all()) if act == "relu" else torch.isnan(got[:, bad]).all()
