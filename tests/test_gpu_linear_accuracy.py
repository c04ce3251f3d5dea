"""GPU accuracy of the activations and slopes of the linear and gated calls
(include/linear.h) relative to their own size, against 64-bit definitions.

Bounds: 16 float32 ulps of the value and of the argument.  An ulp of y is at most
2^-23 |y|; an error of 16 ulps in the argument v moves act by 16 * 2^-23 |v act'(v)|
and a slope by 16 * 2^-23 |v act''(v)|.  Beside that the rounding to the element
type, and 2^-119 (below it a result may be 0)."""
import math

import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_linear import ACTS, T, act64, backward, forward, gated, gated_back, h

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -23
FLOOR = {"f32": 2.0 ** -119, "f16": 2.0 ** -25, "bf16": 2.0 ** -119}
SMOOTH = ["tanh", "sigmoid", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


def value_and_slope(v, act):
    if act == "tanh":  # 1 - tanh^2 cancels in 64 bits too
        return torch.tanh(v), 4 * torch.sigmoid(2 * v) * torch.sigmoid(-2 * v)
    return act64(v, act)


def within(name, got, want, err):
    bad = ~((got - want).abs() <= err)
    if bad.any():
        i = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()}, first {got.flatten()[i].item()} "
                             f"for {want.flatten()[i].item()}, bound {err.flatten()[i].item():.3g}")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", SMOOTH)
def test_relative_to_the_value(act, dtype):
    """y = act(x) through a product with one, and act'(z) as the gradient of a residual."""
    v = torch.cat([torch.linspace(-14, 14, 2801), torch.tensor([20.0, -20, 40, -40, 60, -60, 80, -80])])
    x = v.to(T[dtype]).cuda().view(-1, 1)
    one = torch.ones(1, 1, dtype=T[dtype], device="cuda")
    v = x.double().requires_grad_(True)
    want, slope = value_and_slope(v, act)
    second = torch.autograd.grad(slope.sum(), v)[0]
    v, want, slope = v.detach(), want.detach(), slope.detach()
    y = forward(dtype, x, one, act=act).double()
    within("value", y, want, 16 * ULP * (want.abs() + (v * slope).abs()) + h(dtype) * want.abs() + FLOOR[dtype])
    d = backward(dtype, x, one, x, torch.ones_like(x), act=act, res="before", want="r")[3].double()
    within("slope", d, slope,
           16 * ULP * (slope.abs() + (v * second).abs()) + h(dtype) * slope.abs() + FLOOR[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", SMOOTH)
def test_slopes_of_huge_arguments(act, dtype):
    """Arguments whose square or cube overflows float32: every slope is its limit."""
    v = [s * q for q in (1e10, 7e12, 1e13, 1.8e19, 2e19, 1e25, 3e38) for s in (1, -1)]
    x = torch.tensor(v, dtype=T[dtype], device="cuda").view(-1, 1)
    one = torch.ones(1, 1, dtype=T[dtype], device="cuda")
    want = (x > 0).double() * (0.0 if act in ("tanh", "sigmoid") else 1.0)
    d = backward(dtype, x, one, x, torch.ones_like(x), act=act, res="before", want="r")[3]
    assert torch.equal(d.double(), want)
    # the gate's gradient dg = dh pu act'(pg), as its column sums of one row each
    for i in range(len(v)):
        pg = x[i:i + 1].contiguous()
        dbg = gated_back(dtype, one, one, one, pg, one, one, act=act, want="b")[3]
        assert float(dbg) == float(want[i]), v[i]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
def test_nan_stays_nan(act, dtype):
    """A NaN sum is a NaN output of every activation but relu, whose NaN is 0; beside
    it the other rows are what they are without it."""
    x = torch.tensor([0.5, math.nan, -0.5], dtype=T[dtype], device="cuda").view(-1, 1)
    one = torch.ones(1, 1, dtype=T[dtype], device="cuda")
    y = forward(dtype, x, one, act=act).flatten()
    hid = gated(dtype, x, one, one, act=act).flatten()
    nan = act != "relu"
    assert torch.isnan(y).tolist() == [False, nan, False]
    assert nan or float(y[1]) == 0.0
    assert torch.isnan(hid).tolist() == [False, True, False]  # the other factor is NaN too
    # du = dh act(pg)
    dbu = gated_back(dtype, one, one, one, x[1:2].contiguous(), one, one, act=act, want="b")[4]
    assert math.isnan(float(dbu)) == nan


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_clip_of_bounds_and_infinities(dtype):
    x = torch.tensor([-math.inf, -0.75, -0.0, 1.25, 7.0, math.inf], dtype=T[dtype], device="cuda").view(-1, 1)
    one = torch.ones(1, 1, dtype=T[dtype], device="cuda")
    y = forward(dtype, x, one, act="clip").flatten().tolist()
    assert y == [-0.75, -0.75, 0.0, 1.25, 1.25, 1.25]
    y = forward(dtype, x, one, act="hard_sigmoid").flatten().tolist()
    assert y[0] == 0.0 and y[4:] == [1.0, 1.0]
