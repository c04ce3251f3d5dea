"""GPU parity of gradient clipping (include/grad_clip.h) over lists of more tensors
than one launch takes, whose partial norms a launch of its own joins, and of
tensors at every element address.  Bounds as in test_gpu_grad_clip.py."""
import math

import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_grad_clip import T, check, clip, make

pytestmark = pytest.mark.gpu

# more than 112 tensors and more than 1024 partial norms: several launches, joined
LISTS = [[20_000] * 113, [100_000] * 300, [1500 + 7 * i for i in range(700)]]


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lengths", LISTS, ids=lambda v: f"{len(v)}x{max(v)}")
def test_joined_lists(lengths, dtype, p):
    grads = make(lengths, dtype)
    outs = [torch.full_like(g, 7.0) for g in grads]
    for max_norm in (0.05, 1e9):
        check(grads, outs, clip(grads, outs, dtype, norm=p, max_norm=max_norm), p, max_norm)
    alone = clip(grads, None, dtype, norm=p)
    assert torch.equal(alone, clip(grads, outs, dtype, norm=p, max_norm=0.05))
    kept = [g.clone() for g in grads]
    check(kept, grads, clip(grads, grads, dtype, norm=p, max_norm=0.05), p, 0.05)


@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("at", [0, 111, 112, 299])
def test_joined_lists_with_one_large_element(at, p):
    """An element that outweighs the rest, in the first and in later launches."""
    grads = make([100_000] * 300, "f32", scale=1e-6)
    grads[at][99_999] = -1e6
    outs = [torch.empty_like(g) for g in grads]
    check(grads, outs, clip(grads, outs, "f32", norm=p, max_norm=2.0), p, 2.0)


@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("at", [0, 112, 299])
def test_joined_lists_with_nan_and_infinity(at, p):
    grads = make([100_000] * 300, "bf16")
    outs = [torch.zeros_like(g) for g in grads]
    grads[at][7] = math.inf
    assert float(clip(grads, outs, "bf16", norm=p)) == math.inf
    assert sum(int(torch.isnan(o).sum()) for o in outs) == 1 and math.isnan(float(outs[at][7]))
    assert not any(bool((o == o).logical_and(o != 0).any()) for o in outs)
    grads[at][8] = math.nan
    assert math.isnan(float(clip(grads, outs, "bf16", norm=p)))
    assert all(bool(torch.isnan(o).all()) for o in outs)
