"""GPU parity of dropout (include/dropout.h) against the mask and the formula on the host.

Bounds: an element's product with the scale is rounded once to float32, its sum with the
residual once more (or both at once), and the result once to the element type: u (|x scale|
+ |y|) + h |y|, u = 2^-24.  Which elements are kept is compared exactly."""
import numpy as np
import pytest

import convolution_forward_amd as cf
import mask_reference as mask

torch = pytest.importorskip("torch")

from test_gpu_linear import T, TINY, U, gen, h, rnd, strided, stream  # noqa: E402

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0xFEDCBA9876543210, (1 << 40) + 77


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


def keep_of(m, n, drop, step=0, seed=SEED, offset=OFFSET):
    return torch.from_numpy(mask.keeps(m, n, drop, seed, offset + step)).cuda()


def check(dtype, got, x, r, keep, drop):
    part = torch.where(keep, x.double() * mask.scale(drop), torch.zeros_like(x, dtype=torch.float64))
    want = part if r is None else part + r.double()
    lim = U * (part.abs() + want.abs()) + h(dtype) * want.abs() * (1 + 2 * U) + TINY[dtype]
    assert bool(((got.double() - want).abs() <= lim).all())
    still = torch.zeros_like(got) if r is None else r
    assert torch.equal(got[~keep], still[~keep])
    if r is None and mask.threshold(drop) < 65536:
        assert bool((got[keep & (x != 0)] != 0).all())


def forward(dtype, x, r, drop, y=None, step=None, seed=SEED, offset=OFFSET):
    m, n = x.shape
    y = torch.full((m, n), float("nan"), dtype=T[dtype], device="cuda") if y is None else y
    p = cf.make_dropout_problem(m, n, drop, seed=seed, offset=offset, residual=r is not None,
                                ldx=x.stride(0), ldr=0 if r is None else r.stride(0),
                                ldy=y.stride(0))
    cf.dropout_forward(p, dtype, x, r, y, step, stream())
    return y


def backward(dtype, dy, drop, dx=None, step=None):
    m, n = dy.shape
    dx = torch.full((m, n), float("nan"), dtype=T[dtype], device="cuda") if dx is None else dx
    p = cf.make_dropout_problem(m, n, drop, seed=SEED, offset=OFFSET, ldx=dx.stride(0),
                                ldy=dy.stride(0))
    cf.dropout_backward(p, dtype, dy, dx, step, stream())
    return dx


SIZES = [(1, 1), (3, 7), (5, 8), (1, 9), (64, 100), (777, 1001), (33, 4096), (2, 100_003),
         (5000, 3), (1023, 2048), (4099, 1000)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n", SIZES)
def test_forward_and_backward(dtype, m, n):
    g = gen(m + n)
    x, r = rnd(g, dtype, m, n), rnd(g, dtype, m, n)
    for drop in (0.1, 0.5):
        keep = keep_of(m, n, drop)
        check(dtype, forward(dtype, x, None, drop), x, None, keep, drop)
        check(dtype, forward(dtype, x, r, drop), x, r, keep, drop)
        check(dtype, backward(dtype, x, drop), x, None, keep, drop)


@pytest.mark.parametrize("m,n", [(2051, 4097), (4_200_000, 2), (9, 1_000_003)])
def test_several_runs_a_thread(m, n):
    """Float32 of 2^20 runs and more."""
    assert cf.dropout_describe_variant(cf.make_dropout_problem(m, n, 0.1), "f32").endswith("runs2")
    g = gen(m)
    x, r = rnd(g, "f32", m, n), rnd(g, "f32", m, n)
    keep = keep_of(m, n, 0.1)
    check("f32", forward("f32", x, r, 0.1), x, r, keep, 0.1)
    check("f32", backward("f32", x, 0.1), x, None, keep, 0.1)


@pytest.mark.parametrize("drop", [0.0, 1.0, 2.0 ** -16, 1 - 2.0 ** -16, 2.0 ** -18, 0.9])
def test_probabilities(drop):
    g = gen(1)
    x, r = rnd(g, "f32", 300, 501), rnd(g, "f32", 300, 501)
    keep = keep_of(300, 501, drop)
    if drop in (0.0, 2.0 ** -18):
        assert keep.all() and torch.equal(forward("f32", x, None, drop), x)
    if drop == 1.0:
        assert not keep.any() and torch.equal(forward("f32", x, r, drop), r)
    check("f32", forward("f32", x, r, drop), x, r, keep, drop)
    check("f32", backward("f32", x, drop), x, None, keep, drop)


def test_seed_offset_and_step():
    """offset + step is one 64-bit number, whichever holds it; every half of seed and
    offset enters."""
    x = torch.ones(50, 333, device="cuda")
    step = torch.tensor([5], dtype=torch.int64, device="cuda")
    base = forward("f32", x, None, 0.5, step=step)
    assert torch.equal(base, forward("f32", x, None, 0.5, offset=OFFSET + 5))
    assert torch.equal(base != 0, keep_of(50, 333, 0.5, step=5))
    seen = [base]
    for seed, offset in ((SEED ^ 1, OFFSET + 5), (SEED ^ (1 << 32), OFFSET + 5),
                         (SEED, OFFSET + 6), (SEED, OFFSET + 5 + (1 << 32))):
        y = forward("f32", x, None, 0.5, seed=seed, offset=offset)
        assert torch.equal(y != 0, keep_of(50, 333, 0.5, seed=seed, offset=offset))
        assert all(not torch.equal(y, q) for q in seen)
        seen.append(y)
    step.fill_(-1)  # 2^64 - 1: the sum wraps
    assert torch.equal(forward("f32", x, None, 0.5, step=step, offset=4),
                       forward("f32", x, None, 0.5, offset=3))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,pad,off", [(1001, 6, 1), (64, 7, 3), (4096, 8, 8), (5, 2, 1)])
def test_strides_and_what_lies_between_rows(dtype, n, pad, off):
    g = gen(n)
    x, r = rnd(g, dtype, 37, n), rnd(g, dtype, 37, n)
    (_, xv), (_, rv) = strided(x, pad, off), strided(r, pad + 1, off + 1)
    buf, y = strided(torch.zeros_like(x), pad + 2, off + 2)
    forward(dtype, xv, rv, 0.3, y=y)
    check(dtype, y, x, r, keep_of(37, n, 0.3), 0.3)
    assert int(torch.isnan(buf).sum()) == buf.numel() - y.numel()
    buf, dx = strided(torch.zeros_like(x), pad + 2, off + 2)
    backward(dtype, xv, 0.3, dx=dx)
    check(dtype, dx, x, None, keep_of(37, n, 0.3), 0.3)
    assert int(torch.isnan(buf).sum()) == buf.numel() - dx.numel()


def test_offsets_and_in_place():
    g = gen(3)
    x, r = rnd(g, "f16", 20, 40), rnd(g, "f16", 20, 40)
    want = forward("f16", x, r, 0.4)
    arena = torch.zeros(3, 900, dtype=torch.float16, device="cuda")
    arena[0][7:807], arena[1][8:808] = x.reshape(-1), r.reshape(-1)
    p = cf.make_dropout_problem(20, 40, 0.4, seed=SEED, offset=OFFSET, residual=True,
                                offsets=(7, 8, 1))
    cf.dropout_forward(p, "f16", *arena, None, stream())
    assert torch.equal(arena[2][1:801].view(20, 40), want)
    a, c = x.clone(), r.clone()
    assert torch.equal(forward("f16", a, r, 0.4, y=a), want)
    assert torch.equal(forward("f16", x, c, 0.4, y=c), want)
    grad = backward("f16", x, 0.4)
    a = x.clone()
    assert torch.equal(backward("f16", a, 0.4, dx=a), grad)


def test_not_finite():
    """Kept infinities and NaNs stay, dropped ones are 0."""
    x = torch.full((100, 64), float("inf"), device="cuda")
    x[50:] = float("nan")
    keep = keep_of(100, 64, 0.5)
    y = forward("f32", x, None, 0.5)
    assert torch.equal(y == 0, ~keep)
    assert torch.isinf(y[:50][keep[:50]]).all() and torch.isnan(y[50:][keep[50:]]).all()


def test_no_rows():
    p = cf.make_dropout_problem(0, 8, 0.5)
    assert cf.dropout_forward(p, "f16", None, None, None, None, stream()) == cf.CONV_OK
    assert cf.dropout_backward(p, "f16", None, None, None, stream()) == cf.CONV_OK


def test_gradient_against_differences():
    """The forward is linear in x: any difference is the product with the gradient's mask."""
    g = gen(4)
    x, e, c = (rnd(g, "f32", 40, 50) for _ in range(3))
    d = (forward("f32", x + e, None, 0.3).double() - forward("f32", x, None, 0.3).double()) * c.double()
    got = backward("f32", c, 0.3).double() * e.double()
    # x + e and both outputs are rounded: 4 u of values below 12 times c
    assert float((d - got).abs().max()) <= 4 * U * 12 * 2 * float(c.abs().max())


def test_graph_and_streams():
    """A captured forward and backward draw a new mask on every replay, the same in both."""
    m, n = 300, 1000
    x, r = rnd(gen(0), "bf16", m, n), rnd(gen(1), "bf16", m, n)
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    p = cf.make_dropout_problem(m, n, 0.25, seed=SEED, offset=OFFSET, residual=True)
    q = cf.make_dropout_problem(m, n, 0.25, seed=SEED, offset=OFFSET)

    def call():
        cf.dropout_forward(p, "bf16", x, r, y, step, stream())
        cf.dropout_backward(q, "bf16", x, dx, step, stream())

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        step.add_(1)
    for i in range(4):
        x.copy_(rnd(gen(10 + i), "bf16", m, n))
        call()  # eager, with the step that the replay will see
        want = y.clone(), dx.clone()
        y.zero_(), dx.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
        check("bf16", y, x, r, keep_of(m, n, 0.25, step=i), 0.25)
        check("bf16", dx, x, None, keep_of(m, n, 0.25, step=i), 0.25)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    check("bf16", y, x, r, keep_of(m, n, 0.25, step=4), 0.25)


def test_past_32_bits():
    """More than 2^31 elements."""
    m, n = 300_000, 8_000
    x = torch.ones(m, n, dtype=torch.float16, device="cuda")
    y = forward("f16", x, None, 0.5, y=x)
    for at in (0, 268_000, 268_500, m - 1000):
        words = np.arange(1000) + at
        groups = mask.philox([np.broadcast_to(np.arange(1000, dtype=np.uint64), (1000, 1000)),
                              np.broadcast_to(words[:, None], (1000, 1000)), OFFSET & mask.M32,
                              OFFSET >> 32], [SEED & mask.M32, SEED >> 32])
        bits = np.stack([v for w in groups for v in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 2)
        keep = torch.from_numpy((bits.reshape(1000, n) >= 32768)).cuda()
        assert torch.equal(y[at:at + 1000] != 0, keep)


def test_rows_of_several_launches():
    """Rows of one element, 2^31 and some more of them: two launches' masks follow on."""
    m = 0x7FFF0000 + 3000
    m = min(m, (1 << 31) - 1)
    x = torch.ones(m, 1, dtype=torch.bfloat16, device="cuda")
    y = forward("bf16", x, None, 0.5, y=x)
    at = 0x7FFF0000 - 1000
    words = mask.philox([np.zeros(2000, dtype=np.uint64), np.arange(2000, dtype=np.uint64) + np.uint64(at),
                         OFFSET & mask.M32, OFFSET >> 32], [SEED & mask.M32, SEED >> 32])
    keep = torch.from_numpy((words[0] & np.uint64(0xFFFF)) >= 32768).cuda()
    assert torch.equal(y[at:at + 2000, 0] != 0, keep)
