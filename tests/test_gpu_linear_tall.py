"""GPU parity of the linear and gated calls with more rows than one launch takes:
row counts up to the largest that is valid.  Whole numbers in a repeating pattern of
prime length, so that a row in the wrong place shows; results are compared exactly."""
import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_linear import T, gen, scratch, stream, whole

pytestmark = pytest.mark.gpu

PERIOD = 65_521
MAX = 2 ** 31 - 1


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()
    yield
    torch.cuda.empty_cache()


def tall(pattern, m):
    """m rows that repeat the pattern's."""
    t = torch.empty(m, pattern.shape[1], dtype=pattern.dtype, device="cuda")
    full = m // PERIOD * PERIOD
    t[:full].view(-1, *pattern.shape).copy_(pattern.expand(m // PERIOD, -1, -1))
    t[full:].copy_(pattern[:m - full])
    return t


def repeats(t, pattern):
    m, step = t.shape[0], 1024 * PERIOD
    for i in range(0, m, step):
        part = t[i:i + step]
        full = part.shape[0] // PERIOD * PERIOD
        if not bool((part[:full].view(-1, *pattern.shape) == pattern).all()):
            return False
        if not torch.equal(part[full:], pattern[:part.shape[0] - full]):
            return False
    return True


@pytest.mark.parametrize("dtype,m", [("f32", 2 ** 30 + 77), ("f16", MAX)])
def test_most_rows(dtype, m):
    print(f"[tall] {dtype} {m}", flush=True)
    base, w = whole(gen(1), dtype, PERIOD, 1, lo=-9, hi=10), whole(gen(2), dtype, 1, 1, lo=3, hi=4)
    x = tall(base, m)
    y = torch.full((m, 1), 99.0, dtype=T[dtype], device="cuda")
    p = cf.make_linear_problem(m, 1, 1)
    size = cf.linear_scratch_size(p, dtype)
    cf.linear_forward(p, dtype, x, w, None, None, y, None, scratch(size), size, stream())
    assert repeats(y, base * w[0, 0])


@pytest.mark.parametrize("kn", [False, True])
def test_every_operand_follows_its_rows(kn):
    """Two launches: residual, saved sums and the gradient dx beside x and y."""
    m, n, k, dtype = 2 ** 28 + 300, 8, 8, "f16"
    print(f"[tall] {m} {n} {k} {dtype} kn={kn}", flush=True)
    g = gen(3)
    base, res = whole(g, dtype, PERIOD, k), whole(g, dtype, PERIOD, n, lo=-8, hi=9)
    w, b = whole(g, dtype, *((k, n) if kn else (n, k))), whole(g, dtype, n)
    x, r = tall(base, m), tall(res, m)
    y, z = (torch.empty(m, n, dtype=T[dtype], device="cuda") for _ in range(2))
    p = cf.make_linear_problem(m, n, k, act="relu", bias=True, residual="before", save_z=True,
                               w_layout="kn" if kn else "nk")
    size = cf.linear_scratch_size(p, dtype)
    cf.linear_forward(p, dtype, x, w, b, r, y, z, scratch(size), size, stream())
    wd = w.double() if kn else w.double().t()
    want = base.double() @ wd + b.double() + res.double()
    assert repeats(z, want.to(T[dtype])) and repeats(y, want.clamp(min=0).to(T[dtype]))
    p = cf.make_linear_problem(m, n, k, act="relu", residual="after", w_layout="kn" if kn else "nk")
    cf.linear_forward(p, dtype, x, w, None, r, y, None, scratch(size), size, stream())
    assert repeats(y, ((base.double() @ wd).clamp(min=0) + res.double()).to(T[dtype]))
    # dx = (dy where z > 0) w
    size = cf.linear_backward_scratch_size(p, dtype)
    cf.linear_backward(p, dtype, None, w, z, r, y, None, None, None, scratch(size), size, stream())
    d = res.double() * (want > 0).double()
    assert repeats(y, (d @ wd.t()).to(T[dtype]))


def test_both_gradients_of_many_rows():
    """dy is zero but for rows at both ends and where the second launch starts."""
    m, n, k, dtype = 2 ** 28 + 300, 16, 8, "f16"
    print(f"[tall gradients] {m} {n} {k} {dtype}", flush=True)
    g = gen(5)
    x = tall(whole(g, dtype, PERIOD, k), m)
    w, some = whole(g, dtype, n, k), whole(g, dtype, 40, n)
    rows = torch.cat([torch.arange(10), 2 ** 28 - 10 + torch.arange(20), m - 10 + torch.arange(10)]).cuda()
    dy = torch.zeros(m, n, dtype=T[dtype], device="cuda")
    dy[rows] = some
    dx, dw = torch.full((m, k), 7.0, dtype=T[dtype], device="cuda"), torch.empty_like(w)
    p = cf.make_linear_problem(m, n, k)
    size = cf.linear_backward_scratch_size(p, dtype)
    cf.linear_backward(p, dtype, x, w, None, dy, dx, dw, None, None, scratch(size), size, stream())
    assert torch.equal(dx[rows], (some.double() @ w.double()).to(T[dtype]))
    assert torch.equal(dw, (some.double().t() @ x[rows].double()).to(T[dtype]))
    dx[rows] = 0
    assert not any(bool(part.any()) for part in dx.split(1 << 26))


def test_gated_follows_its_rows():
    m, f, k, dtype = 2 ** 28 + 300, 8, 8, "bf16"
    print(f"[tall gated] {m} {f} {k} {dtype}", flush=True)
    g = gen(4)
    base = whole(g, dtype, PERIOD, k, lo=-1, hi=2)
    wg, wu = (whole(g, dtype, f, k, lo=-1, hi=2) for _ in range(2))
    x = tall(base, m)
    hid, pg, pu = (torch.empty(m, f, dtype=T[dtype], device="cuda") for _ in range(3))
    p = cf.make_gated_problem(m, f, k, act="relu", save=True)
    size = cf.gated_scratch_size(p, dtype)
    cf.gated_forward(p, dtype, x, wg, wu, None, None, hid, pg, pu, scratch(size), size, stream())
    a, b = base.double() @ wg.double().t(), base.double() @ wu.double().t()
    assert repeats(pg, a.to(T[dtype])) and repeats(pu, b.to(T[dtype]))
    assert repeats(hid, (a.clamp(min=0) * b).to(T[dtype]))
    x = None
    dh = tall(whole(g, dtype, PERIOD, f), m)
    dx = torch.empty(m, k, dtype=T[dtype], device="cuda")
    size = cf.gated_backward_scratch_size(p, dtype)
    cf.gated_backward(p, dtype, None, wg, wu, pg, pu, dh, dx, None, None, None, None, scratch(size),
                      size, stream())
    dhb = dh[:PERIOD].double()
    dg, du = dhb * b * (a > 0).double(), dhb * a.clamp(min=0)
    assert repeats(dx, (dg @ wg.double() + du @ wu.double()).to(T[dtype]))
