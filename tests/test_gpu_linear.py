"""GPU parity of the linear and gated feed-forward calls (include/linear.h),
forward and backward, against a plain implementation in 64 bits.

Bounds, per element, with u = 2^-24 (float32 sums) and h = eps / 2 of the element
type (one rounding where a value is stored):
 - a sum of n products whose absolute values add up to S is off by at most
   (n + 2) u S (any order; the products of 16-bit operands are exact, the two
   more are a bias and a residual);
 - an activation passes that on with its largest slope (below 1.2 for each of
   them), and adds its own evaluation: 16 float32 ulps of its value and of its
   argument (exp2 of a scaled argument, a reciprocal);
 - dz, dg and du are rounded once (h) before they enter a product;
 - the result is rounded once: h |y|, or half the least subnormal step.
Small whole numbers make every step exact: those results are compared bit for bit.
"""
import math

import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
ACTS = ("identity", "relu", "tanh", "sigmoid", "silu", "hard_sigmoid", "hard_swish", "clip",
        "leaky_relu", "gelu", "gelu_tanh")
PARAM = {"hard_sigmoid": (0.2, 0.5), "clip": (-0.75, 1.25), "leaky_relu": (0.01, 0.0)}
SLOPE = 1.2


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


def h(dtype):
    return torch.finfo(T[dtype]).eps / 2


def stream():
    return torch.cuda.current_stream().cuda_stream


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, dtype, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(T[dtype])


def whole(g, dtype, *shape, lo=-2, hi=3):
    return torch.randint(lo, hi, shape, generator=g, device="cuda").to(T[dtype])


def strided(t, pad, off):
    """t's values in rows pad elements further apart, off elements into a buffer
    whose other elements are NaN; returns (buffer, view)."""
    rows, cols = t.shape
    ld = cols + pad
    buf = torch.full((off + rows * ld + 3,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[off:off + rows * ld].view(rows, ld)[:, :cols]
    v.copy_(t)
    return buf, v


def scratch(size):
    return torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None


def act64(v, act):
    """Activation and slope in 64 bits."""
    one = torch.ones_like(v)
    a, b = PARAM.get(act, (0.0, 0.0))
    if act == "relu":
        return v.clamp(min=0), (v > 0).double()
    if act == "tanh":
        return torch.tanh(v), 1 - torch.tanh(v) ** 2
    if act == "sigmoid":
        q = torch.sigmoid(v)
        return q, q * torch.sigmoid(-v)
    if act == "silu":
        q = torch.sigmoid(v)
        return v * q, q * (1 + v * torch.sigmoid(-v))
    if act == "hard_sigmoid":
        # the parameters as the struct holds them, in float32
        a, b = (torch.tensor(q, dtype=torch.float32).double().item() for q in (a, b))
        w = a * v + b
        return w.clamp(0, 1), torch.where((w > 0) & (w < 1), a * one, 0 * one)
    if act == "hard_swish":
        y = torch.where(v >= 3, v, torch.where(v <= -3, 0 * v, v * (v + 3) / 6))
        return y, torch.where(v >= 3, one, torch.where(v <= -3, 0 * one, (2 * v + 3) / 6))
    if act == "clip":
        return v.clamp(a, b), ((v > a) & (v < b)).double()
    if act == "leaky_relu":
        a = torch.tensor(a, dtype=torch.float32).double().item()
        return torch.where(v >= 0, v, a * v), torch.where(v >= 0, one, a * one)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-v * math.sqrt(0.5))
        return v * cdf, cdf + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        w = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        s = torch.sigmoid(w)
        dw = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v * v)
        return v * s, s + v * s * torch.sigmoid(-w) * dw
    return v, one


def act_error(v, y, zerr, act):
    if act == "identity":
        return zerr
    return SLOPE * zerr + 16 * U * (v.abs() + y.abs())


def close(name, got, want, err, dtype):
    """err: before the final rounding."""
    d = (got.double() - want).abs()
    lim = err + h(dtype) * (want.abs() + err) + TINY[dtype]
    bad = ~(d <= lim)
    if bad.any():
        i = tuple(int(q) for q in torch.nonzero(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} out of bounds, first at "
                             f"{i}: {got[i].item()} for {want[i].item()}, error {d[i].item():.3g} "
                             f"bound {lim[i].item():.3g}")


def forward(dtype, x, w, b=None, r=None, y=None, act="identity", res="none", kn=False,
            save=False, offs=(0,) * 6, use=None):
    """x, w, r: 2-D views (their strides are passed on)."""
    m, k = x.shape
    n = w.shape[1] if kn else w.shape[0]
    if y is None:
        y = torch.full((m, n), float("nan"), dtype=T[dtype], device="cuda")
    z = torch.full((m, n), float("nan"), dtype=T[dtype], device="cuda") if save else None
    a, be = PARAM.get(act, (0.0, 0.0))
    p = cf.make_linear_problem(m, n, k, act=act, alpha=a, beta=be, bias=b is not None, residual=res,
                               save_z=save, w_layout="kn" if kn else "nk", ldx=x.stride(0),
                               ldw=w.stride(0), ldr=0 if r is None else r.stride(0),
                               ldy=y.stride(0), offsets=offs)
    size = cf.linear_scratch_size(p, dtype)
    s = scratch(size)
    cf.linear_forward(p, dtype, x, w, b, r, y, z, s, size, stream())
    if use is not None:
        use.append((p, s, size))
    return (y, z) if save else y


# sizes: one of everything, pieces of 16 and 64, one more and one less than tiles,
# every kernel (streamed up to 32 rows; 64, 128 and 256 tiles; split k)
SIZES = [(1, 1, 1), (1, 16, 64), (1, 1000, 2048), (2, 33, 7), (15, 17, 129), (16, 64, 1024),
         (17, 40, 24), (32, 100, 333), (33, 64, 64), (40, 65, 520), (64, 130, 4096), (65, 72, 8),
         (127, 129, 200), (200, 264, 1000), (300, 520, 127), (1000, 1001, 66), (4096, 4112, 80),
         (4090, 4104, 200)]


@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_whole_numbers_are_exact(m, n, k, dtype, kn):
    """Sums below 2^24 of whole products: float32 holds them exactly, so the
    output is their one rounding to the element type."""
    g = gen(m * 7 + n * 3 + k)
    print(f"[linear exact] {m} {n} {k} {dtype} kn={kn}", flush=True)
    x, w = whole(g, dtype, m, k), whole(g, dtype, *((k, n) if kn else (n, k)))
    b, r = whole(g, dtype, n, lo=-8, hi=9), whole(g, dtype, m, n, lo=-8, hi=9)
    y, z = forward(dtype, x, w, b, r, act="relu", res="before", kn=kn, save=True)
    want = x.double() @ (w.double() if kn else w.double().t()) + b.double() + r.double()
    assert torch.equal(z, want.to(T[dtype]))
    assert torch.equal(y, want.clamp(min=0).to(T[dtype]))
    y = forward(dtype, x, w, None, r, act="relu", res="after", kn=kn)
    want = (want - b.double() - r.double()).clamp(min=0) + r.double()
    assert torch.equal(y, want.to(T[dtype]))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(3, 50, 96), (130, 72, 160)])
def test_linear_activations(m, n, k, act, dtype):
    g = gen(ACTS.index(act))
    x, w = rnd(g, dtype, m, k), rnd(g, dtype, n, k, scale=3 * k ** -0.5)
    b, r = rnd(g, dtype, n), rnd(g, dtype, m, n)
    xd, wd, bd, rd = x.double(), w.double(), b.double(), r.double()
    mass = xd.abs() @ wd.abs().t() + bd.abs() + rd.abs()
    zerr = (k + 2) * U * mass
    for res in ("before", "after"):
        y, z = forward(dtype, x, w, b, r, act=act, res=res, save=True)
        v = xd @ wd.t() + bd + (rd if res == "before" else 0)
        close("z", z, v, zerr, dtype)
        a = act64(v, act)[0]
        err = act_error(v, a, zerr, act)
        if res == "after":
            a, err = a + rd, err + U * (a.abs() + rd.abs())
        close("y", y, a, err, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("m,n,k,pad,off", [(5, 48, 64, 8, 8), (5, 47, 61, 3, 1), (90, 136, 192, 16, 0),
                                           (90, 135, 191, 1, 5), (90, 136, 192, 5, 2)])
def test_linear_strides_and_offsets(m, n, k, pad, off, kn, dtype):
    """Rows apart, operands inside larger buffers of NaN, aligned and not: the
    NaN around the operands is never read into a result, and none around the
    outputs is overwritten."""
    g = gen(off + pad)
    x, w = whole(g, dtype, m, k), whole(g, dtype, *((k, n) if kn else (n, k)))
    b, r = whole(g, dtype, n), whole(g, dtype, m, n)
    (_, xv), (_, wv), (_, rv) = (strided(t, pad, off) for t in (x, w, r))
    ybuf, yv = strided(torch.zeros(m, n, dtype=T[dtype], device="cuda"), pad, off)
    forward(dtype, xv, wv, b, rv, y=yv, res="before", kn=kn)
    want = x.double() @ (w.double() if kn else w.double().t()) + b.double() + r.double()
    assert torch.equal(yv, want.to(T[dtype]))
    yv.zero_()
    assert int(torch.isnan(ybuf).sum()) == ybuf.numel() - m * n
    # the same through element offsets from the buffers' start
    xb, _ = strided(x, pad, off)
    wb, _ = strided(w, pad, off)
    yb, yv = strided(torch.zeros(m, n, dtype=T[dtype], device="cuda"), pad, off)
    p = cf.make_linear_problem(m, n, k, bias=True, w_layout="kn" if kn else "nk", ldx=k + pad,
                               ldw=(n if kn else k) + pad, ldy=n + pad,
                               offsets=(off, off, 0, 0, off, 0))
    size = cf.linear_scratch_size(p, dtype)
    cf.linear_forward(p, dtype, xb, wb, b, None, yb, None, scratch(size), size, stream())
    assert torch.equal(yv, (want - r.double()).to(T[dtype]))


@pytest.mark.parametrize("m,n,k", [(4, 64, 128), (100, 200, 256), (70, 64, 2048)])
def test_linear_residual_in_place_and_rerun(m, n, k):
    g = gen(3)
    x, w, r = rnd(g, "bf16", m, k), rnd(g, "bf16", n, k), rnd(g, "bf16", m, n)
    apart = forward("bf16", x, w, None, r, res="after", act="silu")
    assert torch.equal(apart, forward("bf16", x, w, None, r, res="after", act="silu"))
    y = r.clone()
    forward("bf16", x, w, None, y, y=y, res="after", act="silu")
    assert torch.equal(apart, y)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(6, 40, 72), (150, 140, 264), (90, 80, 2056)])
def test_linear_nan_and_infinity_stay_in_their_row(m, n, k, dtype):
    g = gen(5)
    x, w = whole(g, dtype, m, k), whole(g, dtype, n, k, lo=1, hi=3)
    clean = forward(dtype, x, w)
    x2 = x.clone()
    x2[2, k - 1] = float("nan")
    x2[4, 0] = float("inf")
    y = forward(dtype, x2, w)
    assert torch.isnan(y[2]).all() and torch.isinf(y[4]).all()
    keep = [i for i in range(m) if i not in (2, 4)]
    assert torch.equal(y[keep], clean[keep])
    w2 = w.clone()
    w2[7, k - 1] = float("nan")
    y = forward(dtype, x, w2)
    assert torch.isnan(y[:, 7]).all()
    cols = [i for i in range(n) if i != 7]
    assert torch.equal(y[:, cols], clean[:, cols])


def test_linear_past_32_bits():
    """Rows 2^20 elements apart: the last ones lie past 2^31 elements, in x, y and
    the weights alike."""
    n, k, m, ld = 2100, 64, 2100, 1 << 20
    g = gen(8)
    x, w = whole(g, "f16", m, k), whole(g, "f16", n, k)
    buf = torch.zeros(m * ld, dtype=torch.float16, device="cuda")
    xv = buf.view(m, ld)[:, :k]
    wv = buf.view(m, ld)[:, 128:128 + k]
    yv = buf.view(m, ld)[:, 512:512 + n]
    xv.copy_(x)
    wv.copy_(w)
    forward("f16", xv, wv, y=yv)
    want = (x.double() @ w.double().t()).to(torch.float16)
    assert torch.equal(yv, want)


def test_linear_other_stream_and_no_rows():
    x = torch.empty(0, 16, dtype=torch.float16, device="cuda")
    w = torch.zeros(8, 16, dtype=torch.float16, device="cuda")
    p = cf.make_linear_problem(0, 8, 16)
    cf.linear_forward(p, "f16", x, w, None, None, torch.empty(0, 8, device="cuda").half())
    dw = torch.full((8, 16), 7.0, dtype=torch.float16, device="cuda")
    db = torch.full((8,), 7.0, dtype=torch.float16, device="cuda")
    size = cf.linear_backward_scratch_size(p, "f16")
    cf.linear_backward(p, "f16", None, w, None, None, None, dw, db, None, scratch(size), size,
                       stream())
    assert not dw.any() and not db.any()
    side = torch.cuda.Stream()
    g = gen(1)
    x, w = whole(g, "f16", 70, 2048), whole(g, "f16", 64, 2048)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y = forward("f16", x, w)
    side.synchronize()
    assert torch.equal(y, (x.double() @ w.double().t()).half())


# ------------------------------------------------------------------ linear gradients

def backward(dtype, x, w, z, dy, act="identity", res="none", kn=False, want="xwbr", back_ld=0):
    m, k = x.shape
    n = dy.shape[1]
    a, be = PARAM.get(act, (0.0, 0.0))
    p = cf.make_linear_problem(m, n, k, act=act, alpha=a, beta=be, residual=res,
                               w_layout="kn" if kn else "nk", ldx=x.stride(0), ldw=w.stride(0),
                               ldy=dy.stride(0), ldz=0 if z is None else z.stride(0),
                               lddx=k + back_ld, lddw=(n if kn else k) + back_ld)
    nan = lambda *s: torch.full(s, float("nan"), dtype=T[dtype], device="cuda")  # noqa: E731
    dx = nan(m, k + back_ld)[:, :k] if "x" in want else None
    dw = nan(w.shape[0], w.shape[1] + back_ld)[:, :w.shape[1]] if "w" in want else None
    db = nan(n) if "b" in want else None
    dr = nan(m, n) if "r" in want and res != "none" else None
    size = cf.linear_backward_scratch_size(p, dtype)
    cf.linear_backward(p, dtype, x, w, z, dy, dx, dw, db, dr, scratch(size), size, stream())
    return dx, dw, db, dr


@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 40, 64), (5, 17, 33), (31, 64, 130), (64, 72, 40),
                                   (129, 130, 131), (200, 264, 136), (2000, 65, 64),
                                   (1030, 136, 264), (300, 4104, 4112), (4112, 4104, 72)])
def test_linear_backward_whole_numbers_are_exact(m, n, k, dtype, kn):
    g = gen(m + n + k)
    print(f"[linear backward exact] {m} {n} {k} {dtype} kn={kn}", flush=True)
    x, w = whole(g, dtype, m, k), whole(g, dtype, *((k, n) if kn else (n, k)))
    z, dy = whole(g, dtype, m, n), whole(g, dtype, m, n)
    for act, pad in (("identity", 0), ("relu", 8)):
        dx, dw, db, dr = backward(dtype, x, w, z, dy, act=act, res="before", kn=kn, back_ld=pad)
        d = dy.double() * ((z > 0).double() if act == "relu" else 1.0)
        wd = w.double().t() if kn else w.double()
        assert torch.equal(dx, (d @ wd).to(T[dtype]))
        want = d.t() @ x.double()
        assert torch.equal(dw, (want.t() if kn else want).to(T[dtype]))
        assert torch.equal(db, d.sum(0).to(T[dtype]))
        assert torch.equal(dr, d.to(T[dtype]))
    _, _, _, dr = backward(dtype, x, w, z, dy, act="relu", res="after", kn=kn, want="r")
    assert torch.equal(dr, dy)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_activations(act, dtype):
    m, n, k = 150, 77, 72
    g = gen(20 + ACTS.index(act))
    x, w = rnd(g, dtype, m, k), rnd(g, dtype, n, k, scale=k ** -0.5)
    z, dy = rnd(g, dtype, m, n, scale=2.0), rnd(g, dtype, m, n)
    z[0, :4] = torch.tensor([0.0, -0.0, 3.0, -3.0])  # corners
    z[1, :4] = torch.tensor([-0.75, 1.25, 2.5, -2.5])
    dx, dw, db, dr = backward(dtype, x, w, z, dy, act=act, res="before")
    xd, wd, v, g64 = x.double(), w.double(), z.double(), dy.double()
    d = g64 * act64(v, act)[1]
    # evaluation: 16 ulps of the slope's terms, at most 1 + |v| in size
    derr = 0 if act in ("identity", "relu", "clip", "leaky_relu") else 16 * U * g64.abs() * (1 + v.abs())
    derr = derr + U * d.abs()
    close("dr", dr, d, derr, dtype)
    sumerr = (m + 2) * U * d.abs().sum(0) + (derr + 0 * d).sum(0)
    close("db", db, d.sum(0), sumerr, dtype)
    rounded = derr + h(dtype) * d.abs() + TINY[dtype]
    close("dx", dx, d @ wd, rounded @ wd.abs() + (n + 2) * U * (d.abs() @ wd.abs()), dtype)
    close("dw", dw, d.t() @ xd, rounded.t() @ xd.abs() + (m + 2) * U * (d.abs().t() @ xd.abs()), dtype)


@pytest.mark.parametrize("want", ["x", "w", "b", "r", "xw", "wb"])
def test_linear_backward_parts(want):
    """Each gradient alone is what it is beside the others."""
    g = gen(2)
    x, w, z, dy = (whole(g, "f16", *s) for s in ((70, 24), (40, 24), (70, 40), (70, 40)))
    full = backward("f16", x, w, z, dy, act="relu", res="before")
    part = backward("f16", x, w, z, dy, act="relu", res="before", want=want)
    for name, f, p in zip("xwbr", full, part):
        assert (p is None) == (name not in want)
        assert p is None or torch.equal(f, p), name


def test_linear_gradient_in_place_and_strides():
    g = gen(4)
    x, w, z, dy = (whole(g, "bf16", *s) for s in ((70, 25), (41, 25), (70, 41), (70, 41)))
    dx, dw, db, dr = backward("bf16", x, w, z, dy, act="relu", res="before")
    (_, xv), (_, wv), (_, zv), (_, dyv) = (strided(t, 3, 1) for t in (x, w, z, dy))
    got = backward("bf16", xv, wv, zv, dyv, act="relu", res="before")
    for a, b in zip((dx, dw, db, dr), got):
        assert torch.equal(a, b)
    p = cf.make_linear_problem(70, 41, 25, act="relu", residual="before")
    size = cf.linear_backward_scratch_size(p, "bf16")
    buf, out = dy.clone(), torch.empty_like(dx)
    cf.linear_backward(p, "bf16", x, w, z, buf, out, None, None, buf, scratch(size), size, stream())
    assert torch.equal(buf, dr) and torch.equal(out, dx)


@pytest.mark.parametrize("act", ["tanh", "silu", "gelu", "gelu_tanh", "sigmoid"])
def test_linear_gradient_against_differences(act):
    """Central differences of the 64-bit definition, step d = 2^-13: their error is
    d^2 / 6 of a third derivative (below 4 in size for these sums), so 1e-6 of the
    terms' sizes covers it and the kernel's float32."""
    m, n, k = 5, 9, 13
    g = gen(11)
    x, w, b = rnd(g, "f32", m, k), rnd(g, "f32", n, k, scale=k ** -0.5), rnd(g, "f32", n)
    dy = rnd(g, "f32", m, n)
    _, z = forward("f32", x, w, b, act=act, save=True)
    dx, dw, db, _ = backward("f32", x, w, z, dy, act=act)

    def loss(xd, wd, bd):
        return (act64(xd @ wd.t() + bd, act)[0] * dy.double()).sum().item()

    ops = [x.double(), w.double(), b.double()]
    for i, got in enumerate((dx, dw, db)):
        flat = got.flatten()
        for e in range(0, flat.numel(), 3):
            d = 2.0 ** -13
            side = []
            for s in (d, -d):
                o = [t.clone() for t in ops]
                o[i].view(-1)[e] += s
                side.append(loss(*o))
            num = (side[0] - side[1]) / (2 * d)
            assert abs(num - flat[e].item()) <= 2e-6 * (m + n) * (1 + abs(num)), (i, e)


# ------------------------------------------------------------------------------ gated

def gated(dtype, x, wg, wu, bg=None, bu=None, act="silu", save=False, packed=False, h_out=None):
    m, k = x.shape
    f = wg.shape[0]
    a, be = PARAM.get(act, (0.0, 0.0))
    nan = lambda *s: torch.full(s, float("nan"), dtype=T[dtype], device="cuda")  # noqa: E731
    out = nan(m, f) if h_out is None else h_out
    pg = pu = None
    if save and packed:
        both = nan(m, 2 * f)
        pg, pu = both[:, :f], both[:, f:]
    elif save:
        pg, pu = nan(m, f), nan(m, f)
    p = cf.make_gated_problem(m, f, k, act=act, alpha=a, beta=be, bias=bg is not None, save=save,
                              ldx=x.stride(0), ldw=wg.stride(0), ldh=out.stride(0),
                              ldp=pg.stride(0) if save else 0)
    size = cf.gated_scratch_size(p, dtype)
    cf.gated_forward(p, dtype, x, wg, wu, bg, bu, out, pg, pu, scratch(size), size, stream())
    return (out, pg, pu) if save else out


GATED_SIZES = [(1, 1, 1), (1, 16, 64), (3, 50, 72), (16, 100, 129), (17, 33, 40), (32, 64, 2048),
               (33, 40, 64), (64, 65, 4096), (100, 130, 66), (129, 72, 200), (300, 520, 127),
               (4096, 2056, 80), (4090, 2100, 72)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,f,k", GATED_SIZES)
def test_gated_whole_numbers_are_exact(m, f, k, dtype):
    """Ranges that keep |pu| * |pg| below 2^24, so float32 holds the product."""
    g = gen(m + f + k)
    print(f"[gated exact] {m} {f} {k} {dtype}", flush=True)
    x, wg, wu = (whole(g, dtype, *s, lo=-1, hi=2) for s in ((m, k), (f, k), (f, k)))
    bg, bu = whole(g, dtype, f), whole(g, dtype, f)
    out, pg, pu = gated(dtype, x, wg, wu, bg, bu, act="relu", save=True, packed=m % 2 == 0)
    a = x.double() @ wg.double().t() + bg.double()
    b = x.double() @ wu.double().t() + bu.double()
    assert float((a.abs().max() * b.abs().max())) < 2 ** 24
    assert torch.equal(pg, a.to(T[dtype])) and torch.equal(pu, b.to(T[dtype]))
    assert torch.equal(out, (a.clamp(min=0) * b).to(T[dtype]))
    out = gated(dtype, x, wg, wu, act="identity")
    assert torch.equal(out, ((a - bg.double()) * (b - bu.double())).to(T[dtype]))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,f,k", [(3, 40, 96), (90, 72, 130)])
def test_gated_activations(m, f, k, act, dtype):
    g = gen(40 + ACTS.index(act))
    x, wg, wu = rnd(g, dtype, m, k), rnd(g, dtype, f, k, scale=2 * k ** -0.5), rnd(g, dtype, f, k, scale=k ** -0.5)
    bg, bu = rnd(g, dtype, f), rnd(g, dtype, f)
    out, pg, pu = gated(dtype, x, wg, wu, bg, bu, act=act, save=True)
    xd = x.double()
    a, b = xd @ wg.double().t() + bg.double(), xd @ wu.double().t() + bu.double()
    ae = (k + 2) * U * (xd.abs() @ wg.double().abs().t() + bg.double().abs())
    be = (k + 2) * U * (xd.abs() @ wu.double().abs().t() + bu.double().abs())
    close("pg", pg, a, ae, dtype)
    close("pu", pu, b, be, dtype)
    y = act64(a, act)[0]
    ye = act_error(a, y, ae, act)
    close("h", out, y * b, ye * b.abs() + be * y.abs() + ye * be + U * (y * b).abs(), dtype)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("m,f,k,pad,off", [(4, 48, 64, 8, 8), (4, 47, 61, 3, 1), (90, 72, 192, 16, 0),
                                           (90, 71, 191, 5, 3)])
def test_gated_strides(m, f, k, pad, off, dtype):
    g = gen(pad)
    x, wg, wu = (whole(g, dtype, *s, lo=-1, hi=2) for s in ((m, k), (f, k), (f, k)))
    (_, xv), (_, gv), (_, uv) = (strided(t, pad, off) for t in (x, wg, wu))
    hbuf, hv = strided(torch.zeros(m, f, dtype=T[dtype], device="cuda"), pad, off)
    gated(dtype, xv, gv, uv, act="relu", h_out=hv)
    want = (x.double() @ wg.double().t()).clamp(min=0) * (x.double() @ wu.double().t())
    assert torch.equal(hv, want.to(T[dtype]))
    hv.zero_()
    assert int(torch.isnan(hbuf).sum()) == hbuf.numel() - m * f


def gated_back(dtype, x, wg, wu, pg, pu, dh, act="silu", want="xwb"):
    m, k = x.shape
    f = wg.shape[0]
    a, be = PARAM.get(act, (0.0, 0.0))
    nan = lambda *s: torch.full(s, float("nan"), dtype=T[dtype], device="cuda")  # noqa: E731
    p = cf.make_gated_problem(m, f, k, act=act, alpha=a, beta=be, ldx=x.stride(0),
                              ldw=wg.stride(0), ldh=dh.stride(0), ldp=pg.stride(0))
    dx = nan(m, k) if "x" in want else None
    dwg, dwu = (nan(f, k) if "w" in want else None for _ in range(2))
    dbg, dbu = (nan(f) if "b" in want else None for _ in range(2))
    size = cf.gated_backward_scratch_size(p, dtype)
    cf.gated_backward(p, dtype, x, wg, wu, pg, pu, dh, dx, dwg, dwu, dbg, dbu, scratch(size), size,
                      stream())
    return dx, dwg, dwu, dbg, dbu


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,f,k", [(1, 1, 1), (1, 40, 64), (5, 17, 33), (64, 72, 40), (129, 65, 131),
                                   (200, 136, 264), (2000, 33, 64), (1030, 136, 264),
                                   (300, 2056, 4112), (4112, 2100, 72)])
def test_gated_backward_whole_numbers_are_exact(m, f, k, dtype):
    g = gen(m + f + k)
    print(f"[gated backward exact] {m} {f} {k} {dtype}", flush=True)
    x, wg, wu = (whole(g, dtype, *s) for s in ((m, k), (f, k), (f, k)))
    pg, pu, dh = (whole(g, dtype, m, f) for _ in range(3))
    dx, dwg, dwu, dbg, dbu = gated_back(dtype, x, wg, wu, pg, pu, dh, act="relu")
    dg = dh.double() * pu.double() * (pg > 0).double()
    du = dh.double() * pg.double().clamp(min=0)
    assert torch.equal(dx, (dg @ wg.double() + du @ wu.double()).to(T[dtype]))
    assert torch.equal(dwg, (dg.t() @ x.double()).to(T[dtype]))
    assert torch.equal(dwu, (du.t() @ x.double()).to(T[dtype]))
    assert torch.equal(dbg, dg.sum(0).to(T[dtype])) and torch.equal(dbu, du.sum(0).to(T[dtype]))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_gated_backward_activations(act, dtype):
    m, f, k = 140, 75, 64
    g = gen(60 + ACTS.index(act))
    x, wg, wu = rnd(g, dtype, m, k), rnd(g, dtype, f, k, scale=k ** -0.5), rnd(g, dtype, f, k, scale=k ** -0.5)
    pg, pu, dh = rnd(g, dtype, m, f, scale=2.0), rnd(g, dtype, m, f), rnd(g, dtype, m, f)
    dx, dwg, dwu, dbg, dbu = gated_back(dtype, x, wg, wu, pg, pu, dh, act=act)
    v, u, d = pg.double(), pu.double(), dh.double()
    y, slope = act64(v, act)
    dg, du = d * u * slope, d * y
    ev = 16 * U * (1 + v.abs())
    ge = d.abs() * u.abs() * ev + 2 * U * dg.abs()
    ue = d.abs() * ev + U * du.abs()
    close("dbg", dbg, dg.sum(0), (m + 2) * U * dg.abs().sum(0) + ge.sum(0), dtype)
    close("dbu", dbu, du.sum(0), (m + 2) * U * du.abs().sum(0) + ue.sum(0), dtype)
    gr, ur = ge + h(dtype) * dg.abs() + TINY[dtype], ue + h(dtype) * du.abs() + TINY[dtype]
    xa, wa, ua = x.double().abs(), wg.double().abs(), wu.double().abs()
    close("dx", dx, dg @ wg.double() + du @ wu.double(),
          gr @ wa + ur @ ua + (2 * f + 2) * U * (dg.abs() @ wa + du.abs() @ ua), dtype)
    close("dwg", dwg, dg.t() @ x.double(), gr.t() @ xa + (m + 2) * U * (dg.abs().t() @ xa), dtype)
    close("dwu", dwu, du.t() @ x.double(), ur.t() @ xa + (m + 2) * U * (du.abs().t() @ xa), dtype)


@pytest.mark.parametrize("want", ["x", "w", "b"])
def test_gated_backward_parts_and_packed(want):
    g = gen(9)
    x, wg, wu = (whole(g, "f16", *s) for s in ((70, 24), (41, 24), (41, 24)))
    both, dh = whole(g, "f16", 70, 82), whole(g, "f16", 70, 41)
    full = gated_back("f16", x, wg, wu, both[:, :41], both[:, 41:], dh, act="relu")
    part = gated_back("f16", x, wg, wu, both[:, :41].contiguous(), both[:, 41:].contiguous(), dh,
                      act="relu", want=want)
    for name, a, b in zip("xwwbb", full, part):
        assert (b is None) == (name != want)
        assert b is None or torch.equal(a, b)


def test_gated_no_rows():
    w = torch.zeros(8, 16, dtype=torch.float16, device="cuda")
    p = cf.make_gated_problem(0, 8, 16)
    cf.gated_forward(p, "f16", None, w, w.clone(), None, None, None)
    outs = [torch.full(s, 7.0, dtype=torch.float16, device="cuda") for s in ((8, 16), (8, 16), (8,), (8,))]
    size = cf.gated_backward_scratch_size(p, "f16")
    cf.gated_backward(p, "f16", None, w, w.clone(), None, None, None, None, *outs, scratch(size), size,
                      stream())
    assert not any(bool(o.any()) for o in outs)


@pytest.mark.parametrize("m", [3, 80])
def test_block_in_a_graph(m):
    """A block's forward and backward captured and replayed on new inputs, with
    eager work between the replays, against the eager calls."""
    f, k, dt = 136, 2048, "bf16"
    g = gen(13)
    wg, wu, wd = rnd(g, dt, f, k, scale=0.02), rnd(g, dt, f, k, scale=0.02), rnd(g, dt, k, f, scale=0.1)
    x, dy = torch.zeros(m, k, dtype=T[dt], device="cuda"), torch.zeros(m, k, dtype=T[dt], device="cuda")
    gp = cf.make_gated_problem(m, f, k, save=True)
    lp = cf.make_linear_problem(m, k, f, residual="after")
    e = lambda *s: torch.empty(s, dtype=T[dt], device="cuda")  # noqa: E731
    hid, pg, pu, y = e(m, f), e(m, f), e(m, f), e(m, k)
    dh, dwd, dx, dwg, dwu = e(m, f), e(k, f), e(m, k), e(f, k), e(f, k)
    size = max(cf.gated_scratch_size(gp, dt), cf.linear_scratch_size(lp, dt),
               cf.linear_backward_scratch_size(lp, dt), cf.gated_backward_scratch_size(gp, dt))
    ws = scratch(size)

    def step():
        s = stream()
        cf.gated_forward(gp, dt, x, wg, wu, None, None, hid, pg, pu, ws, size, s)
        cf.linear_forward(lp, dt, hid, wd, None, x, y, None, ws, size, s)
        cf.linear_backward(lp, dt, hid, wd, None, dy, dh, dwd, None, None, ws, size, s)
        cf.gated_backward(gp, dt, x, wg, wu, pg, pu, dh, dx, dwg, dwu, None, None, ws, size, s)

    outs = (y, dwd, dx, dwg, dwu)
    graph = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(rnd(g, dt, m, k))
        dy.copy_(rnd(g, dt, m, k))
        step()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), i
